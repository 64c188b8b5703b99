// INT8 product, the consumer of the symmetric INT8 codes (page "14. 量化：让每一步
// 搬更少的字节", 量化在做什么: q = round(x / s) of activations and weights, their
// products summed as integers and scaled once):
//
//   C[m, n] = ((float(S) * sA[m]) * sB[n]) + bias[n],   S = sum_k a[m, k] b[n, k],
//
// S exact in int32 (K <= 131071 keeps |S| <= 2^14 K below 2^31), so neither the
// order of the sum nor a split of K changes a bit of C.
//
// A workgroup owns a kTM x kTN tile; both operands' kBK = 128 bytes of K go straight
// from global memory into LDS (buffer_load_dwordx4 ... lds) in a ring of two slots,
// the next block's while this one is multiplied.  A row is 8 chunks of 16 bytes, chunk c
// of row r at position c ^ (r & 7): the 8 lanes that read one chunk of 8 rows touch 8
// different groups of banks.  A lane whose row or chunk lies outside the matrix
// gives the load an offset past the buffer's end, which reads as zeros.
// v_mfma_i32_32x32x32_i8 takes the weights as its first operand: lane l holds row l & 31
// and the 16 bytes of chunk l >> 5; result register r is weight row
// 8 (r / 4) + 4 (l >> 5) + r % 4 of activation row l & 31.
#include "launch.h"
#include "quant.h"

namespace pqb {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

constexpr int kBK = 128;                  // bytes of K per block
constexpr uint32_t kOutside = 0x80000000u;  // a buffer's size, and an offset past it

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) void*)p);
}

// Raw buffer of kOutside bytes at a wave-uniform address.
__device__ __forceinline__ v4i buffer_at(const void* p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  return v4i{__builtin_amdgcn_readfirstlane((int)(uint32_t)u),
             __builtin_amdgcn_readfirstlane((int)((uint32_t)(u >> 32) & 0xFFFFu)), (int)kOutside, 0x00020000};
}

// Wave-wide DMA of 16 bytes per lane from buffer + soff + off to LDS address lds + 16 l.
__device__ __forceinline__ void dma16(v4i buf, uint32_t off, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(off), "s"(buf),
               "s"(soff), "s"(lds)
               : "memory");
}

template <int kN>
__device__ __forceinline__ void wait_vmcnt() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kN) : "memory");
}
// With this wave's LDS reads done: another wave may overwrite what they read.
__device__ __forceinline__ void barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// LDS written by some lanes of a wave and read by others.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Tile (tm, tn) of workgroup t of tiles_m x tiles_n: workgroups i, i + 8, ... share an
// XCD and its L2, and take a contiguous run of tiles down bands of kBand tile rows.
template <int kBand>
__device__ __forceinline__ void tile_of(int tiles_m, int tiles_n, int& tm, int& tn) {
  const int nwg = tiles_m * tiles_n, xcd = blockIdx.x & 7, per = nwg >> 3, more = nwg & 7;
  const int t = xcd * per + min(xcd, more) + (blockIdx.x >> 3);
  const int band = t / (kBand * tiles_n), rem = t - band * kBand * tiles_n;
  const int rows = min(kBand, tiles_m - band * kBand);
  tn = rem / rows;
  tm = band * kBand + rem - tn * rows;
}

// Eight results of row m from column n on (n % 8 == 0).
template <bool kBf16>
__device__ __forceinline__ void store_out8(void* c, int64_t m, int n, int N, const float (&v)[8]) {
  if (N % 8 == 0) {
    if (n >= N) return;
    if constexpr (kBf16) {
      st_nt16(reinterpret_cast<uint16_t*>(c) + m * N + n, bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]),
              bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7]));
    } else {
      float* p = reinterpret_cast<float*>(c) + m * N + n;
      st_nt16(p, as_u(v[0]), as_u(v[1]), as_u(v[2]), as_u(v[3]));
      st_nt16(p + 4, as_u(v[4]), as_u(v[5]), as_u(v[6]), as_u(v[7]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (n + j < N) {
        if constexpr (kBf16)
          reinterpret_cast<uint16_t*>(c)[m * N + n + j] = (uint16_t)(bf16x2_rne(v[j], 0.0f) & 0xFFFFu);
        else
          reinterpret_cast<float*>(c)[m * N + n + j] = v[j];
      }
  }
}

// Scales and bias of eight columns from n on, 0 behind the last.
struct Columns {
  float s[8], b[8];
};
__device__ __forceinline__ Columns columns_at(const Int8Args& g, int n) {
  Columns c;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool in = n + j < g.N;
    c.s[j] = in ? g.b_scales[(int64_t)(n + j) * g.b_step] : 0.0f;
    c.b[j] = in && g.bias ? g.bias[n + j] : 0.0f;
  }
  return c;
}
__device__ __forceinline__ void scaled(const int (&x)[8], float sa, const Columns& c, bool bias, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = (float)x[j] * sa * c.s[j];
    if (bias) v[j] += c.b[j];
  }
}

template <int kTM, int kTN, int kWM, int kWN>
struct Tile {
  static constexpr int waves = kWM * kWN, threads = 64 * waves;
  static constexpr int mt = kTM / kWM / 32, nt = kTN / kWN / 32;     // 32 x 32 products of a wave
  static constexpr int slot = (kTM + kTN) * kBK;
  static constexpr int stage_ld = 32 * nt + 4;                       // ints per staged row
  static constexpr int stage = waves * 32 * stage_ld * 4;
  static constexpr int lds = 2 * slot > stage ? 2 * slot : stage;
  static constexpr int a_loads = kTM / 8 / waves, b_loads = kTN / 8 / waves;
  static_assert(a_loads * 8 * waves == kTM && b_loads * 8 * waves == kTN && nt == 2, "tile shape");
};

template <int kTM, int kTN, int kWM, int kWN, bool kBf16>
__global__ __launch_bounds__(64 * kWM * kWN) void k_gemm_int8(Int8Args g, int tiles_m, int tiles_n) {
  using S = Tile<kTM, kTN, kWM, kWN>;
  __shared__ __align__(16) uint8_t lds[S::lds];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tm, tn;
  tile_of<1024 / kTM>(tiles_m, tiles_n, tm, tn);
  const int m0 = tm * kTM, n0 = tn * kTN;
  const int nkb = (g.K + kBK - 1) / kBK;

  // Instruction j of a wave fills rows 8 (j waves + wave) .. + 7 of a tile
  const int drow = lane >> 3, chunk = (lane & 7) ^ drow;
  const v4i buf_a = buffer_at(g.a + (int64_t)m0 * g.a_stride), buf_b = buffer_at(g.b + (int64_t)n0 * g.b_stride);
  uint32_t off_a[S::a_loads], off_b[S::b_loads];
#pragma unroll
  for (int j = 0; j < S::a_loads; ++j) {
    const int r = (j * S::waves + wave) * 8 + drow;
    off_a[j] = m0 + r < g.M ? (uint32_t)r * (uint32_t)g.a_stride + 16u * chunk : kOutside;
  }
#pragma unroll
  for (int j = 0; j < S::b_loads; ++j) {
    const int r = (j * S::waves + wave) * 8 + drow;
    off_b[j] = n0 + r < g.N ? (uint32_t)r * (uint32_t)g.b_stride + 16u * chunk : kOutside;
  }
  const uint32_t base = __builtin_amdgcn_readfirstlane(lds_addr(lds) + wave * 1024);
  auto issue = [&](int kb) {
    const bool out = kb * kBK + 16 * chunk >= g.K;                   // behind the last chunk of K
    const uint32_t to = base + (kb & 1) * S::slot;
#pragma unroll
    for (int j = 0; j < S::a_loads; ++j)
      dma16(buf_a, out ? kOutside : off_a[j], kb * kBK, to + j * S::waves * 1024);
#pragma unroll
    for (int j = 0; j < S::b_loads; ++j)
      dma16(buf_b, out ? kOutside : off_b[j], kb * kBK, to + kTM * kBK + j * S::waves * 1024);
  };

  const int wm = wave / kWN * (32 * S::mt), wn = wave % kWN * (32 * S::nt);
  const int r32 = lane & 31, up = lane >> 5;
  v16i acc[S::mt][S::nt];
#pragma unroll
  for (int i = 0; i < S::mt; ++i)
#pragma unroll
    for (int j = 0; j < S::nt; ++j) acc[i][j] = v16i{};

  if (nkb > 0) issue(0);
  for (int kb = 0; kb < nkb; ++kb) {
    wait_vmcnt<0>();
    barrier();
    if (kb + 1 < nkb) issue(kb + 1);
    const uint8_t* sl = lds + (kb & 1) * S::slot;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int at = ((2 * s + up) ^ (r32 & 7)) << 4;
      v4i a[S::mt], b[S::nt];
#pragma unroll
      for (int i = 0; i < S::mt; ++i)
        a[i] = *reinterpret_cast<const v4i*>(sl + (wm + 32 * i + r32) * kBK + at);
#pragma unroll
      for (int j = 0; j < S::nt; ++j)
        b[j] = *reinterpret_cast<const v4i*>(sl + (kTM + wn + 32 * j + r32) * kBK + at);
#pragma unroll
      for (int i = 0; i < S::mt; ++i)
#pragma unroll
        for (int j = 0; j < S::nt; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b[j], a[i], acc[i][j], 0, 0, 0);
    }
  }
  barrier();   // every wave done with the ring before it becomes the output stage

  // 32 rows at a time through the wave's part of LDS, then eight columns a lane
  int* out = reinterpret_cast<int*>(lds) + wave * 32 * S::stage_ld;
  const int n = n0 + wn + 8 * (lane & 7);
  const Columns cols = columns_at(g, n);
#pragma unroll
  for (int i = 0; i < S::mt; ++i) {
#pragma unroll
    for (int j = 0; j < S::nt; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *reinterpret_cast<v4i*>(out + r32 * S::stage_ld + 32 * j + 8 * r + 4 * up) =
            v4i{acc[i][j][4 * r], acc[i][j][4 * r + 1], acc[i][j][4 * r + 2], acc[i][j][4 * r + 3]};
    wave_sync();
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int row = 8 * s + (lane >> 3), m = m0 + wm + 32 * i + row;
      int x[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const v4i y = *reinterpret_cast<const v4i*>(out + row * S::stage_ld + 8 * (lane & 7) + 4 * h);
        x[4 * h] = y[0], x[4 * h + 1] = y[1], x[4 * h + 2] = y[2], x[4 * h + 3] = y[3];
      }
      if (m < g.M) {
        float v[8];
        scaled(x, g.a_scales[(int64_t)m * g.a_step], cols, g.bias != nullptr, v);
        store_out8<kBf16>(g.c, m, n, g.N, v);
      }
    }
    wave_sync();
  }
}

template <int kTM, int kTN, int kWM, int kWN>
hipError_t launch_tile(const Int8Args& g, bool out_bf16, hipStream_t st) {
  const int tiles_m = (g.M + kTM - 1) / kTM, tiles_n = (g.N + kTN - 1) / kTN;
  const uint32_t grid = (uint32_t)tiles_m * (uint32_t)tiles_n;
  if (out_bf16) k_gemm_int8<kTM, kTN, kWM, kWN, true><<<grid, 64 * kWM * kWN, 0, st>>>(g, tiles_m, tiles_n);
  else k_gemm_int8<kTM, kTN, kWM, kWN, false><<<grid, 64 * kWM * kWN, 0, st>>>(g, tiles_m, tiles_n);
  return hipGetLastError();
}

}  // namespace

size_t gemm_int8_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_gemm_int8(Int8Args g, bool out_bf16, void*, hipStream_t st) {
  return launch_tile<128, 128, 2, 2>(g, out_bf16, st);
}

}  // namespace pqb
