// INT8 product, the consumer of the symmetric INT8 codes (page "14. 量化：让每一步
// 搬更少的字节", 量化在做什么: q = round(x / s) of activations and weights, their
// products summed as integers and scaled once):
//
//   C[m, n] = ((float(S) * sA[m]) * sB[n]) + bias[n],   S = sum_k a[m, k] b[n, k],
//
// S exact in int32 (K <= 131056 keeps |S| <= 2^14 K below 2^31), so neither the
// order of the sum nor how K is shared out changes a bit of C.
//
// Both operands' blocks of K go straight from global memory into LDS
// (buffer_load_dwordx4 ... lds, issued from inline assembly and waited for with explicit
// counts: the compiler would wait for all of them before every LDS read).  A lane whose
// row or chunk lies outside the matrix gives the load an offset past the buffer's end,
// which reads as zeros.  Rows in LDS are chunks of 16 bytes, permuted by row so that the 16
// lanes which read one chunk of 16 rows touch all 64 banks once.
// v_mfma_i32_16x16x64_i8 takes the weights as its first operand: lane l holds row l & 15
// and chunk l >> 4 of 64 bytes of K, and result register r is weight row 4 (l >> 4) + r of
// activation row l & 15, so that a lane has four columns of one row of C.  (Its loop of random
// operands runs at 3.8-4.1 POP/s here, the 32x32x32 product's at 3.4-3.5: power.)
//
// Two kernels: k_int8_ring where the matrices are read about once (decode steps, chunks),
// k_int8_tile where they are read often.
#include <algorithm>

#include "int8_tiles.h"
#include "launch.h"
#include "quant.h"

namespace pqb {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

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

// Tile (tm, tn) of number t: down bands of kBand tile rows, so that tiles of neighbouring
// numbers share rows of A and of B.
template <int kBand>
__device__ __forceinline__ void tile_at(int t, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int band = t / (kBand * tiles_n), rem = t - band * kBand * tiles_n;
  const int rows = min(kBand, tiles_m - band * kBand);
  tn = rem / rows;
  tm = band * kBand + rem - tn * rows;
}

enum Out { kF32 = 0, kBf16 = 1 };

typedef float v4f __attribute__((ext_vector_type(4)));

// Rows of C that are whole lines are stored with the streaming hint: 8192 x 8192 of 64, bf16, 41
// us, 49 without.  Others share lines and go without it, up to 16 bytes at the alignment of a
// result (8192 x 8200 54 us, 73 with it; one by one 6826 x 5735 of 48 65 us, 48 so).  (The larger
// tiles' float32 rows gain by it from 64 bytes on: 4614 x 12208 of 592 81 us, 91 without.)
template <int kOut>
__device__ __forceinline__ bool whole_lines(int N) { return N % (kOut == kBf16 ? 64 : 32) == 0; }

template <bool kLines, int kWords>
__device__ __forceinline__ void store_words(void* p, const uint32_t* w) {
  if constexpr (kWords > 4) {
    store_words<kLines, 4>(p, w);
    store_words<kLines, kWords - 4>(reinterpret_cast<uint32_t*>(p) + 4, w + 4);
  } else if constexpr (kLines && kWords == 4) {
    st_nt16(p, w[0], w[1], w[2], w[3]);
  } else {
    typedef uint32_t words __attribute__((ext_vector_type(kWords), aligned(2)));
    words x;
#pragma unroll
    for (int j = 0; j < kWords; ++j) x[j] = w[j];
    *reinterpret_cast<words*>(p) = x;
  }
}

// kV results of row m from column n on, those in front of N.
template <int kOut, bool kLines, int kV>
__device__ __forceinline__ void store_out(void* c, int64_t m, int n, int N, const float (&v)[kV]) {
  const bool all = kLines || n + kV <= N;
  if constexpr (kOut == kBf16) {
    uint16_t* p = reinterpret_cast<uint16_t*>(c) + m * N + n;
    uint32_t w[(kV + 1) / 2];
#pragma unroll
    for (int j = 0; j < kV; j += 2) w[j / 2] = bf16x2_rne(v[j], v[j + 1 < kV ? j + 1 : j]);
    if (kV > 1 && all) store_words<kLines, (kV + 1) / 2>(p, w);
    else
#pragma unroll
      for (int j = 0; j < kV; ++j)
        if (n + j < N) p[j] = (uint16_t)(w[j / 2] >> (j & 1) * 16);
  } else {
    float* p = reinterpret_cast<float*>(c) + m * N + n;
    if (kV > 1 && all) {
      uint32_t w[kV];
#pragma unroll
      for (int j = 0; j < kV; ++j) w[j] = as_u(v[j]);
      store_words<kLines, kV>(p, w);
    } else {
#pragma unroll
      for (int j = 0; j < kV; ++j)
        if (n + j < N) p[j] = v[j];
    }
  }
}

// p[n .. n + kN - 1] (p[0] with step 0), 0 at and behind N; at most four.
template <int kN>
__device__ __forceinline__ auto some_at(const float* p, int step, int n, int N) {
  typedef float some __attribute__((ext_vector_type(kN)));
  typedef float any __attribute__((ext_vector_type(kN), aligned(4)));
  some v{};
  if (step == 0) {
#pragma unroll
    for (int j = 0; j < kN; ++j) v[j] = p[0];
  } else if (n + kN <= N) {
    v = *reinterpret_cast<const any*>(p + n);
  } else {
#pragma unroll
    for (int j = 0; j < kN - 1; ++j)
      if (n + j < N) v[j] = p[n + j];
  }
  return v;
}

template <int kTM, int kTN, int kWM, int kWN>
struct Tile {
  static constexpr int waves = kWM * kWN;
  static constexpr int mt = kTM / kWM / 16, nt = kTN / kWN / 16;     // 16 x 16 products of a wave
  static constexpr int slot = (kTM + kTN) * kBK;
  static constexpr int stage = 4096;                                 // bytes of a wave's staged results
  static constexpr int lds = 2 * slot + waves * stage;
  static constexpr int a_loads = kTM / 8 / waves, b_loads = kTN / 8 / waves;
  static_assert(a_loads * 8 * waves == kTM && b_loads * 8 * waves == kTN && nt == 4 && mt % 2 == 0, "tile shape");
  static_assert(a_loads <= mt && b_loads <= mt, "one load of each operand per row of products at most");
};

// Many tiles.  A wave's products of one half of a 128-byte block run while its fragments of
// the next are read and, behind the barrier, the next but one block is loaded: reads, loads and
// products issue one between the other (left to the compiler, every read was waited for at
// once: 8192^3 445 us, 435 so).  Chunk c of row r lies at c ^ (r / 2); at c ^ r the 16 rows met in
// pairs, half of the LDS cycles.  Workgroups stay and take tiles in turn, and the blocks of
// all their tiles are one stream: before a tile's results are scaled, the next tile's first block is in
// LDS, its first fragments in registers, and its second block on its way; the results' stores drain while
// the first is multiplied (8192 x 7168 x 2048 142 to 122 us).  (Scales and bias are loaded behind that
// second block, and loads return in order, so the first result waits for it.)  256 x 256 tiles, 8 waves of 128 x 64: 8192^3 in 410-425 us, 2.6 POP/s (the
// vendor's 521); the same without its loads 354, without LDS reads too 314: what is left is
// the operand stream and the clock that the power leaves (2.0 GHz).  These tiles take all 256 registers, and
// 9 more (6 for float32 results) that are spilled and read again between tiles, not in the loop over K.
template <int kTM, int kTN, int kWM, int kWN, int kOut>
__global__ __launch_bounds__(64 * kWM * kWN) void k_int8_tile(Int8Args g, int tiles_m, int tiles_n) {
  using S = Tile<kTM, kTN, kWM, kWN>;
  __shared__ __align__(16) uint8_t lds[S::lds];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nkb = max((g.K + kBK - 1) / kBK, 1);
  // Workgroups i, i + 8, ... share an XCD and its L2: they take a contiguous run of tiles
  const int all = tiles_m * tiles_n, xcd = blockIdx.x & 7, per = all >> 3, more = all & 7;
  const int stride = ((int)gridDim.x - xcd + 7) >> 3;
  const int end = (xcd + 1) * per + min(xcd + 1, more);
  int tile = xcd * per + min(xcd, more) + (blockIdx.x >> 3);

  auto place = [&](int t, int& m0, int& n0) {
    tile_at<1024 / kTM>(t, tiles_m, tiles_n, m0, n0);
    m0 *= kTM;
    n0 *= kTN;
  };

  // The stream's next block: kb_in of tile tile_in.  Instruction j of a wave fills rows
  // 8 (j waves + wave) .. + 7 of a tile.
  const int drow = lane >> 3, chunk = (lane & 7) ^ ((drow >> 1) | (wave & 1) << 2);
  int tile_in = tile, kb_in = 0;
  v4i buf_a, buf_b;
  uint32_t off_a[S::a_loads], off_b[S::b_loads];
  auto enter = [&]() {
    int m0 = 0, n0 = 0;
    if (tile_in < end) place(tile_in, m0, n0);
    const int rows_a = tile_in < end ? g.M - m0 : 0, rows_b = tile_in < end ? g.N - n0 : 0;
    buf_a = buffer_at(g.a + (int64_t)m0 * g.a_stride);
    buf_b = buffer_at(g.b + (int64_t)n0 * g.b_stride);
#pragma unroll
    for (int j = 0; j < S::a_loads; ++j) {
      const int r = (j * S::waves + wave) * 8 + drow;
      off_a[j] = r < rows_a ? (uint32_t)r * (uint32_t)g.a_stride + 16u * chunk : kOutside;
    }
#pragma unroll
    for (int j = 0; j < S::b_loads; ++j) {
      const int r = (j * S::waves + wave) * 8 + drow;
      off_b[j] = r < rows_b ? (uint32_t)r * (uint32_t)g.b_stride + 16u * chunk : kOutside;
    }
  };
  const uint32_t base = __builtin_amdgcn_readfirstlane(lds_addr(lds) + wave * 1024);
  auto issue_a = [&](int slot, int j) {
    const bool out = kb_in * kBK + 16 * chunk >= g.K;                // behind the last chunk of K
    dma16(buf_a, out ? kOutside : off_a[j], kb_in * kBK, base + slot * S::slot + j * S::waves * 1024);
  };
  auto issue_b = [&](int slot, int j) {
    const bool out = kb_in * kBK + 16 * chunk >= g.K;
    dma16(buf_b, out ? kOutside : off_b[j], kb_in * kBK, base + slot * S::slot + kTM * kBK + j * S::waves * 1024);
  };
  auto advance = [&]() {
    if (++kb_in < nkb) return;
    kb_in = 0;
    tile_in += stride;
    enter();
  };

  const int wm = wave / kWN * (16 * S::mt), wn = wave % kWN * (16 * S::nt);
  const int r16 = lane & 15, quarter = lane >> 4;
  v4i acc[S::mt][S::nt];
  // Fragments of 64 bytes of K (half s of a block).  Those of A are read for the next half as
  // soon as their products of this one are issued, those of B into a second set.
  v4i a[S::mt], b[2][S::nt];
  const int row_a = (wm + r16) * kBK, row_b = (kTM + wn + r16) * kBK;
  auto read_a = [&](int slot, int s, int i) {
    a[i] = *reinterpret_cast<const v4i*>(lds + slot * S::slot + row_a + 16 * i * kBK +
                                         (((4 * s + quarter) ^ (r16 >> 1)) << 4));
  };
  auto read_b = [&](int slot, int s, int j) {
    b[s][j] = *reinterpret_cast<const v4i*>(lds + slot * S::slot + row_b + 16 * j * kBK +
                                            (((4 * s + quarter) ^ (r16 >> 1)) << 4));
  };

  enter();
#pragma unroll
  for (int t = 0; t < 2; ++t) {
#pragma unroll
    for (int j = 0; j < S::a_loads; ++j) issue_a(t, j);
#pragma unroll
    for (int j = 0; j < S::b_loads; ++j) issue_b(t, j);
    advance();
  }
  wait_vmcnt<S::a_loads + S::b_loads>();
  barrier();
#pragma unroll
  for (int j = 0; j < S::nt; ++j) read_b(0, 0, j);
#pragma unroll
  for (int i = 0; i < S::mt; ++i) read_a(0, 0, i);

  // A wave's stores of a whole tile.  The vector memory counter counts down in order, and they
  // are behind the loads of the block that the next wait is for, so it need not be for them.
  constexpr int kRows = kOut == kBf16 ? 32 : 16, kStores = 16 * S::mt / kRows * 4;
  bool stored = false;
  int slot = 0;
  for (;;) {
#pragma unroll
    for (int i = 0; i < S::mt; ++i)
#pragma unroll
      for (int j = 0; j < S::nt; ++j) acc[i][j] = v4i{};
    for (int kb = 0; kb < nkb; ++kb) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (s == 1) {
          // The next block has landed for every wave, and every wave has read this one: the
          // next but one takes its slot (blocks behind the last tile read no memory)
          if (stored) wait_vmcnt<kStores>();
          else wait_vmcnt<0>();
          stored = false;
          barrier();
        }
#pragma unroll
        for (int i = 0; i < S::mt; ++i) {
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int j = 0; j < S::nt; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[s][j], a[i], acc[i][j], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
          if (i < S::nt) read_b(slot ^ s, s ^ 1, i);
          read_a(slot ^ s, s ^ 1, i);
          if (s == 1) {
            if (i < S::a_loads) issue_a(slot, i);
            if (i >= S::mt - S::b_loads) issue_b(slot, i - (S::mt - S::b_loads));
          }
        }
      }
      advance();
      slot ^= 1;
    }

    int m0, n0;
    place(tile, m0, n0);
    m0 += wm;
    n0 += wn;
    v4f sb[S::nt];
    float sa[S::mt];
#pragma unroll
    for (int j = 0; j < S::nt; ++j) sb[j] = some_at<4>(g.b_scales, g.b_step, n0 + 16 * j + 4 * quarter, g.N);
#pragma unroll
    for (int i = 0; i < S::mt; ++i)
      sa[i] = g.a_scales[(int64_t)min(m0 + 16 * i + r16, g.M - 1) * g.a_step];
    // kRows rows of 64 results at a time through the wave's own part of LDS, then 16 bytes a
    // lane; 16-byte chunk c of row r at c ^ r, so that rows meet in no bank
    uint8_t* out = lds + 2 * S::slot + wave * S::stage;
    constexpr int kChunks = kOut == kBf16 ? 8 : 16, kEach = 64 / kChunks;   // chunks of a row, results of a chunk
    const bool whole = m0 + 16 * S::mt <= g.M && n0 + 64 <= g.N && (kOut == kBf16 ? whole_lines<kOut>(g.N) : g.N % 16 == 0);
#pragma unroll
    for (int i = 0; i < S::mt; i += kRows / 16) {
#pragma unroll
      for (int h = 0; h < kRows / 16; ++h)
#pragma unroll
        for (int j = 0; j < S::nt; ++j) {
          float v[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = (float)acc[i + h][j][r] * sa[i + h] * sb[j][r];
          if (g.bias) {   // (read again for every row: held, its 16 registers spilled others)
            const v4f bias = some_at<4>(g.bias, 1, n0 + 16 * j + 4 * quarter, g.N);
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] += bias[r];
          }
          const int row = 16 * h + r16;
          if constexpr (kOut == kBf16)
            *reinterpret_cast<uint2*>(out + row * 128 + (((2 * j + (quarter >> 1)) ^ (row & 7)) << 4) +
                                      8 * (quarter & 1)) = make_uint2(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]));
          else
            *reinterpret_cast<v4f*>(out + row * 256 + (((4 * j + quarter) ^ row) << 4)) = v4f{v[0], v[1], v[2], v[3]};
        }
      wave_sync();
      if (whole) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int row = s * (kRows / 4) + lane / kChunks, c = lane % kChunks;
          const uint4 x = *reinterpret_cast<const uint4*>(out + row * (kChunks * 16) + ((c ^ (row & (kChunks - 1))) << 4));
          st_nt16(reinterpret_cast<uint8_t*>(g.c) + ((int64_t)(m0 + 16 * i + row) * g.N + n0 + kEach * c) * (16 / kEach),
                  x.x, x.y, x.z, x.w);
        }
      } else {
        const int rows = min(kRows, g.M - m0 - 16 * i), c = lane % kChunks, most = g.N - n0 - kEach * c;
        for (int row = lane / kChunks; row < rows; row += kRows / 4) {
          const uint8_t* x = out + row * (kChunks * 16) + ((c ^ (row & (kChunks - 1))) << 4);
          uint8_t* at = reinterpret_cast<uint8_t*>(g.c) + ((int64_t)(m0 + 16 * i + row) * g.N + n0 + kEach * c) * (16 / kEach);
          if (most >= kEach) {
            const uint4 w = *reinterpret_cast<const uint4*>(x);
            const uint32_t words[4] = {w.x, w.y, w.z, w.w};
            store_words<false, 4>(at, words);
          } else {
            for (int j = 0; j < most; ++j) {
              if constexpr (kOut == kBf16) reinterpret_cast<uint16_t*>(at)[j] = reinterpret_cast<const uint16_t*>(x)[j];
              else reinterpret_cast<uint32_t*>(at)[j] = reinterpret_cast<const uint32_t*>(x)[j];
            }
          }
        }
      }
      wave_sync();
    }
    stored = whole;
    tile += stride;
    if (tile >= end) break;
  }
  wait_vmcnt<0>();   // no load into LDS outlives the workgroup
}

// ---------------------------------------------------------------------------
// Few rows of A (decode steps), and few tiles: what is read once streams through LDS.
// A workgroup owns kTM rows of A (zeros behind the last) and kTN rows of B, few enough
// that the workgroups fill the chip, and its 8 waves share them out: kWM x kWN over the
// products, the rest over the blocks' K, whose sums meet in LDS at the end.  Blocks of kBK
// bytes of K pass through a ring of as many slots as fit: what memory latency asks to be
// in flight.  A row of a block is kBK / 16 chunks, chunk c of row r at c ^ mix(r).  (Straight
// from global memory into registers, 64 rows over 14336 channels of 4096 took 23 us, 12 so:
// a fragment's rows are 64-byte pieces, and each line was fetched twice.)  One row over 4096
// channels of 14336 from HBM 12.7 us, 4.6 TB/s; 64 over 14336 of 4096 16 us from HBM, 12 from
// the Infinity Cache (5 TB/s).
// ---------------------------------------------------------------------------
template <int kTM, int kTN, int kBK, int kWM, int kWN, int kPer>
struct Ring {
  static constexpr int waves = 8, wk = waves / kWM / kWN;
  static constexpr int mt = kTM / 16 / kWM, nt = kTN / 16 / kWN, steps = kBK / 64 / wk;
  static constexpr int chunks = kBK / 16, rows = 64 / chunks;   // of one DMA instruction
  static constexpr int slot = (kTM + kTN) * kBK;
  static constexpr int loads = slot / 1024 / waves;
  static constexpr int most = 163840 / kPer / slot, slots = most < 8 ? most : 8;
  static constexpr int ld = kTN + 4, sums = wk * kTM * ld * 4;
  static constexpr int most_cols = kTM * kTN / 512, cols = most_cols < 1 ? 1 : most_cols < 8 ? most_cols : 8;
  static constexpr int lds = slots * slot > sums ? slots * slot : sums;
  static_assert(wk * kWM * kWN == waves && mt * kWM * 16 == kTM && nt * kWN * 16 == kTN, "waves");
  static_assert(steps * wk * 64 == kBK && loads * waves * 1024 == slot && slots >= 3, "blocks");
  static_assert(lds * kPer <= 163840 && (slots - 2) * loads < 64, "LDS and the load counter");
  static __device__ __forceinline__ int mix(int r) { return chunks >= 16 ? r & 15 : r >> 1 & 7; }
};

template <int kTM, int kTN, int kBK, int kWM, int kWN, int kPer, int kOut>
__global__ __launch_bounds__(512, 2 * kPer) void k_int8_ring(Int8Args g, int inner, bool along_n) {
  using S = Ring<kTM, kTN, kBK, kWM, kWN, kPer>;
  __shared__ __align__(16) uint8_t lds[S::lds];
  const int lane = threadIdx.x & 63, r16 = lane & 15, quarter = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Workgroups of one XCD take tiles in turn that share their rows of the larger matrix
  const int nwg = gridDim.x, xcd = blockIdx.x & 7, per = nwg >> 3, more = nwg & 7;
  const int tile = xcd * per + min(xcd, more) + (blockIdx.x >> 3);
  const int shared = tile / inner, other = tile - shared * inner;
  const int m0 = (along_n ? shared : other) * kTM, n0 = (along_n ? other : shared) * kTN;
  const int nkb = (g.K + kBK - 1) / kBK;

  // Instruction j of a wave fills rows (j waves + wave) S::rows ... of [A | B]
  const v4i buf_a = buffer_at(g.a + (int64_t)m0 * g.a_stride), buf_b = buffer_at(g.b + (int64_t)n0 * g.b_stride);
  uint32_t off[S::loads];
  int chunk[S::loads];
#pragma unroll
  for (int j = 0; j < S::loads; ++j) {
    const int r = (j * S::waves + wave) * S::rows + lane / S::chunks;
    chunk[j] = (lane % S::chunks) ^ S::mix(r);
    const bool in = r < kTM ? m0 + r < g.M : n0 + r - kTM < g.N;
    const uint32_t at = r < kTM ? (uint32_t)r * (uint32_t)g.a_stride : (uint32_t)(r - kTM) * (uint32_t)g.b_stride;
    off[j] = in ? at + 16u * chunk[j] : kOutside;
  }
  const uint32_t base = __builtin_amdgcn_readfirstlane(lds_addr(lds) + wave * 1024);
  // Workgroups start at different blocks: rows that lie a power of two apart would all be read from
  // the same few memory channels at a time (16 rows over 28672 channels of 4096 26 to 24 us).
  const int turn = nkb ? shared % nkb : 0;
  auto issue = [&](int kb, int slot) {
    const int at = kb + turn, k = kb < nkb ? (at < nkb ? at : at - nkb) * kBK : g.K;
#pragma unroll
    for (int j = 0; j < S::loads; ++j) {
      const bool of_a = (j * S::waves + wave) * S::rows < kTM;
      dma16(of_a ? buf_a : buf_b, k + 16 * chunk[j] >= g.K ? kOutside : off[j], k,
            base + slot * S::slot + j * S::waves * 1024);
    }
  };

  const int wn = wave % kWN, wm = wave / kWN % kWM, part = wave / (kWN * kWM);
  v4i acc[S::mt][S::nt];
#pragma unroll
  for (int i = 0; i < S::mt; ++i)
#pragma unroll
    for (int j = 0; j < S::nt; ++j) acc[i][j] = v4i{};
  // The fragments of one block are read from LDS while the ones before it are multiplied
  v4i a[2][S::steps][S::mt], b[2][S::steps][S::nt];
  auto read = [&](int slot, int set) {
    const uint8_t* sl = lds + slot * S::slot;
#pragma unroll
    for (int s = 0; s < S::steps; ++s) {
      const int at = ((4 * (part * S::steps + s) + quarter) ^ S::mix(r16)) << 4;
#pragma unroll
      for (int j = 0; j < S::nt; ++j)
        b[set][s][j] = *reinterpret_cast<const v4i*>(sl + (kTM + 16 * (wn * S::nt + j) + r16) * kBK + at);
#pragma unroll
      for (int i = 0; i < S::mt; ++i)
        a[set][s][i] = *reinterpret_cast<const v4i*>(sl + (16 * (wm * S::mt + i) + r16) * kBK + at);
    }
  };
#pragma unroll
  for (int t = 0; t < S::slots; ++t) issue(t, t);
  wait_vmcnt<(S::slots - 1) * S::loads>();
  barrier();
  read(0, 0);
  int slot = 0;
  for (int t = 0; t < nkb; t += 2) {
#pragma unroll
    for (int set = 0; set < 2; ++set) {
      // The next block has landed for every wave, and every wave has read this one: its
      // slot is filled again (blocks behind the last read no memory and hold zeros)
      wait_vmcnt<(S::slots - 2) * S::loads>();
      barrier();
      issue(t + set + S::slots, slot);
      slot = slot + 1 == S::slots ? 0 : slot + 1;
      read(slot, set ^ 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int s = 0; s < S::steps; ++s)
#pragma unroll
        for (int i = 0; i < S::mt; ++i)
#pragma unroll
          for (int j = 0; j < S::nt; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[set][s][j], a[set][s][i], acc[i][j], 0, 0, 0);
    }
  }
  wait_vmcnt<0>();
  barrier();   // every wave done with the ring before it holds the sums

  int* sums = reinterpret_cast<int*>(lds);
#pragma unroll
  for (int i = 0; i < S::mt; ++i)
#pragma unroll
    for (int j = 0; j < S::nt; ++j)
      *reinterpret_cast<v4i*>(sums + (part * kTM + 16 * (wm * S::mt + i) + r16) * S::ld + 16 * (wn * S::nt + j) +
                              4 * quarter) = acc[i][j];
  __syncthreads();
  const int rows = min(g.M - m0, kTM);
  // A thread takes kV columns of a row: up to eight, if all threads have some (one row over 4096
  // channels of 4096 6.3 us with eight, 5.6 with the one that its 16 x 16 tiles give)
  constexpr int kV = S::cols, groups = kTN / kV, kRead = kV < 4 ? kV : 4;
  typedef int some __attribute__((ext_vector_type(kRead)));
  auto store = [&](auto lines) {
    for (int u = threadIdx.x; u < rows * groups; u += 512) {
      const int r = u / groups, c = kV * (u % groups), n = n0 + c;
      if (n >= g.N) continue;
      const float sa = g.a_scales[(int64_t)(m0 + r) * g.a_step];
      float v[kV];
#pragma unroll
      for (int h = 0; h < kV; h += kRead) {
        some x{};
#pragma unroll
        for (int w = 0; w < S::wk; ++w) x += *reinterpret_cast<const some*>(sums + (w * kTM + r) * S::ld + c + h);
        const auto sb = some_at<kRead>(g.b_scales, g.b_step, n + h, g.N);
#pragma unroll
        for (int j = 0; j < kRead; ++j) v[h + j] = (float)x[j] * sa * sb[j];
        if (g.bias) {
          const auto bias = some_at<kRead>(g.bias, 1, n + h, g.N);
#pragma unroll
          for (int j = 0; j < kRead; ++j) v[h + j] += bias[j];
        }
      }
      store_out<kOut, decltype(lines)::value>(g.c, m0 + r, n, g.N, v);
    }
  };
  if (kV == 8 && whole_lines<kOut>(g.N)) store(std::bool_constant<kV == 8>{});
  else store(std::false_type{});
}

template <int kTM, int kTN, int kBK, int kWM, int kWN, int kPer>
hipError_t launch_ring(const Int8Args& g, bool out_bf16, hipStream_t st) {
  const int tiles_m = (g.M + kTM - 1) / kTM, tiles_n = (g.N + kTN - 1) / kTN;
  const uint32_t grid = (uint32_t)tiles_m * (uint32_t)tiles_n;
  const bool along_n = int8_along_n(g.M, g.N);
  const int inner = along_n ? tiles_n : tiles_m;
  if (out_bf16) k_int8_ring<kTM, kTN, kBK, kWM, kWN, kPer, kBf16><<<grid, 512, 0, st>>>(g, inner, along_n);
  else k_int8_ring<kTM, kTN, kBK, kWM, kWN, kPer, kF32><<<grid, 512, 0, st>>>(g, inner, along_n);
  return hipGetLastError();
}

// `most` workgroups take the tiles in turn.
template <int kTM, int kTN, int kWM, int kWN>
hipError_t launch_tile(const Int8Args& g, bool out_bf16, int64_t most, hipStream_t st) {
  const int tiles_m = (g.M + kTM - 1) / kTM, tiles_n = (g.N + kTN - 1) / kTN;
  const uint32_t grid = (uint32_t)std::min((int64_t)tiles_m * tiles_n, most);
  if (out_bf16) k_int8_tile<kTM, kTN, kWM, kWN, kBf16><<<grid, 64 * kWM * kWN, 0, st>>>(g, tiles_m, tiles_n);
  else k_int8_tile<kTM, kTN, kWM, kWN, kF32><<<grid, 64 * kWM * kWN, 0, st>>>(g, tiles_m, tiles_n);
  return hipGetLastError();
}

// In the order of kInt8Rings.
constexpr hipError_t (*kRingLaunch[])(const Int8Args&, bool, hipStream_t) = {
    launch_ring<16, 16, 512, 1, 1, 2>, launch_ring<16, 32, 512, 1, 2, 2>,  launch_ring<32, 16, 512, 1, 1, 2>,
    launch_ring<32, 32, 256, 1, 2, 2>, launch_ring<32, 64, 256, 1, 4, 2>,  launch_ring<64, 32, 256, 2, 1, 2>,
    launch_ring<64, 64, 128, 2, 2, 2>, launch_ring<128, 64, 128, 2, 2, 2>, launch_ring<64, 128, 128, 1, 4, 2>};
static_assert(sizeof(kRingLaunch) / sizeof(kRingLaunch[0]) == sizeof(kInt8Rings) / sizeof(kInt8Rings[0]), "rings");

}  // namespace

hipError_t launch_gemm_int8(const Int8Args& g, bool out_bf16, hipStream_t st) {
  const Int8Tile t = choose_int8(g.M, g.N, g.K);
  if (t.kernel == Int8Kernel::kRing) return kRingLaunch[t.ring](g, out_bf16, st);
  if (t.kernel == Int8Kernel::kDeepRing) return launch_ring<128, 64, 256, 1, 2, 1>(g, out_bf16, st);
  if (t.tm == 128) return launch_tile<128, 128, 2, 2>(g, out_bf16, kInt8SmallGrid, st);
  return launch_tile<256, 256, 2, 4>(g, out_bf16, kInt8LargeGrid, st);
}

}  // namespace pqb
