// Attention over the paged 8-bit KV cache (layouts in paged.h):
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - max),  over the tokens j
// that the query row sees: j < kv_len, and for causal rows j <= kv_len - n + i
// (query i of n).  A row that sees nothing gives 0.  A tile's rows are the
// n * group (token, query head) pairs that share one KV head.
//
// Both products run on the matrix cores with the keys as rows: S^T = K Q^T, then
// O^T = V^T P^T.  Key row m of 16-row tile t stands for token 16 (m / 4) + 4 t +
// m % 4 of a 64-token unit, so that a lane's 16 results of S^T are 16 consecutive
// tokens of its query row: exactly the operand P^T needs, with no exchange
// between lanes, and exactly 16 bytes of V^T.
//
// Numbers: a key is dec(c) 2^X, exact in bf16, times q's bf16 (float32 q is taken
// as the exact sum of three bf16 parts).  The maximum, the sum and O are float32.
// The row kernel rounds P to f16 as 2^15 p: 11 significant bits for every p >= 2^-29, three
// more than bf16 has, and below that to 2^-40 of the largest (float32 rows add
// the rounding's remainder as a second f16 part).  V enters as dec(c) 2^(X - R),
// exact in f16 unless X is over 15 below R, the largest V exponent met so far; O
// is kept in units of 2^R and rescaled when R or the row's maximum rises.
#include <algorithm>

#include "launch.h"
#include "paged.h"
#include "units.h"

namespace pqb {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kTile = 16;        // query rows of a tile
constexpr int kWaves = kUnitWaves, kThreads = kWaves * kWave;
constexpr int kMaxPartRows = 64;                  // rows of a request that the row kernel may split
constexpr int64_t kMaxGroups = 1 << 23;            // workgroups that splits or joins lead to
constexpr int kMinWideUnits = 8;                  // fewest units of a split of the wide kernel
// 512: the places of bf16 and heads up to 128 wide, two workgroups a CU, for which it was
// measured best of 256 to 1024.  The other forms have 256 places and share the number.
constexpr int64_t kMaxWideSplits = 32, kWideGroupsWanted = 512;

// ---------------------------------------------------------------------------
// Work items.  Request b has u_b = ceil(kv_len / 64) units and is cut into
// max(1, ceil(u_b / C)) items, C chosen from the sum of all u_b so that about
// kGroupsWanted workgroups run whatever the lengths are (the host does not know
// them).  Every wave works out its own item from the lengths.
// ---------------------------------------------------------------------------

struct Request {
  int32_t start, n, kv;   // first query row, query tokens, tokens in the cache
};

__device__ __forceinline__ Request request(const AttendArgs& a, int64_t b) {
  Request r;
  const int64_t s0 = min((int64_t)max(a.starts[b], 0), a.q_rows);
  const int64_t s1 = min((int64_t)max(a.starts[b + 1], 0), a.q_rows);
  r.start = (int32_t)s0;
  r.n = (int32_t)max(s1 - s0, (int64_t)0);
  r.kv = (int32_t)min((int64_t)max(a.kv_lens[b], 0), a.width << a.shift);
  return r;
}

__device__ __forceinline__ int units_of(int32_t kv) { return (int)(((int64_t)kv + kUnit - 1) / kUnit); }

// A request's rows, and its items' units at C units an item.
__device__ __forceinline__ int items_of(const AttendArgs& a, const Request& r, int C) {
  const int64_t rows = (int64_t)r.n * a.group;
  if (rows == 0) return 0;
  if (rows > a.part_rows) return a.wide ? 0 : 1;  // the wide kernel's, or not cut
  return items_of_units(units_of(r.kv), C);
}

__device__ __forceinline__ int64_t wave_sum64(int64_t v) {
#pragma unroll
  for (int d = kWave / 2; d; d >>= 1) v += (int64_t)__shfl_xor((long long)v, d);
  return v;
}

// Request b0 + lane (none behind the last), and the one that lane `src` holds.
__device__ __forceinline__ Request lane_request(const AttendArgs& a, int64_t b0) {
  const int64_t b = b0 + (threadIdx.x & (kWave - 1));
  return b < a.batch ? request(a, b) : Request{0, 0, 0};
}
__device__ __forceinline__ Request from_lane(const Request& r, int src) {
  return Request{__builtin_amdgcn_readlane(r.start, src), __builtin_amdgcn_readlane(r.n, src),
                 __builtin_amdgcn_readlane(r.kv, src)};
}

// The units of an item.  `first`: requests 0 .. 63, one a lane.
__device__ __forceinline__ int split_units(const AttendArgs& a, const Request& first) {
  int64_t total = 0;
  for (int64_t b0 = 0; b0 < a.batch; b0 += kWave) {
    const Request r = b0 ? lane_request(a, b0) : first;
    const int64_t rows = (int64_t)r.n * a.group;
    if (rows > 0 && rows <= a.part_rows) total += units_of(r.kv);
  }
  return __builtin_amdgcn_readfirstlane(units_an_item(wave_sum64(total) * a.heads));
}

struct Item {
  int64_t b, first;      // request, and its first item
  int32_t index, count;  // this item among the request's
  Request rq;
};

// Item x (or, by_request, the items of request x); b = -1 if there is none.
template <bool kByRequest>
__device__ __forceinline__ Item find_item(const AttendArgs& a, int64_t x, int C, const Request& first) {
  const int lane = threadIdx.x & (kWave - 1);
  int64_t base = 0;
  for (int64_t b0 = 0; b0 < a.batch; b0 += kWave) {
    const int64_t b = b0 + lane;
    const Request r = b0 ? lane_request(a, b0) : first;
    const int mine = items_of(a, r, C);
    int incl = mine;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int o = __shfl_up(incl, d);
      if (lane >= d) incl += o;
    }
    const bool hit = kByRequest ? b == x : (x >= base + incl - mine && x < base + incl);
    const uint64_t m = __ballot(hit);
    if (m) {
      const int src = __builtin_ctzll(m);
      const int cnt = __builtin_amdgcn_readlane(mine, src), upto = __builtin_amdgcn_readlane(incl, src);
      Item it;
      it.b = b0 + src;
      it.first = base + upto - cnt;
      it.index = kByRequest ? 0 : (int32_t)(x - it.first);
      it.count = cnt;
      it.rq = from_lane(r, src);
      return it;
    }
    base += __builtin_amdgcn_readlane(incl, kWave - 1);
  }
  return Item{-1, 0, 0, 0, Request{0, 0, 0}};
}

// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t cvt_f16x2(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}

// 8 codes -> 8 bf16 (f16) of value dec(c) * s, s a power of two.
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t lo, uint32_t hi, float s) {
  return __builtin_bit_cast(
      bf16x8, make_uint4(
                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, s, false)),
                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, s, true)),
                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, s, false)),
                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, s, true))));
}
__device__ __forceinline__ f16x8 codes_f16(uint32_t lo, uint32_t hi, float s) {
  return __builtin_bit_cast(
      f16x8, make_uint4(
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)lo, s, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)lo, s, true)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)hi, s, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)hi, s, true))));
}

// Eight q values as bf16 parts: themselves, or three parts whose sum is exact.
template <bool kF32>
__device__ __forceinline__ void load_q8(const void* q, int64_t at, bool valid, bf16x8* part) {
  if constexpr (!kF32) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (valid) w = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(q) + at);
    part[0] = __builtin_bit_cast(bf16x8, w);
  } else {
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (valid) {
      const float* p = reinterpret_cast<const float*>(q) + at;
      const uint4 x = *reinterpret_cast<const uint4*>(p), y = *reinterpret_cast<const uint4*>(p + 4);
      v[0] = as_f(x.x), v[1] = as_f(x.y), v[2] = as_f(x.z), v[3] = as_f(x.w);
      v[4] = as_f(y.x), v[5] = as_f(y.y), v[6] = as_f(y.z), v[7] = as_f(y.w);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = bf16x2_rne(v[2 * j], v[2 * j + 1]);
        v[2 * j] -= as_f(w[j] << 16);
        v[2 * j + 1] -= as_f(w[j] & 0xFFFF0000u);
      }
      part[k] = __builtin_bit_cast(bf16x8, make_uint4(w[0], w[1], w[2], w[3]));
    }
  }
}

// Stores kN consecutive results as float32 or RNE bf16.
template <bool kF32, int kN>
__device__ __forceinline__ void store_row(void* out, int64_t at, const float* o) {
  if constexpr (kF32) {
    float* p = reinterpret_cast<float*>(out) + at;
#pragma unroll
    for (int i = 0; i < kN; i += 4)
      *reinterpret_cast<uint4*>(p + i) = make_uint4(as_u(o[i]), as_u(o[i + 1]), as_u(o[i + 2]), as_u(o[i + 3]));
  } else {
    uint16_t* p = reinterpret_cast<uint16_t*>(out) + at;
#pragma unroll
    for (int i = 0; i < kN; i += 4)
      *reinterpret_cast<uint2*>(p + i) = make_uint2(bf16x2_rne(o[i], o[i + 1]), bf16x2_rne(o[i + 2], o[i + 3]));
  }
}

// What a part of a row counts beside one with the maximum M.
__device__ __forceinline__ float part_weight(float m, float M, float c) {
  return m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m - M) * c);
}

// Sums of p v in units of 2^R (biased), and l of p, to averages.  A part keeps its
// average and its l: the sum of p v may pass float32's range where no average does, and
// 2^R / l its smallest normal.  (l holds the p of the row's reference, 1 times 2^9 or
// 2^15, and of at most 2^31 tokens more: well inside recip_rn's range.)
template <int kN>
__device__ __forceinline__ void average(float* o, float l, int R) {
  const float inv = l > 0 ? recip_rn(l) : 0.0f, unit = as_f((uint32_t)R << 23);
#pragma unroll
  for (int i = 0; i < kN; ++i) o[i] = o[i] * inv * unit;
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) void*)p);
}

// Wave-wide DMA of 16 bytes per lane from g to LDS address lds + 16 lane; kNt: with
// the streaming hint.
template <bool kNt = false>
__device__ __forceinline__ void dma16(const void* g, uint32_t lds) {
  if constexpr (kNt)
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off nt" ::"v"(g), "s"(lds) : "memory");
  else
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(g), "s"(lds) : "memory");
}

// The same from a wave-uniform base plus an unsigned 32-bit offset per lane.
template <bool kNt = false>
__device__ __forceinline__ void dma16s(const void* g, uint32_t off, uint32_t lds) {
  if constexpr (kNt)
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt" ::"v"(off), "s"(g), "s"(lds)
                 : "memory");
  else
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(g), "s"(lds)
                 : "memory");
}

template <int kN>
__device__ __forceinline__ void wait_vmcnt() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kN) : "memory");
}

__device__ __forceinline__ float swap_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(as_u(x), as_u(x), false, false);
  return fmaxf(as_f(r[0]), as_f(r[1]));
}
__device__ __forceinline__ float swap_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(as_u(x), as_u(x), false, false);
  return as_f(r[0]) + as_f(r[1]);
}

// Over the whole wave, in one order whatever the lane.
template <typename F>
__device__ __forceinline__ float wave_fold(float x, F f) {
  x = f(x, as_f(dpp<kDppXor1>(as_u(x))));
  x = f(x, as_f(dpp<kDppXor2>(as_u(x))));
  x = f(x, as_f(dpp<kDppHalfMirror>(as_u(x))));
  x = f(x, as_f(dpp<kDppMirror>(as_u(x))));
  x = f(x, __shfl_xor(x, 16));
  return f(x, __shfl_xor(x, 32));
}

// ---------------------------------------------------------------------------
// Few query rows: single tokens, 16 rows a tile.
// Bound by the bytes of the cache.
//
// One workgroup takes an item's units for one KV head, its waves every fourth
// unit.  A wave has LDS of its own for one unit's keys and one unit's V and fills
// it by DMA: the next keys go out once S^T is formed, the next V once O^T has its
// products, so 8 KB (D = 128) are in flight through most of a unit and no barrier
// is met before the waves' partial results join.  The DMA reads whole pages in
// order; loading the matrix operands straight into registers takes half lines of
// a key row at a time.  Rows of one tile read their keys and V once and carry the
// streaming hint.  On 64 requests of 269 K tokens, 8 heads x 128: 107 us, against
// 125 without the hint and 130 from registers, where the hint gains nothing.
// ---------------------------------------------------------------------------

// 16-byte chunk of a token's key row in LDS, spread so that the rows of a matrix
// operand (tokens 0-3 and 16-19 of a unit) fall on eight different 16-byte columns.
template <int kD>
__device__ __forceinline__ int row_swizzle(int token) {
  if constexpr (kD % 128 == 0)
    return (token & 3) | (((token >> 4) & 1) << 2);
  else
    return ((token >> 1) & 1) | (((token >> 4) & 1) << 1);
}

template <int kD, bool kWholePages>
struct RowsLds {
  static constexpr int kGroups = kWholePages ? 1 : 4;   // pages that a unit may lie in
  union {
    struct {
      uint8_t k[kWaves][kUnit * kD], v[kWaves][kUnit * kD];
    } in;
    float o[kWaves][kTile][kD + 4];
  };
  float m[kWaves][kTile], l[kWaves][kTile];
  int R[kWaves];
  // page (-1: none) and scales (K's byte, V's << 8) of a wave's next units
  int pg[kWaves][kMetaUnits * kGroups], xs[kWaves][kMetaUnits * kGroups];
};

// Item x for KV head h, row tiles z, z + nz, ... (more than one where the wide kernel
// does not go, or the hint of the most query tokens was wrong).
template <int kD, bool kF32, bool kWholePages>
__device__ __forceinline__ void attend_rows(const AttendArgs& a, int64_t x, int h, int z, int nz,
                                            RowsLds<kD, kWholePages>& lds) {
  constexpr int kKC = kD / 64;       // 16-byte key reads of a lane per 16-row tile
  constexpr int kDT = kD / 16;       // 16-channel tiles of O; also the DMA steps of a unit's keys, or V
  constexpr int kKeyChunks = kD / 16;
  constexpr int kParts = kF32 ? 3 : 1;
  constexpr int kGroups = RowsLds<kD, kWholePages>::kGroups;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int col = lane & 15, g4 = lane >> 4;
  uint8_t *kb = lds.in.k[wave], *vb = lds.in.v[wave];
  int *pg = lds.pg[wave], *xs = lds.xs[wave];

  const Request first = lane_request(a, 0);
  const int C = split_units(a, first);
  const Item it = find_item<false>(a, x, C, first);
  if (it.b < 0) return;
  const Request rq = it.rq;
  const int32_t rows = rq.n * a.group;
  const bool stream = rows <= kTile;
  const int all_units = units_of(rq.kv);
  const int unit0 = it.count == 1 ? 0 : it.index * C;
  const int unit_end = it.count == 1 ? all_units : min(all_units, unit0 + C);
  const int32_t* table = a.table + it.b * a.width;
  const int64_t page_bytes = (int64_t)kD << a.shift;
  const uint8_t *k_head = a.k_codes + h * page_bytes, *v_head = a.v_codes + h * page_bytes;
  const uint32_t page_step = (uint32_t)(a.heads * page_bytes);   // at most 4096 heads of 64 KiB
  const int ps1 = (1 << a.shift) - 1;

  // this lane's part of a DMA step: keys of a 16-token group, V of token group vg
  const int vg = (lane & 3) ^ ((lane >> 3) & 3);
  uint32_t koff[kKC], voff;
#pragma unroll
  for (int i = 0; i < kKC; ++i) {
    const int j = i * kWave + lane, token = j / kKeyChunks;   // the swizzle of groups 1 and 3 flips one bit more
    koff[i] = (uint32_t)(token * kD + (((j % kKeyChunks) ^ row_swizzle<kD>(token)) << 4));
  }
  voff = (uint32_t)(((lane >> 2) << a.shift) + (kWholePages ? 16 * vg : 0));
  constexpr uint32_t kFlip = kD % 128 == 0 ? 64 : 32;         // row_swizzle(16), in bytes

  for (int rt = z; rt * kTile < rows; rt += nz) {
    if (rt != z) __syncthreads();  // the last tile's reads of LDS are done
    const int row = rt * kTile + col;
    const bool valid = row < rows;
    const int tok = row / a.group, hq = h * a.group + row % a.group;
    // what this lane's row, the tile's first row and its last row see
    const int ahead = rq.kv - rq.n + 1;
    const int limit = !valid ? 0 : a.causal ? ahead + tok : rq.kv;
    const int first_limit = a.flat ? 0 : a.causal ? ahead + rt * kTile / a.group : rq.kv;
    const int last_limit = a.causal ? ahead + (min(rt * kTile + kTile, rows) - 1) / a.group : rq.kv;
    const int u0 = unit0 + wave;
    const int end = __builtin_amdgcn_readfirstlane(min(unit_end, last_limit > 0 ? units_of(last_limit) : 0));

    // pages and scales of this wave's units u, u + kWaves, ..., kMetaUnits of them
    auto load_pages = [&](int u) {
#pragma unroll
      for (int i = lane; i < kMetaUnits * kGroups; i += kWave) {
        const int at = table_column(u + i / kGroups * kWaves, i % kGroups, rq.kv, a.shift);
        const int p = at >= 0 ? table[at] : -1;
        pg[i] = (uint32_t)p < (uint64_t)a.pages ? p : -1;
      }
    };
    auto load_scales = [&]() {
#pragma unroll
      for (int i = lane; i < kMetaUnits * kGroups; i += kWave) {
        const int p = pg[i];
        int x = 0x0101;
        if (p >= 0) {
          const int64_t at = (int64_t)p * a.heads + h;
          x = min(max((int)a.k_scales[at], 1), 254) | min(max((int)a.v_scales[at], 1), 254) << 8;
        }
        xs[i] = x;
      }
    };
    auto meta_at = [&](int u, int group) {
      return ((u - u0) / kWaves & (kMetaUnits - 1)) * kGroups + (kWholePages ? 0 : group);
    };
    auto stage_k = [&](int u) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint32_t p = (uint32_t)max(__builtin_amdgcn_readfirstlane(pg[meta_at(u, g)]), 0);
        const uint8_t* kp = k_head + (uint64_t)p * page_step + (uint32_t)(((u * kUnit + 16 * g) & ps1) * kD);
#pragma unroll
        for (int i = 0; i < kKC; ++i) {
          const uint32_t off = g & 1 ? koff[i] ^ kFlip : koff[i], to = lds_addr(kb + (g * kKC + i) * 1024);
          if (stream)
            dma16s<true>(kp, off, to);
          else
            dma16s(kp, off, to);
        }
      }
    };
    auto stage_v = [&](int u) {
      int p = pg[meta_at(u, vg)];
      if constexpr (kWholePages) p = __builtin_amdgcn_readfirstlane(p);
      const uint8_t* vp = v_head + (uint64_t)(uint32_t)max(p, 0) * page_step +
                          ((u * kUnit + (kWholePages ? 0 : 16 * vg)) & ps1);
#pragma unroll
      for (int i = 0; i < kDT; ++i) {
        const uint32_t to = lds_addr(vb + i * 1024);
        const uint8_t* from = vp + ((int64_t)i << (a.shift + 4));
        if constexpr (kWholePages) {
          if (stream)
            dma16s<true>(from, voff, to);
          else
            dma16s(from, voff, to);
        } else {
          if (stream)
            dma16<true>(from + voff, to);
          else
            dma16(from + voff, to);
        }
      }
    };

    bf16x8 qf[2 * kKC][kParts];
#pragma unroll
    for (int s = 0; s < 2 * kKC; ++s)
      load_q8<kF32>(a.q, (int64_t)(rq.start + tok) * a.q_stride + (int64_t)hq * kD + (s >> 1) * 64 + g4 * 16 + (s & 1) * 8,
                    valid, qf[s]);
    if (u0 < end) {
      load_pages(u0);
      stage_k(u0);
      stage_v(u0);
      load_scales();
    }

    float m = -INFINITY, l = 0;
    int R = 1;
    f32x4 o[kDT];
#pragma unroll
    for (int i = 0; i < kDT; ++i) o[i] = f32x4{0, 0, 0, 0};

    for (int u = u0; u < end; u += kWaves) {
      const bool more = u + kWaves < end;
      const int tv = u * kUnit + 16 * g4;
      const int sk_at = meta_at(u, col >> 2), v_at = meta_at(u, g4);
      const float sk = as_f((uint32_t)(xs[sk_at] & 0xFF) << 23);
      const bool okv = pg[v_at] >= 0;
      const int xv = xs[v_at] >> 8;
      if (more && ((u + kWaves - u0) / kWaves & (kMetaUnits - 1)) == 0) {
        load_pages(u + kWaves);
        load_scales();
      }

      wait_vmcnt<kDT>();   // the keys: V's DMA may still run
      f32x4 s[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int token = 16 * (col >> 2) + 4 * t + (col & 3), key = row_swizzle<kD>(token);
        s[t] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < kKC; ++i) {
          const uint4 w = *reinterpret_cast<const uint4*>(kb + token * kD + (((4 * i + g4) ^ key) << 4));
          const bf16x8 k0 = codes_bf16(w.x, w.y, sk), k1 = codes_bf16(w.z, w.w, sk);
#pragma unroll
          for (int p = kParts - 1; p >= 0; --p) {
            s[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, qf[2 * i][p], s[t], 0, 0, 0);
            s[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, qf[2 * i + 1][p], s[t], 0, 0, 0);
          }
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the key reads have returned
      if (more) stage_k(u + kWaves);

      // Tokens outside the row's view, and tokens of a page id outside the cache
      // (first_limit 0: every unit, if scores are all 0).
      const bool whole = (u + 1) * kUnit <= first_limit && __ballot(!okv) == 0;
      uint32_t keep[4] = {~0u, ~0u, ~0u, ~0u};
      if (!whole) {
        const int cnt = okv ? min(max(limit - tv, 0), 16) : 0, held = okv ? min(max(rq.kv - tv, 0), 16) : 0;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (a.flat) s[t][i] = 0;
            if (4 * t + i >= cnt) s[t][i] = -INFINITY;
          }
        // codes behind the last token may be anything (NaN times p = 0 is NaN)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int nb = min(max(held - 4 * w, 0), 4);
          keep[w] = nb == 4 ? ~0u : (1u << (8 * nb)) - 1;
        }
      }
      float mx = max3f(s[0][0], s[0][1], s[0][2]);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = (t == 0 ? 3 : 0); i < 4; ++i) mx = fmaxf(mx, s[t][i]);
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = swap_max(mx);
      int xr = xv;   // of a page that is none: 1
      if constexpr (!kWholePages) {
        xr = max(xr, __shfl_xor(xr, 16));
        xr = max(xr, __shfl_xor(xr, 32));
      }
      const float m_new = fmaxf(m, mx), top = m_new == -INFINITY ? 0.0f : m_new;
      const float alpha = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m - top) * a.c);
      const int R_new = max(R, xr);
      const float grow = R_new - R > 126 ? 0.0f : as_f((uint32_t)(127 - (R_new - R)) << 23);
      const float sv = as_f((uint32_t)(127 - min(R_new - xv, 60)) << 23);
      m = m_new;
      R = R_new;
      float p[16], sum = 0;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e >> 2][e & 3] - top, a.c, 15.0f));
        sum += p[e];
      }
      l = l * alpha + sum;
      const float f = alpha * grow;
      if (__ballot(f != 1.0f)) {
#pragma unroll
        for (int i = 0; i < kDT; ++i) o[i] *= f;
      }
      f16x8 ph[2], pl[2];
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x = p[8 * st + 2 * j], y = p[8 * st + 2 * j + 1];
          hi[j] = cvt_f16x2(x, y);
          const f16x2 b = __builtin_bit_cast(f16x2, hi[j]);
          lo[j] = kF32 ? cvt_f16x2(x - (float)b[0], y - (float)b[1]) : 0;
        }
        ph[st] = __builtin_bit_cast(f16x8, make_uint4(hi[0], hi[1], hi[2], hi[3]));
        pl[st] = __builtin_bit_cast(f16x8, make_uint4(lo[0], lo[1], lo[2], lo[3]));
      }
      if (more)
        wait_vmcnt<kDT>();   // V: the next keys may still run
      else
        wait_vmcnt<0>();
#pragma unroll
      for (int i = 0; i < kDT; ++i) {
        const int d = 16 * i + col;
        uint4 w = *reinterpret_cast<const uint4*>(vb + d * 64 + ((g4 ^ ((d >> 1) & 3)) << 4));
        if (!whole) w = make_uint4(w.x & keep[0], w.y & keep[1], w.z & keep[2], w.w & keep[3]);
        const f16x8 v0 = codes_f16(w.x, w.y, sv), v1 = codes_f16(w.z, w.w, sv);
        if constexpr (kF32) {
          o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pl[0], o[i], 0, 0, 0);
          o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pl[1], o[i], 0, 0, 0);
        }
        o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, ph[0], o[i], 0, 0, 0);
        o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, ph[1], o[i], 0, 0, 0);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the V reads have returned
      if (more) stage_v(u + kWaves);
    }

    l += __shfl_xor(l, 16);
    l = swap_sum(l);
    __syncthreads();  // every wave is done with its K and V, whose LDS O takes
#pragma unroll
    for (int i = 0; i < kDT; ++i) *reinterpret_cast<f32x4*>(&lds.o[wave][col][16 * i + 4 * g4]) = o[i];
    if (g4 == 0) {
      lds.m[wave][col] = m;
      lds.l[wave][col] = l;
    }
    if (lane == 0) lds.R[wave] = R;
    __syncthreads();
    // 16 threads a row, kD / 16 channels each
    const int r = tid / 16, d0 = (tid % 16) * (kD / 16), grow_row = rt * kTile + r;
    if (grow_row < rows) {
      float M = lds.m[0][r];
      int top = lds.R[0];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) {
        M = fmaxf(M, lds.m[w][r]);
        top = max(top, lds.R[w]);
      }
      float L = 0, acc[kD / 16];
#pragma unroll
      for (int j = 0; j < kD / 16; ++j) acc[j] = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float wt = part_weight(lds.m[w][r], M, a.c);
        const int down = top - lds.R[w];
        const float wo = down > 126 ? 0.0f : wt * as_f((uint32_t)(127 - down) << 23);
        L += lds.l[w][r] * wt;
#pragma unroll
        for (int j = 0; j < kD / 16; ++j) acc[j] += lds.o[w][r][d0 + j] * wo;
      }
      average<kD / 16>(acc, L, top);
      if (it.count == 1) {
        store_row<kF32, kD / 16>(a.out, ((int64_t)(rq.start + grow_row / a.group) * a.heads * a.group +
                                         h * a.group + grow_row % a.group) * kD + d0, acc);
      } else {
        const int64_t slot = (x * a.heads + h) * a.part_rows + grow_row;
        store_row<true, kD / 16>(a.part_o, slot * kD + d0, acc);
        if (tid % 16 == 0) {
          a.part_ml[2 * slot] = M;
          a.part_ml[2 * slot + 1] = L;
        }
      }
    }
  }
}

template <int kD, bool kF32, bool kWholePages>
__global__ __launch_bounds__(kThreads) void k_attend_rows(const AttendArgs a) {
  __shared__ __align__(16) RowsLds<kD, kWholePages> lds;
  attend_rows<kD, kF32, kWholePages>(a, blockIdx.x, blockIdx.y, blockIdx.z, gridDim.z, lds);
}

// ---------------------------------------------------------------------------
// Many query rows: prompts and chunks.
//
// A workgroup takes 128 rows of one KV head, 32 a wave, over its request's
// units of 64 tokens; both tiles of a unit (64 D bytes each) go straight into
// LDS by DMA, the next unit's under this one's products, one barrier a unit.
//
// S^T: the keys are decoded to bf16 beside the products, where dec(c) 2^X is exact,
// against q's bf16 (or a float32 q's three parts).  The FP8 products would take the
// codes as they are, but sum eight products at a time with 13 bits below the largest
// (beside 2^16 one of 2^3 counts, one of 2^2 is lost): where a channel of the keys stands
// out, that drops what the others say.  The bf16 products keep float32's 24 bits and
// cost what two FP8 ones would (q in two E4M3 parts), but for 64 conversions more a
// wave and unit (D = 128): the two prompts below took 265-280 us with FP8 products.
// O^T: V is decoded to f16 beside the products (v_cvt_scalef32_pk_f16_fp8).
//
// Key row m = 8 a + 4 h + b of tile t stands for token 32 h + 16 t + 4 a + b: a
// lane (column n, half h) then holds 32 consecutive tokens of its query row.
// The maximum is followed loosely: p is held as 2^9 p' in f16 relative to a
// reference that moves to the maximum (and O and l with it) only when a lane's
// sum of its 32 p of a unit passes 65000, so that no p passes f16's 65504.  Just
// after a move that sum is 2^14 at most, however flat the row, so a move is rare;
// 11 significant bits reach down to 2^-23 of the reference.
//
// Bound by the issue of vector and matrix instructions together: three units are
// in the pipeline (O^T of one, P of the next, S^T of the one behind it), so that
// the matrix core works under the exponentials and conversions.  Two prompts of
// 4096 tokens (32 heads over 8, 128 wide, bf16): 295-305 us, 0.92 PFLOP/s, where the
// library's bf16 product of 8192^3 reaches 1.19.
// ---------------------------------------------------------------------------

constexpr float kPExp = 9.0f;      // p is held times 2^9
constexpr float kFar = 0x1p20f;   // |r| up to here is right to 2^-5
constexpr int kStages = 4;        // units in LDS at a time
constexpr int kWideRows = 32, kWideTile = kWaves * kWideRows;

// The wide kernel's head dimensions.  Three parts of a wider float32 q do not fit its
// registers beside O; such rows stay with the row kernel, 16 at a time.
constexpr bool wide_takes(int head_dim, bool bf16) { return bf16 || head_dim <= 128; }

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// 16-byte chunk of a key row in LDS: eight neighbouring key rows of a matrix
// operand (tokens 0-3 and 32-35 of a unit) fall on eight different 16-byte columns.
template <int kD>
__device__ __forceinline__ int key_swizzle(int token) {
  if constexpr (kD % 128 == 0)
    return (token & 3) | ((token >> 5) << 2);
  else
    return ((token >> 1) & 1) | ((token >> 5) << 1);
}

// Tile y of 128 rows, counted over the requests of more than part_rows rows; b = -1
// behind the last.
struct WideTile {
  int64_t b;
  int tile;
  Request rq;
};
__device__ __forceinline__ WideTile find_wide(const AttendArgs& a, int64_t y) {
  const int lane = threadIdx.x & (kWave - 1);
  int64_t base = 0;
  for (int64_t b0 = 0; b0 < a.batch; b0 += kWave) {
    const Request r = lane_request(a, b0);
    const int64_t rows = (int64_t)r.n * a.group;
    const int tiles = rows > a.part_rows ? (int)((rows + kWideTile - 1) / kWideTile) : 0;
    int incl = tiles;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int o = __shfl_up(incl, d);
      if (lane >= d) incl += o;
    }
    const uint64_t m = __ballot(y >= base + incl - tiles && y < base + incl);
    if (m) {
      const int src = __builtin_ctzll(m);
      // the last tile sees the most tokens: first
      const int i = (int)(y - base) - __builtin_amdgcn_readlane(incl - tiles, src);
      return WideTile{b0 + src, __builtin_amdgcn_readlane(tiles, src) - 1 - i, from_lane(r, src)};
    }
    base += __builtin_amdgcn_readlane(incl, kWave - 1);
  }
  return WideTile{-1, 0, Request{0, 0, 0}};
}

// A tile whose rows see `end` tokens at most is cut into `count` splits of `per`
// units (the grid's z), so that few tiles over long requests fill the chip.
struct WideSplit {
  int units, per, count;
};
__device__ __forceinline__ WideSplit wide_split(const AttendArgs& a, int end) {
  WideSplit w;
  w.units = end > 0 ? units_of(end) : 0;
  w.per = max((w.units + a.wide_splits - 1) / a.wide_splits, kMinWideUnits);
  w.count = max((w.units + w.per - 1) / w.per, 1);
  return w;
}

template <int kD, bool kWholePages>
struct WideLds {
  static constexpr int kGroups = kWholePages ? 1 : 4;   // pages that a unit may lie in
  uint8_t kbuf[kStages][kUnit * kD], vbuf[kStages][kUnit * kD];
  // page (-1: none) and scales (K's byte, V's << 8) of the units ahead
  int pg[2 * kMetaUnits * kGroups], xs[2 * kMetaUnits * kGroups];
};

// Row tile y of KV head h, one of its splits.
template <int kD, bool kF32, bool kWholePages>
__device__ __forceinline__ void attend_wide(const AttendArgs& a, int h, int64_t y, int split,
                                            WideLds<kD, kWholePages>& lds) {
  constexpr int kKS = kD / 64;    // 64-deep steps of S^T; also the DMA steps of a wave and tensor
  constexpr int kDT = kD / 32;    // 32-channel tiles of O^T
  constexpr int kKeyChunks = kD / 16;
  constexpr int kParts = kF32 ? 3 : 1;    // bf16 parts of q
  constexpr int kPParts = kF32 ? 2 : 1;   // f16 parts of P
  constexpr int kGroups = WideLds<kD, kWholePages>::kGroups;
  auto &kbuf = lds.kbuf, &vbuf = lds.vbuf;
  auto &pg = lds.pg, &xs = lds.xs;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int n = lane & 31, half = lane >> 5;
  const WideTile wt = find_wide(a, y);
  if (wt.b < 0) return;
  const Request rq = wt.rq;
  const int rows = rq.n * a.group, row0 = wt.tile * kWideTile + wave * kWideRows, row = row0 + n;
  const bool valid = row < rows;
  const int tok = row / a.group;
  const int ahead = rq.kv - rq.n + 1;
  const int limit = a.causal && valid ? ahead + tok : rq.kv;
  const int first_limit = a.flat ? 0 : a.causal ? ahead + row0 / a.group : rq.kv;
  const int wave_end = row0 >= rows ? 0 : a.causal ? ahead + (min(row0 + kWideRows, rows) - 1) / a.group : rq.kv;
  const int tile_end = a.causal ? ahead + (min((wt.tile + 1) * kWideTile, rows) - 1) / a.group : rq.kv;
  const WideSplit ws = wide_split(a, tile_end);
  if (split >= ws.count) return;
  const int u0 = __builtin_amdgcn_readfirstlane(split * ws.per);
  const int units = __builtin_amdgcn_readfirstlane(min(ws.units, u0 + ws.per));
  const int32_t* table = a.table + wt.b * a.width;
  const int64_t page_bytes = (int64_t)kD << a.shift;
  const uint32_t ps1 = (1u << a.shift) - 1;

  // q's loads go out first: they return under the page lookups and the first DMA.
  // This lane's 32 channels of each 64.
  const int64_t q_at = (int64_t)(rq.start + tok) * a.q_stride + (int64_t)(h * a.group + row % a.group) * kD + half * 32;
  bf16x8 qf[kKS][4][kParts];
#pragma unroll
  for (int s = 0; s < kKS; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) load_q8<kF32>(a.q, q_at + s * 64 + i * 8, valid, qf[s][i]);

  // What the units lie in: kMetaUnits units' pages and scales at a time.
  auto meta_at = [&](int u, int group) { return (u & (2 * kMetaUnits - 1)) * kGroups + (kWholePages ? 0 : group); };
  auto load_pages = [&](int first) {
    for (int i = tid; i < kMetaUnits * kGroups; i += kThreads) {
      const int u = first + i / kGroups, at = table_column(u, i % kGroups, rq.kv, a.shift);
      const int p = u < units && at >= 0 ? table[at] : -1;
      pg[meta_at(u, i % kGroups)] = (uint32_t)p < (uint64_t)a.pages ? p : -1;
    }
  };
  auto load_scales = [&](int first) {   // each thread's own entries
    for (int i = tid; i < kMetaUnits * kGroups; i += kThreads) {
      const int e = meta_at(first + i / kGroups, i % kGroups), p = pg[e];
      int x = 0x0101;
      if (p >= 0) {
        const int64_t at = (int64_t)p * a.heads + h;
        x = min(max((int)a.k_scales[at], 1), 254) | min(max((int)a.v_scales[at], 1), 254) << 8;
      }
      xs[e] = x;
    }
  };

  // Staging.  While unit u has its O^T formed, u + 1 has its P and u + 2 its S^T: V is
  // staged kStages - 1 units ahead of u and keys two more.  A wave's DMA takes the keys of
  // 16-token group `wave` and a quarter of V's channels; this lane's V bytes are
  // of group vg.  A key group lies in one page, so its address is uniform.
  const int vg = (lane & 3) ^ ((lane >> 3) & 3);
  uint32_t koff[kKS], voff[kKS];
#pragma unroll
  for (int i = 0; i < kKS; ++i) {
    const int j = i * kWave + lane, token = 16 * wave + j / kKeyChunks;
    const int chunk = (j % kKeyChunks) ^ key_swizzle<kD>(token), d = (wave * kKS + i) * 16 + (lane >> 2);
    koff[i] = (uint32_t)((token & 15) * kD + chunk * 16);
    voff[i] = (uint32_t)((d << a.shift) + (kWholePages ? 16 * vg : 0));
  }
  const uint8_t *k_head = a.k_codes + h * page_bytes, *v_head = a.v_codes + h * page_bytes;
  const uint32_t page_step = (uint32_t)(a.heads * page_bytes);   // at most 4096 heads of 64 KiB
  auto k_from = [&](int u) {
    const uint32_t p = (uint32_t)max(__builtin_amdgcn_readfirstlane(pg[meta_at(u, wave)]), 0);
    return k_head + (uint64_t)p * page_step + ((((uint32_t)u * kUnit + 16 * wave) & ps1) * kD);
  };
  auto v_from = [&](int u) {
    int p = pg[meta_at(u, vg)];
    if constexpr (kWholePages) p = __builtin_amdgcn_readfirstlane(p);
    return v_head + (uint64_t)(uint32_t)max(p, 0) * page_step + (((uint32_t)u * kUnit + (kWholePages ? 0 : 16 * vg)) & ps1);
  };
  auto stage_k = [&](int u, const uint8_t* kp) {
#pragma unroll
    for (int i = 0; i < kKS; ++i) dma16s(kp, koff[i], lds_addr(&kbuf[u % kStages][16 * wave * kD + i * 1024]));
  };
  auto stage_v = [&](int u, const uint8_t* vp) {
#pragma unroll
    for (int i = 0; i < kKS; ++i) {
      const uint32_t to = lds_addr(&vbuf[u % kStages][(wave * kKS + i) * 1024]);
      if constexpr (kWholePages)
        dma16s(vp, voff[i], to);
      else
        dma16(vp + voff[i], to);
    }
  };
  // Waits until at most `steps` of this wave's newest staging steps (V of a unit and
  // keys of the second behind it: 2 kKS loads) are in flight.
  auto wait_steps = [&](int steps) {
    static_assert(kStages == 4, "one wait for each number of steps");
    if (steps >= 3)
      wait_vmcnt<6 * kKS>();
    else if (steps == 2)
      wait_vmcnt<4 * kKS>();
    else if (steps == 1)
      wait_vmcnt<2 * kKS>();
    else
      wait_vmcnt<0>();
  };
  load_pages(u0);
  __syncthreads();
  const uint8_t *k_next = nullptr, *v_next = nullptr;   // where the next staging step reads
  if (u0 < units) {
    stage_k(u0, k_from(u0));
    stage_k(u0 + 1, k_from(u0 + 1));   // behind the last unit: page 0's bytes, unused
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
      if (u0 + i < units) {
        stage_v(u0 + i, v_from(u0 + i));
        // (of the fourth unit's keys, in the first's place, only when those are used up)
        if (i < kStages - 2) stage_k(u0 + i + 2, k_from(u0 + i + 2));
      }
  }
  load_scales(u0);

  const float c = a.c;
  // m: the row's reference (the maximum when it was last moved), r = 9 - m c; O
  // and l hold 2^9 p' relative to it.  r starts infinite: the first unit moves it.
  // It is rounded, so exactly they hold 2^e p', e = m c + r.  Where m c passes kFar and
  // that is no longer close to 9, r stays infinite: every unit then settles its row anew,
  // from s - m and with e = 9.
  float m = -INFINITY, r = INFINITY, l = 0;
  auto held_exp = [&](float m, float r) { return r == INFINITY ? kPExp : __builtin_fmaf(m, c, r); };
  int R = 1;
  f32x16 o[kDT];
#pragma unroll
  for (int i = 0; i < kDT; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) o[i][j] = 0;

  auto scores = [&](int u, f32x16* to) {   // S^T of unit u
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int token = 32 * ((n >> 2) & 1) + 16 * t + 4 * (n >> 3) + (n & 3), key = key_swizzle<kD>(token);
      const float sk = as_f((uint32_t)(xs[meta_at(u, 2 * ((n >> 2) & 1) + t)] & 0xFF) << 23);
#pragma unroll
      for (int j = 0; j < 16; ++j) to[t][j] = 0;
#pragma unroll
      for (int ks = 0; ks < kKS; ++ks) {
        const int ch = ks * 4 + half * 2;
        const uint4 lo = *reinterpret_cast<const uint4*>(&kbuf[u % kStages][token * kD + ((ch ^ key) << 4)]);
        const uint4 hi = *reinterpret_cast<const uint4*>(&kbuf[u % kStages][token * kD + (((ch + 1) ^ key) << 4)]);
        const uint32_t kw[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bf16x8 kf = codes_bf16(kw[2 * i], kw[2 * i + 1], sk);
#pragma unroll
          for (int p = kParts - 1; p >= 0; --p)
            to[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[ks][i][p], to[t], 0, 0, 0);
        }
      }
    }
  };
  // P of one unit as f16 pairs (float32: and what they leave over), and this lane's sum
  typedef uint32_t Weights[kPParts][2][8];
  auto weights = [&](const f32x16* s, float r, Weights& pw) {
    float sum = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][2 * j], c, r));
        const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][2 * j + 1], c, r));
        sum += p0;
        sum += p1;
        pw[0][t][j] = cvt_f16x2(p0, p1);
        if constexpr (kF32) {
          const f16x2 b = __builtin_bit_cast(f16x2, pw[0][t][j]);
          pw[kPParts - 1][t][j] = cvt_f16x2(p0 - (float)b[0], p1 - (float)b[1]);
        }
      }
    return sum;
  };
  // What unit u's pages say: its largest V exponent, negative `lo` where some page
  // is none, and the V exponents of this lane's two token groups.
  struct Scales {
    int xr, lo, xv[2];
  };
  auto scales_of = [&](int u) {
    Scales c;
    if constexpr (kWholePages) {
      c.xr = __builtin_amdgcn_readfirstlane(xs[meta_at(u, 0)]) >> 8;
      c.lo = __builtin_amdgcn_readfirstlane(pg[meta_at(u, 0)]);
      c.xv[0] = c.xv[1] = c.xr;
    } else {
      const int4 x = *reinterpret_cast<const int4*>(&xs[meta_at(u, 0)]), p = *reinterpret_cast<const int4*>(&pg[meta_at(u, 0)]);
      c.xr = max(max(x.x, x.y), max(x.z, x.w)) >> 8;
      c.lo = min(min(p.x, p.y), min(p.z, p.w));
      c.xv[0] = (half ? x.z : x.x) >> 8;
      c.xv[1] = (half ? x.w : x.y) >> 8;
    }
    return c;
  };
  // -inf for what unit u's rows do not see (all of them pass here if scores are all 0)
  auto mask = [&](int u, int lo, f32x16* s) {
    if (lo < 0 || (u + 1) * kUnit > first_limit) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int g = 2 * half + t, cnt = pg[meta_at(u, g)] < 0 ? 0 : limit - (u * kUnit + 16 * g);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          if (a.flat) s[t][j] = 0;
          if (j >= cnt) s[t][j] = -INFINITY;
        }
      }
    }
  };
  // No maximum is taken while P fits f16: what does not, or the first unit's
  // infinite r, shows in the sum.  Then the reference moves to the maximum, and O
  // and l with it; and to a larger V exponent.
  auto settle = [&](int xr, f32x16* s, const f32x16* later, Weights& pw, float sum) {
    if (__ballot(!(sum <= 65000.0f)) || xr > R) {
      asm volatile("" ::"v"(later[0]), "v"(later[1]));   // keeps their products above this branch
      float mx = s[0][0];
#pragma unroll
      for (int j = 1; j < 16; ++j) mx = fmaxf(mx, s[0][j]);
#pragma unroll
      for (int j = 0; j < 16; ++j) mx = fmaxf(mx, s[1][j]);
      const float m_new = fmaxf(m, swap_max(mx));
      const bool none = m_new == -INFINITY;
      const float r_new = none ? kPExp : __builtin_fmaf(-m_new, c, kPExp);
      const bool far = fabsf(r_new) > kFar;
      const float at = far ? kPExp : r_new, off = far ? m_new : 0.0f;
      const float held = far ? kPExp : __builtin_fmaf(m_new, c, r_new);
      const float alpha =
          m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(__builtin_fmaf(m - m_new, c, held - held_exp(m, r)));
      const int R_new = max(R, xr);
      const float f = R_new - R > 126 ? 0.0f : alpha * as_f((uint32_t)(127 - (R_new - R)) << 23);
      l *= alpha;
#pragma unroll
      for (int i = 0; i < kDT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] *= f;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < 16; ++j) s[t][j] -= off;
      sum = weights(s, at, pw);
      m = m_new;
      r = none || far ? INFINITY : r_new;
      R = R_new;
    }
    l += sum;
  };
  // O^T += V^T P^T of unit u
  auto values = [&](int u, const int* xv, const Weights& pw) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const float sv = as_f((uint32_t)(127 - min(max(R - xv[t], 0), 60)) << 23);
      f16x8 pf[kPParts][2];
#pragma unroll
      for (int k = 0; k < kPParts; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          pf[k][e] = __builtin_bit_cast(f16x8, make_uint4(pw[k][t][4 * e], pw[k][t][4 * e + 1], pw[k][t][4 * e + 2], pw[k][t][4 * e + 3]));
#pragma unroll
      for (int i = 0; i < kDT; ++i) {
        const int d = 32 * i + n;
        const uint4 w = *reinterpret_cast<const uint4*>(&vbuf[u % kStages][d * 64 + (((2 * half + t) ^ ((d >> 1) & 3)) << 4)]);
        if constexpr (kF32) {
          const f16x8 v0 = codes_f16(w.x, w.y, sv), v1 = codes_f16(w.z, w.w, sv);
          o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v0, pf[kPParts - 1][0], o[i], 0, 0, 0);
          o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v1, pf[kPParts - 1][1], o[i], 0, 0, 0);
          o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v0, pf[0][0], o[i], 0, 0, 0);
          o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v1, pf[0][1], o[i], 0, 0, 0);
        } else {
          o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(codes_f16(w.x, w.y, sv), pf[0][0], o[i], 0, 0, 0);
          o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(codes_f16(w.z, w.w, sv), pf[0][1], o[i], 0, 0, 0);
        }
      }
    }
  };
  // Waits for unit u's V and unit u + 2's keys, sends the next staging step out, and
  // clears the V codes of unit u behind the last token or of no page (they may be
  // anything).
  auto advance = [&](int u, int lo) {
    wait_steps(min(kStages - 2, units - 1 - u));
    __syncthreads();
    if (u + kStages - 1 < units) {
      stage_v(u + kStages - 1, v_next);
      stage_k(u + kStages + 1, k_next);
      if (((u + kStages + 2 - u0) & (kMetaUnits - 1)) == 0) {
        load_pages(u + kStages + 2);
        load_scales(u + kStages + 2);
        __syncthreads();
      }
    }
    if (lo < 0 || (u + 1) * kUnit > rq.kv) {
      for (int i = tid; i < 4 * kD; i += kThreads) {
        const int d = i >> 2, g = (i & 3) ^ ((d >> 1) & 3);
        const int held = pg[meta_at(u, g)] < 0 ? 0 : min(max(rq.kv - (u * kUnit + 16 * g), 0), 16);
        uint32_t* p = reinterpret_cast<uint32_t*>(&vbuf[u % kStages][i * 16]);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int nb = min(max(held - 4 * w, 0), 4);
          if (nb < 4) p[w] &= (1u << (8 * nb)) - 1;
        }
      }
      __syncthreads();
    }
    k_next = k_from(u + kStages + 2), v_next = v_from(u + kStages);
  };

  // One unit that has a next: O^T of unit u, P of u + 1 and S^T of u + 2 (of whatever
  // LDS holds behind the last: unused), three independent things in one block.
  Scales now, ahead1;
  auto unit = [&](int u, const Weights& pw, f32x16* s1, Weights& pw1, f32x16* s2) {
    advance(u, now.lo);
    const Scales then = scales_of(u + 2);
    if (u * kUnit < wave_end) {
      mask(u + 1, ahead1.lo, s1);
      scores(u + 2, s2);
      values(u, now.xv, pw);
      const float sum = weights(s1, r, pw1);
      settle(ahead1.xr, s1, s2, pw1, sum);
    }
    now = ahead1;
    ahead1 = then;
  };

  f32x16 sa[2], sb[2];
  Weights pa, pb;
  if (u0 < units) {
    wait_steps(min(kStages - 2, units - u0));   // the keys of the first two units
    __syncthreads();
    now = scales_of(u0);
    ahead1 = scales_of(u0 + 1);
    scores(u0, sa);
    scores(u0 + 1, sb);
    mask(u0, now.lo, sa);
    settle(now.xr, sa, sb, pa, INFINITY);
    __syncthreads();                  // the first unit's keys are used up
    if (u0 + kStages - 2 < units) stage_k(u0 + kStages, k_from(u0 + kStages));
    k_next = k_from(u0 + kStages + 1), v_next = v_from(u0 + kStages - 1);
  }
  int u = u0;
  for (; u + 2 < units; u += 2) {
    unit(u, pa, sb, pb, sa);
    unit(u + 1, pb, sa, pa, sb);
  }
  if (u + 1 < units) {
    unit(u, pa, sb, pb, sa);
    advance(u + 1, now.lo);
    if ((u + 1) * kUnit < wave_end) values(u + 1, now.xv, pb);
  } else if (u < units) {
    advance(u, now.lo);
    if (u * kUnit < wave_end) values(u, now.xv, pa);
  }

  if (!valid) return;
  l = swap_sum(l);
  const int64_t out_row = (int64_t)(rq.start + tok) * a.heads * a.group + h * a.group + row % a.group;
  const bool whole = ws.count == 1;
  const int64_t slot = whole ? out_row : (int64_t)split * a.q_rows * a.heads * a.group + out_row;
#pragma unroll
  for (int i = 0; i < kDT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[4] = {o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]};
      average<4>(v, l, R);
      const int64_t at = slot * kD + 4 * half + 32 * i + 8 * j;
      if (whole)
        store_row<kF32, 4>(a.out, at, v);
      else
        store_row<true, 4>(a.wide_o, at, v);
    }
  if (!whole) {
    if (half == 0) {
      a.wide_ml[2 * slot] = m;
      a.wide_ml[2 * slot + 1] = l * __builtin_amdgcn_exp2f(-held_exp(m, r));
    }
  }
}

// Both kinds in one launch, for calls whose requests may have many rows: the wide
// tiles first, the few-row items behind them, where they fill the places that the
// last tiles leave (the other order, or alternating, was 5-10% slower).  Tiles are
// counted without gaps, so that the workgroups that find none come last: among
// the others they hold places while the dispatcher deals out, and leave some CUs
// with three workgroups and some with one.  Head by head: where the KV heads
// divide by 8, a head's tiles keep to one XCD and share its L2.
template <int kD, bool kF32, bool kWholePages>
__global__ __launch_bounds__(kThreads, kD <= 128 && !kF32 ? 2 : 1) void k_attend_both(const AttendArgs a,
                                                                             int64_t wide_groups) {
  __shared__ __align__(16) union Lds {
    RowsLds<kD, kWholePages> rows;
    WideLds<kD, kWholePages> wide;
  } lds;
  const int64_t x = blockIdx.x, item = x / a.heads;
  const int h = (int)(x % a.heads);
  if (x < wide_groups)
    attend_wide<kD, kF32, kWholePages>(a, h, item / a.wide_splits, (int)(item % a.wide_splits), lds.wide);
  else
    attend_rows<kD, kF32, kWholePages>(a, item - wide_groups / a.heads, h, 0, 1, lds.rows);
}

// Joins what was split: workgroups below `row_groups` take one request, KV head and
// row (z, strided) of the row kernel's items; the others kGroups rows of the wide
// kernel's each.  D / 4 threads cover a row.
template <int kD, bool kF32>
__device__ __forceinline__ void join_items(const AttendArgs& a, int64_t b, int h, int z, int nz) {
  constexpr int kQuads = kD / 4, kGroups = kThreads / kQuads;
  __shared__ float red_m[kWaves], red_l[kWaves];
  __shared__ f32x4 red_o[kGroups][kQuads];
  const Request first = lane_request(a, 0);
  const Item it = find_item<true>(a, b, split_units(a, first), first);
  if (it.count < 2) return;
  const Request rq = it.rq;
  const int rows = rq.n * a.group, tid = threadIdx.x, lane = tid & (kWave - 1);
  const int quad = tid % kQuads, grp = tid / kQuads;   // every kGroups-th item; the sums meet in LDS
  const int64_t step = (int64_t)a.heads * a.part_rows;
  for (int row = z; row < rows; row += nz) {
    const int64_t slot0 = (it.first * a.heads + h) * a.part_rows + row;
    float M = -INFINITY, L = 0;
    for (int i = tid; i < it.count; i += kThreads) {
      const int64_t slot = slot0 + i * step;
      const float mi = a.part_ml[2 * slot], top = fmaxf(M, mi);
      L = L * part_weight(M, top, a.c) + a.part_ml[2 * slot + 1] * part_weight(mi, top, a.c);
      M = top;
    }
    const float mine = M;
    M = wave_fold(M, [](float x, float y) { return fmaxf(x, y); });
    L = wave_fold(L * part_weight(mine, M, a.c), [](float x, float y) { return x + y; });
    __syncthreads();  // the last row's reads of LDS are done
    if (lane == 0) {
      red_m[tid / kWave] = M;
      red_l[tid / kWave] = L;
    }
    __syncthreads();
    L = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) M = fmaxf(M, red_m[w]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) L += red_l[w] * part_weight(red_m[w], M, a.c);
    const float inv = L > 0 ? recip_rn(L) : 0.0f;
    f32x4 acc = {0, 0, 0, 0};
    if (grp < kGroups) {
      for (int i = grp; i < it.count; i += kGroups) {
        const int64_t slot = slot0 + i * step;
        const float wt = a.part_ml[2 * slot + 1] * inv * part_weight(a.part_ml[2 * slot], M, a.c);
        acc += *reinterpret_cast<const f32x4*>(a.part_o + slot * kD + 4 * quad) * wt;
      }
      red_o[grp][quad] = acc;
    }
    __syncthreads();
    if (grp == 0) {
#pragma unroll
      for (int g = 1; g < kGroups; ++g) acc += red_o[g][quad];
      const float v[4] = {acc[0], acc[1], acc[2], acc[3]};
      store_row<kF32, 4>(a.out, ((int64_t)(rq.start + row / a.group) * a.heads * a.group + h * a.group +
                                 row % a.group) * kD + 4 * quad, v);
    }
  }
}

template <int kD, bool kF32>
__device__ __forceinline__ void join_wide(const AttendArgs& a, int64_t group) {
  constexpr int kQuads = kD / 4, kGroups = kThreads / kQuads;
  const int tid = threadIdx.x, quad = tid % kQuads, grp = tid / kQuads, q_heads = a.heads * a.group;
  const int64_t total = a.q_rows * q_heads, at = group * kGroups + grp;
  const bool inside = grp < kGroups && at < total;
  const int t = inside ? (int)(at / q_heads) : -1, g = (int)(at % q_heads) % a.group;
  // the request of each row's query token, all of the wave's at once
  Request rq{0, 0, 0};
  for (int64_t b0 = 0; b0 < a.batch; b0 += kWave) {
    const Request r = lane_request(a, b0);
    uint64_t left = __ballot(inside);
    while (left) {   // one token a turn
      const int ts = __builtin_amdgcn_readlane(t, __builtin_ctzll(left));
      const uint64_t m = __ballot(ts >= r.start && ts < r.start + r.n);
      if (m && t == ts) rq = from_lane(r, __builtin_ctzll(m));
      left &= ~__ballot(t == ts);
    }
  }
  const int rows = rq.n * a.group, tok = t - rq.start;
  if (!inside || rows <= a.part_rows) return;
  const int last = min((tok * a.group + g) / kWideTile * kWideTile + kWideTile, rows) - 1;
  const int n = wide_split(a, a.causal ? rq.kv - rq.n + 1 + last / a.group : rq.kv).count;
  if (n < 2) return;
  float M = -INFINITY, L = 0;
  f32x4 acc = {0, 0, 0, 0};
  for (int i0 = 0; i0 < n; i0 += 4) {   // four parts' loads at a time
    float mi[4], li[4];
    f32x4 oi[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t slot = (int64_t)min(i0 + k, n - 1) * total + at;
      mi[k] = i0 + k < n ? a.wide_ml[2 * slot] : -INFINITY;
      li[k] = a.wide_ml[2 * slot + 1];
      oi[k] = *reinterpret_cast<const f32x4*>(a.wide_o + slot * kD + 4 * quad);
    }
    const float top = fmaxf(M, fmaxf(fmaxf(mi[0], mi[1]), fmaxf(mi[2], mi[3])));
    // the average so far, and the parts', by their shares of p
    const float keep = L * part_weight(M, top, a.c);
    L = keep;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      li[k] *= part_weight(mi[k], top, a.c);
      L += li[k];
    }
    const float inv = L > 0 ? recip_rn(L) : 0.0f;
    acc *= keep * inv;
#pragma unroll
    for (int k = 0; k < 4; ++k) acc += oi[k] * (li[k] * inv);
    M = top;
  }
  const float v[4] = {acc[0], acc[1], acc[2], acc[3]};
  store_row<kF32, 4>(a.out, at * kD + 4 * quad, v);
}

template <int kD, bool kF32>
__global__ __launch_bounds__(kThreads) void k_attend_join(const AttendArgs a, int64_t row_groups, int nz) {
  const int64_t x = blockIdx.x;
  if (x < row_groups) {
    const int64_t bh = x / nz;
    join_items<kD, kF32>(a, bh / a.heads, (int)(bh % a.heads), (int)(x % nz), nz);
  } else if constexpr (wide_takes(kD, !kF32)) {
    join_wide<kD, kF32>(a, x - row_groups);
  }
}

bool may_split(int64_t width, int shift) { return (width << shift) > (int64_t)kMinUnits * kUnit; }

// How a call is laid out; the workspace query and the launch agree on it.
struct Plan {
  bool wide;
  int part_rows;       // most rows of a request that the row kernel splits
  int64_t items;       // of the row kernel (0: nothing can be split)
  int wide_splits;
  size_t part_o, part_ml, wide_o, wide_ml, bytes;   // floats before each part, and all bytes
};

// Tiles that the lengths can lead to: one more than whole ones for each request.
int64_t wide_tiles(int64_t q_rows, int64_t batch, int64_t group) {
  return q_rows * group / kWideTile + std::min(batch, q_rows);
}

Plan plan_of(int64_t q_rows, int64_t batch, int64_t heads, int64_t group, int64_t max_rows, int64_t width,
             int shift, int head_dim, bool bf16) {
  Plan p{};
  p.wide = max_rows > kTile && wide_takes(head_dim, bf16);
  const int64_t most = p.wide ? kTile : kMaxPartRows;
  p.part_rows = (int)((max_rows < most ? max_rows + kTile - 1 : most) / kTile * kTile);
  p.items = may_split(width, shift) ? most_items(batch, heads, width, shift) : 0;
  p.wide_splits = 1;
  if (p.wide && (width << shift) > (int64_t)kMinWideUnits * kUnit) {
    const int64_t groups = (q_rows * group + kWideTile - 1) / kWideTile * heads;
    const int64_t most = kMaxGroups / (wide_tiles(q_rows, batch, group) * heads);
    p.wide_splits = (int)std::max<int64_t>(1, std::min<int64_t>({kMaxWideSplits, kWideGroupsWanted / groups, most}));
  }
  const size_t rows = (size_t)p.items * heads * p.part_rows;
  const size_t wide = p.wide_splits > 1 ? (size_t)p.wide_splits * q_rows * heads * group : 0;
  p.part_ml = rows * head_dim;
  p.wide_o = p.part_ml + (rows * 2 + 3) / 4 * 4;
  p.wide_ml = p.wide_o + wide * head_dim;
  p.bytes = 4 * (p.wide_ml + wide * 2);
  return p;
}

template <int kD, bool kF32, bool kWholePages>
void run_parts(const AttendArgs& a, const Plan& p, int64_t max_rows, hipStream_t st) {
  const int64_t items = p.items ? p.items : a.batch;
  if constexpr (wide_takes(kD, !kF32)) {
    if (p.wide) {
      const int64_t wide_groups = wide_tiles(a.q_rows, a.batch, a.group) * p.wide_splits * a.heads;
      hipLaunchKernelGGL((k_attend_both<kD, kF32, kWholePages>), dim3((unsigned)(wide_groups + items * a.heads)),
                         dim3(kThreads), 0, st, a, wide_groups);
      return;
    }
  }
  const int64_t tiles = (max_rows + kTile - 1) / kTile;
  hipLaunchKernelGGL((k_attend_rows<kD, kF32, kWholePages>),
                     dim3((unsigned)items, (unsigned)a.heads, (unsigned)(tiles < 64 ? tiles : 64)), dim3(kThreads), 0,
                     st, a);
}

template <int kD, bool kF32>
hipError_t run(const AttendArgs& a, const Plan& p, int64_t max_rows, hipStream_t st) {
  if ((1 << a.shift) >= kUnit)
    run_parts<kD, kF32, true>(a, p, max_rows, st);
  else
    run_parts<kD, kF32, false>(a, p, max_rows, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!p.items && p.wide_splits == 1)) return e;
  constexpr int64_t kJoinRows = kThreads / (kD / 4);
  // Rows of a request that are joined beside each other.  Beside the wide kernel these are
  // mostly single tokens' (a row for each query head), and most requests have none: 16
  // workgroups for each delayed the wide rows (cross attention 38.7 us, with 4 36.0).
  const int64_t beside = p.wide ? std::min<int64_t>(std::max<int64_t>(a.group, 4), 16) : 16;
  const int nz = (int)std::max<int64_t>(1, std::min<int64_t>({max_rows, beside, kMaxGroups / (a.batch * a.heads)}));
  const int64_t row_groups = p.items ? a.batch * a.heads * nz : 0;
  const int64_t wide_groups =
      p.wide_splits > 1 ? (a.q_rows * a.heads * a.group + kJoinRows - 1) / kJoinRows : 0;
  hipLaunchKernelGGL((k_attend_join<kD, kF32>), dim3((unsigned)(row_groups + wide_groups)), dim3(kThreads), 0, st, a,
                     row_groups, nz);
  return hipGetLastError();
}

template <bool kF32>
hipError_t run_d(const AttendArgs& a, const Plan& p, int head_dim, int64_t max_rows, hipStream_t st) {
  switch (head_dim) {
    case 64: return run<64, kF32>(a, p, max_rows, st);
    case 128: return run<128, kF32>(a, p, max_rows, st);
    case 192: return run<192, kF32>(a, p, max_rows, st);
    default: return run<256, kF32>(a, p, max_rows, st);
  }
}

}  // namespace

size_t attend_workspace_bytes(int64_t q_rows, int64_t batch, int64_t heads, int64_t group, int64_t max_rows,
                              int64_t width, int shift, int head_dim, bool bf16) {
  if (batch == 0 || q_rows == 0) return 0;
  return plan_of(q_rows, batch, heads, group, max_rows, width, shift, head_dim, bf16).bytes;
}

hipError_t launch_attend(AttendArgs a, bool bf16, int head_dim, int64_t max_rows, void* workspace,
                         hipStream_t st) {
  const Plan p = plan_of(a.q_rows, a.batch, a.heads, a.group, max_rows, a.width, a.shift, head_dim, bf16);
  float* ws = (float*)workspace;
  a.part_rows = p.part_rows;
  a.part_o = ws;
  a.part_ml = ws + p.part_ml;
  a.wide = p.wide;
  a.wide_splits = p.wide_splits;
  a.wide_o = ws + p.wide_o;
  a.wide_ml = ws + p.wide_ml;
  // Scale 0: all scores 0, set before the mask, whose -inf has to stay -inf through the
  // product.
  if (a.c == 0) {
    a.flat = 1;
    a.c = 1;
  }
  return bf16 ? run_d<false>(a, p, head_dim, max_rows, st) : run_d<true>(a, p, head_dim, max_rows, st);
}

}  // namespace pqb
