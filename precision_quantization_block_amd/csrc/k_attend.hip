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
// P is rounded to f16 as 2^15 p: 11 significant bits for every p >= 2^-29, three
// more than bf16 has, and below that to 2^-40 of the largest (float32 rows add
// the rounding's remainder as a second f16 part).  V enters as dec(c) 2^(X - R),
// exact in f16 unless X is over 15 below R, the largest V exponent met so far; O
// is kept in units of 2^R and rescaled when R or the row's maximum rises.
#include "launch.h"
#include "paged.h"

namespace pqb {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kUnit = 64;        // tokens a wave takes at a time
constexpr int kTile = 16;        // query rows of a tile
constexpr int kWaves = 4, kThreads = kWaves * kWave;
constexpr int kMinUnits = kWaves;                 // fewest units of a split
constexpr int kMaxPartRows = 64;                  // rows of a request that may be split
constexpr int64_t kGroupsWanted = 1024;           // workgroups a split aims at

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
  if (rows > a.part_rows) return 1;
  return max(1, (units_of(r.kv) + C - 1) / C);
}

__device__ __forceinline__ int64_t wave_sum64(int64_t v) {
#pragma unroll
  for (int d = kWave / 2; d; d >>= 1) v += (int64_t)__shfl_xor((long long)v, d);
  return v;
}

__device__ __forceinline__ int split_units(const AttendArgs& a) {
  const int lane = threadIdx.x & (kWave - 1);
  int64_t total = 0;
  for (int64_t b = lane; b < a.batch; b += kWave) {
    const Request r = request(a, b);
    const int64_t rows = (int64_t)r.n * a.group;
    if (rows > 0 && rows <= a.part_rows) total += units_of(r.kv);
  }
  total = wave_sum64(total) * a.heads;
  const int64_t c = (total + kGroupsWanted - 1) / kGroupsWanted;
  return (int)((max(c, (int64_t)kMinUnits) + kWaves - 1) / kWaves * kWaves);
}

struct Item {
  int64_t b, first;      // request, and its first item
  int32_t index, count;  // this item among the request's
};

// Item x (or, by_request, the items of request x); b = -1 if there is none.
template <bool kByRequest>
__device__ __forceinline__ Item find_item(const AttendArgs& a, int64_t x, int C) {
  const int lane = threadIdx.x & (kWave - 1);
  int64_t base = 0;
  for (int64_t b0 = 0; b0 < a.batch; b0 += kWave) {
    const int64_t b = b0 + lane;
    const int mine = b < a.batch ? items_of(a, request(a, b), C) : 0;
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
      const int cnt = __shfl(mine, src), upto = __shfl(incl, src);
      Item it;
      it.b = b0 + src;
      it.first = base + upto - cnt;
      it.index = kByRequest ? 0 : (int32_t)(x - it.first);
      it.count = cnt;
      return it;
    }
    base += __shfl(incl, kWave - 1);
  }
  return Item{-1, 0, 0, 0};
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

// One workgroup: an item's units for one KV head, its waves taking every fourth
// unit, 16 query rows at a time; the waves' partial results meet in LDS.
template <int kD, bool kF32>
__global__ __launch_bounds__(kThreads) void k_attend_rows(const AttendArgs a) {
  constexpr int kKC = kD / 64;    // 16-byte key loads of a lane per 16-row tile
  constexpr int kDT = kD / 16;    // 16-channel tiles of O
  constexpr int kParts = kF32 ? 3 : 1;
  constexpr int kLd = kD + 4;
  __shared__ float lds_o[kWaves][kTile][kLd];
  __shared__ float lds_m[kWaves][kTile], lds_l[kWaves][kTile];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int col = lane & 15, g4 = lane >> 4;
  const int h = blockIdx.y;

  const int C = split_units(a);
  const Item it = find_item<false>(a, blockIdx.x, C);
  if (it.b < 0) return;
  const Request rq = request(a, it.b);
  const int32_t rows = rq.n * a.group;
  const int all_units = units_of(rq.kv);
  const int unit0 = it.count == 1 ? 0 : it.index * C;
  const int unit_end = it.count == 1 ? all_units : min(all_units, unit0 + C);
  const int32_t* table = a.table + it.b * a.width;
  const int64_t tile_bytes = (int64_t)kD << a.shift;
  const int ps1 = (1 << a.shift) - 1;

  for (int rt = blockIdx.z; rt * kTile < rows; rt += gridDim.z) {
    const int row = rt * kTile + col;
    const bool valid = row < rows;
    const int tok = row / a.group, hq = h * a.group + row % a.group;
    bf16x8 qf[2 * kKC][kParts];
#pragma unroll
    for (int s = 0; s < 2 * kKC; ++s)
      load_q8<kF32>(a.q, (int64_t)(rq.start + tok) * a.q_stride + (int64_t)hq * kD + (s >> 1) * 64 + g4 * 16 + (s & 1) * 8,
                    valid, qf[s]);
    // what this lane's row, the tile's first row and its last row see
    const int ahead = rq.kv - rq.n + 1;
    const int limit = !valid ? 0 : a.causal ? ahead + tok : rq.kv;
    const int first_limit = a.causal ? ahead + rt * kTile / a.group : rq.kv;
    const int last_limit = a.causal ? ahead + (min(rt * kTile + kTile, rows) - 1) / a.group : rq.kv;
    const int end = min(unit_end, last_limit > 0 ? units_of(last_limit) : 0);

    float m = -INFINITY, l = 0;
    int R = 1;
    f32x4 o[kDT];
#pragma unroll
    for (int i = 0; i < kDT; ++i) o[i] = f32x4{0, 0, 0, 0};

    for (int u = unit0 + wave; u < end; u += kWaves) {
      // the page of this lane's key rows (group col / 4) and of its V tokens (group g4)
      const int tk = u * kUnit + 16 * (col >> 2), tv = u * kUnit + 16 * g4;
      const int pk0 = tk < rq.kv ? table[tk >> a.shift] : -1, pv0 = tv < rq.kv ? table[tv >> a.shift] : -1;
      const bool okk = (uint32_t)pk0 < (uint64_t)a.pages, okv = (uint32_t)pv0 < (uint64_t)a.pages;
      const int64_t pk = (int64_t)(okk ? pk0 : 0) * a.heads + h, pv = (int64_t)(okv ? pv0 : 0) * a.heads + h;
      uint4 kw[4][kKC], vw[kDT];
      const uint8_t* kp = a.k_codes + pk * tile_bytes + (int64_t)((tk & ps1) + (col & 3)) * kD + g4 * 16;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < kKC; ++i) kw[t][i] = *reinterpret_cast<const uint4*>(kp + 4 * t * kD + 64 * i);
      const uint8_t* vp = a.v_codes + pv * tile_bytes + ((int64_t)col << a.shift) + (tv & ps1);
#pragma unroll
      for (int i = 0; i < kDT; ++i)
        vw[i] = *reinterpret_cast<const uint4*>(vp + ((int64_t)i << (a.shift + 4)));
      const float sk = e8m0_pow2(a.k_scales[pk]);
      const int xv = min(max((int)a.v_scales[pv], 1), 254);

      f32x4 s[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        s[t] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < kKC; ++i) {
          const bf16x8 k0 = codes_bf16(kw[t][i].x, kw[t][i].y, sk), k1 = codes_bf16(kw[t][i].z, kw[t][i].w, sk);
#pragma unroll
          for (int p = kParts - 1; p >= 0; --p) {
            s[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, qf[2 * i][p], s[t], 0, 0, 0);
            s[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, qf[2 * i + 1][p], s[t], 0, 0, 0);
          }
        }
      }
      // Tokens outside the row's view, and tokens of a page id outside the cache.
      const bool whole = (u + 1) * kUnit <= first_limit && __ballot(!okv) == 0;
      uint32_t seen = 0xFFFFu;
      if (!whole) {
        const int cnt = okv ? min(max(limit - tv, 0), 16) : 0, held = okv ? min(max(rq.kv - tv, 0), 16) : 0;
        seen = (1u << cnt) - 1;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!((seen >> (4 * t + i)) & 1)) s[t][i] = -INFINITY;
        // codes behind the last token may be anything (NaN times p = 0 is NaN)
        uint32_t keep[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int nb = min(max(held - 4 * w, 0), 4);
          keep[w] = nb == 4 ? ~0u : (1u << (8 * nb)) - 1;
        }
#pragma unroll
        for (int i = 0; i < kDT; ++i) {
          vw[i].x &= keep[0];
          vw[i].y &= keep[1];
          vw[i].z &= keep[2];
          vw[i].w &= keep[3];
        }
      }
      float mx = max3f(s[0][0], s[0][1], s[0][2]);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = (t == 0 ? 3 : 0); i < 4; ++i) mx = fmaxf(mx, s[t][i]);
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      int xr = okv ? xv : 1;
      xr = max(xr, __shfl_xor(xr, 16));
      xr = max(xr, __shfl_xor(xr, 32));
      const float m_new = fmaxf(m, mx), top = m_new == -INFINITY ? 0.0f : m_new;
      const float alpha = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m - top) * a.c);
      const int R_new = max(R, xr);
      const float grow = R_new - R > 126 ? 0.0f : as_f((uint32_t)(127 - (R_new - R)) << 23);
      const float sv = as_f((uint32_t)(127 - min(max(R_new - xv, 0), 60)) << 23);
      m = m_new;
      R = R_new;
      float p[16], sum = 0;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e >> 2][e & 3] - top, a.c, 15.0f));
        if (!whole && !((seen >> e) & 1)) p[e] = 0;
        sum += p[e];
      }
      l = l * alpha + sum;
      const float f = alpha * grow;
      if (__ballot(f != 1.0f)) {
#pragma unroll
        for (int i = 0; i < kDT; ++i) o[i] *= f;
      }
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        uint32_t ph[4], pl[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x = p[8 * st + 2 * j], y = p[8 * st + 2 * j + 1];
          ph[j] = cvt_f16x2(x, y);
          if constexpr (kF32) {
            const f16x2 hi = __builtin_bit_cast(f16x2, ph[j]);
            pl[j] = cvt_f16x2(x - (float)hi[0], y - (float)hi[1]);
          }
        }
        const f16x8 pf = __builtin_bit_cast(f16x8, make_uint4(ph[0], ph[1], ph[2], ph[3]));
#pragma unroll
        for (int i = 0; i < kDT; ++i) {
          const f16x8 vf = st ? codes_f16(vw[i].z, vw[i].w, sv) : codes_f16(vw[i].x, vw[i].y, sv);
          if constexpr (kF32)
            o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                vf, __builtin_bit_cast(f16x8, make_uint4(pl[0], pl[1], pl[2], pl[3])), o[i], 0, 0, 0);
          o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pf, o[i], 0, 0, 0);
        }
      }
    }

    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    const float unit = as_f((uint32_t)R << 23) * 0x1p-15f;  // O and l in units of 1 from here on
    if (rt != (int)blockIdx.z) __syncthreads();  // the last tile's reads of LDS are done
#pragma unroll
    for (int i = 0; i < kDT; ++i)
      *reinterpret_cast<f32x4*>(&lds_o[wave][col][16 * i + 4 * g4]) = o[i] * unit;
    if (g4 == 0) {
      lds_m[wave][col] = m;
      lds_l[wave][col] = l * 0x1p-15f;
    }
    __syncthreads();
    // 16 threads a row, kD / 16 channels each
    const int r = tid / 16, d0 = (tid % 16) * (kD / 16), grow_row = rt * kTile + r;
    if (grow_row < rows) {
      float M = lds_m[0][r];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) M = fmaxf(M, lds_m[w][r]);
      float L = 0, acc[kD / 16];
#pragma unroll
      for (int j = 0; j < kD / 16; ++j) acc[j] = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float mw = lds_m[w][r], wt = mw == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((mw - M) * a.c);
        L += lds_l[w][r] * wt;
#pragma unroll
        for (int j = 0; j < kD / 16; ++j) acc[j] += lds_o[w][r][d0 + j] * wt;
      }
      if (it.count == 1) {
        const float inv = L > 0 ? 1.0f / L : 0.0f;
#pragma unroll
        for (int j = 0; j < kD / 16; ++j) acc[j] *= inv;
        store_row<kF32, kD / 16>(a.out, ((int64_t)(rq.start + grow_row / a.group) * a.heads * a.group +
                                         h * a.group + grow_row % a.group) * kD + d0, acc);
      } else {
        const int64_t slot = ((int64_t)blockIdx.x * a.heads + h) * a.part_rows + grow_row;
        store_row<true, kD / 16>(a.part_o, slot * kD + d0, acc);
        if (tid % 16 == 0) {
          a.part_ml[2 * slot] = M;
          a.part_ml[2 * slot + 1] = L;
        }
      }
    }
  }
}

// Joins the items of each split request: one workgroup per request and KV head.
template <int kD, bool kF32>
__global__ __launch_bounds__(kThreads) void k_attend_join(const AttendArgs a) {
  const int h = blockIdx.y, C = split_units(a);
  const Item it = find_item<true>(a, blockIdx.x, C);
  if (it.count < 2) return;
  const Request rq = request(a, it.b);
  const int rows = rq.n * a.group, tid = threadIdx.x;
  for (int e = tid; e < rows * (kD / 4); e += kThreads) {
    const int row = e / (kD / 4), d = e % (kD / 4) * 4;
    const int64_t step = (int64_t)a.heads * a.part_rows;
    const int64_t slot0 = (it.first * a.heads + h) * a.part_rows + row;
    float M = -INFINITY;
    for (int i = 0; i < it.count; ++i) M = fmaxf(M, a.part_ml[2 * (slot0 + i * step)]);
    float L = 0, acc[4] = {0, 0, 0, 0};
    for (int i = 0; i < it.count; ++i) {
      const int64_t slot = slot0 + i * step;
      const float mi = a.part_ml[2 * slot], wt = mi == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((mi - M) * a.c);
      const uint4 w = *reinterpret_cast<const uint4*>(a.part_o + slot * kD + d);
      L += a.part_ml[2 * slot + 1] * wt;
      acc[0] += as_f(w.x) * wt;
      acc[1] += as_f(w.y) * wt;
      acc[2] += as_f(w.z) * wt;
      acc[3] += as_f(w.w) * wt;
    }
    const float inv = L > 0 ? 1.0f / L : 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] *= inv;
    store_row<kF32, 4>(a.out, ((int64_t)(rq.start + row / a.group) * a.heads * a.group + h * a.group +
                               row % a.group) * kD + d, acc);
  }
}

int64_t most_items(int64_t batch, int64_t heads) { return (kGroupsWanted + heads - 1) / heads + batch; }

bool may_split(int64_t width, int shift) { return (width << shift) > (int64_t)kMinUnits * kUnit; }

int part_rows_of(int64_t max_rows) {
  return (int)((max_rows < kMaxPartRows ? max_rows + kTile - 1 : kMaxPartRows) / kTile * kTile);
}

template <int kD, bool kF32>
hipError_t run(const AttendArgs& a, int64_t max_rows, hipStream_t st) {
  const int64_t tiles = (max_rows + kTile - 1) / kTile;
  const dim3 grid((unsigned)(a.part_o ? most_items(a.batch, a.heads) : a.batch), (unsigned)a.heads,
                  (unsigned)(tiles < 64 ? tiles : 64));
  hipLaunchKernelGGL((k_attend_rows<kD, kF32>), grid, dim3(kThreads), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.part_o) return e;
  hipLaunchKernelGGL((k_attend_join<kD, kF32>), dim3((unsigned)a.batch, (unsigned)a.heads), dim3(kThreads), 0,
                     st, a);
  return hipGetLastError();
}

template <bool kF32>
hipError_t run_d(const AttendArgs& a, int head_dim, int64_t max_rows, hipStream_t st) {
  switch (head_dim) {
    case 64: return run<64, kF32>(a, max_rows, st);
    case 128: return run<128, kF32>(a, max_rows, st);
    case 192: return run<192, kF32>(a, max_rows, st);
    default: return run<256, kF32>(a, max_rows, st);
  }
}

}  // namespace

size_t attend_workspace_bytes(int64_t batch, int64_t heads, int64_t max_rows, int64_t width, int shift,
                              int head_dim) {
  if (!may_split(width, shift) || batch == 0 || max_rows == 0) return 0;
  return (size_t)most_items(batch, heads) * heads * part_rows_of(max_rows) * (head_dim + 2) * 4;
}

hipError_t launch_attend(AttendArgs a, bool bf16, int head_dim, int64_t max_rows, void* workspace,
                         hipStream_t st) {
  a.part_rows = part_rows_of(max_rows);
  a.part_o = a.part_ml = nullptr;
  if (may_split(a.width, a.shift)) {
    a.part_o = (float*)workspace;
    a.part_ml = a.part_o + (size_t)most_items(a.batch, a.heads) * a.heads * a.part_rows * head_dim;
  }
  return bf16 ? run_d<false>(a, head_dim, max_rows, st) : run_d<true>(a, head_dim, max_rows, st);
}

}  // namespace pqb
