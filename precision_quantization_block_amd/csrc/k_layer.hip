// What a decoder layer does between its products, fused with the quantization of
// the next product's activations: norms with their residual and gate (k_norm), and
// gated activations (k_act_row, k_act_flat).
//
//   y = x, or N(x) post                   h = RN_T(gate y + c residual)
//   RMS:   u = h w,        r = (mean h^2 + eps)^-1/2,            value u r
//   layer: u = (h - mu) r w + b,   r = (mean (h - mu)^2 + eps)^-1/2,   value u
//   act:   u = f(g) up
//
// Codes are those of the quantizers: s = max(amax |u|, 1e-12) / M over a row or 128
// columns and Q(RN(u / s)).  An RMS norm's r is common to the row, so it cancels
// in the codes: they are formed from u, before r is known, and the stored scale is
// s r.  So an RMS norm's codes depend on no sum.
//
// A row stays in registers (kU units of 8 elements a thread) from its one read to its one
// write; the row's sums and maxima meet by DPP, two shuffles and one LDS exchange.  A
// workgroup has one row and as many waves as that takes, or several narrow ones (a wave or part
// of one each).  All of it is bound by HBM, and by latency where there are few rows:
// 8192 rows of 7168 (bf16, residual, E4M3 1x128) 70 us, 5.9 TB/s; 4096 rows of 14336 through
// SwiGLU to E4M3 1x128 53 us, 5.5 TB/s; 64 rows of 4096 to INT8 3.7 us.  (Norms of more than 16384
// columns, four units to each of 1024 threads, pass the 128 registers that leaves them by 14 to 37, which
// are spilled: 1024 rows of 32768, bf16, with residual to INT8 70 us, 3.4 TB/s; 2048 of 16384 50 us,
// 4.7.)
#include "launch.h"
#include "quant.h"

namespace pqb {
namespace {

// ---------------------------------------------------------------------------
// A row in registers: unit k of thread t of n is elements 8 (k n + t) ....  kVec: units are whole
// and 16-byte aligned.  Otherwise (odd widths, strides or addresses) the same accesses at the
// elements' own alignment, which this GPU's memory instructions allow; a row's last unit is
// loaded with the elements in front of it, and stored one by one.  (One by one throughout, 8192
// rows of 1005, bf16, with residual to INT8 31 us, 14 so; 2048 of 4097 45 and 17.)
// ---------------------------------------------------------------------------
struct Who {
  int t, n;
};
__device__ __forceinline__ int elem_at(int k, int j, Who w) { return 8 * (k * w.n + w.t) + j; }

__device__ __forceinline__ Raw8 load_cached8(const uint16_t* p) {
  return Raw8{*reinterpret_cast<const uint4*>(p), make_uint4(0, 0, 0, 0)};
}
__device__ __forceinline__ Raw8 load_cached8(const float* p) {
  return Raw8{*reinterpret_cast<const uint4*>(p), *reinterpret_cast<const uint4*>(p + 4)};
}

// 16 and 8 bytes at the alignment of what they hold (no hints: neighbours share the lines).
typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_at4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_at1 __attribute__((ext_vector_type(2), aligned(1)));
__device__ __forceinline__ Raw8 load_any8(const uint16_t* p) {
  const u32x4_at2 w = *reinterpret_cast<const u32x4_at2*>(p);
  return Raw8{make_uint4(w.x, w.y, w.z, w.w), make_uint4(0, 0, 0, 0)};
}
__device__ __forceinline__ Raw8 load_any8(const float* p) {
  const u32x4_at4 w = reinterpret_cast<const u32x4_at4*>(p)[0], z = reinterpret_cast<const u32x4_at4*>(p)[1];
  return Raw8{make_uint4(w.x, w.y, w.z, w.w), make_uint4(z.x, z.y, z.z, z.w)};
}

// The elements of a unit from d on (below 8), zeros behind them.
__device__ __forceinline__ Raw8 without(Raw8 r, const uint16_t*, int d) {
  if (d & 4) r.a = make_uint4(r.a.z, r.a.w, 0, 0);
  if (d & 2) r.a = make_uint4(r.a.y, r.a.z, r.a.w, 0);
  if (d & 1)
    r.a = make_uint4(r.a.x >> 16 | r.a.y << 16, r.a.y >> 16 | r.a.z << 16, r.a.z >> 16 | r.a.w << 16, r.a.w >> 16);
  return r;
}
__device__ __forceinline__ Raw8 without(Raw8 r, const float*, int d) {
  if (d & 4) r = Raw8{r.b, make_uint4(0, 0, 0, 0)};
  if (d & 2) r = Raw8{make_uint4(r.a.z, r.a.w, r.b.x, r.b.y), make_uint4(r.b.z, r.b.w, 0, 0)};
  if (d & 1) r = Raw8{make_uint4(r.a.y, r.a.z, r.a.w, r.b.x), make_uint4(r.b.y, r.b.z, r.b.w, 0)};
  return r;
}

// A row's units as loaded, and as floats: apart, so that several arrays' loads are on their way
// before the first is waited for.  kOnce: read by this thread only (non-temporal); else shared with
// other rows.  `front` elements of the row lie in front of p.
template <bool kVec, int kU, bool kOnce, typename T>
__device__ __forceinline__ void fetch(const T* __restrict__ p, int cols, Who t, Raw8 (&raw)[kU], int front = 0) {
  if (!kVec && kU == 1 && front + cols < 8) {   // (such rows have one unit a thread)
    uint32_t x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = elem_at(0, j, t) < cols ? as_u(ld1(p + elem_at(0, j, t))) : 0;
    if constexpr (sizeof(T) == 2)
      raw[0] = Raw8{make_uint4(x[0] >> 16 | x[1], x[2] >> 16 | x[3], x[4] >> 16 | x[5], x[6] >> 16 | x[7]), {}};
    else raw[0] = Raw8{make_uint4(x[0], x[1], x[2], x[3]), make_uint4(x[4], x[5], x[6], x[7])};
    return;
  }
#pragma unroll
  for (int k = 0; k < kU; ++k) {
    const int e = elem_at(k, 0, t);
    if constexpr (kVec) raw[k] = e < cols ? (kOnce ? load_raw8(p + e) : load_cached8(p + e)) : Raw8{};
    else raw[k] = e < cols ? load_any8(p + min(e, cols - 8)) : Raw8{};
  }
}
template <bool kVec, int kU, typename T>
__device__ __forceinline__ void widen(const T* p, int cols, Who t, const Raw8 (&raw)[kU], float (&v)[kU][8], int front = 0) {
#pragma unroll
  for (int k = 0; k < kU; ++k) {
    const int e = elem_at(k, 0, t);
    Raw8 r = raw[k];
    if (!kVec && front + cols >= 8 && e < cols && e > cols - 8) r = without(r, p, e - (cols - 8));
    widen8(r, p, v[k]);
  }
}
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = (uint16_t)(bf16x2_rne(v, 0.0f) & 0xFFFFu); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ float rounded(const uint16_t*, float v) { return as_f(bf16x2_rne(v, 0.0f) << 16); }
__device__ __forceinline__ float rounded(const float*, float v) { return v; }

__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  st_nt16(p, bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  st_nt16(p, as_u(v[0]), as_u(v[1]), as_u(v[2]), as_u(v[3]));
  st_nt16(p + 4, as_u(v[4]), as_u(v[5]), as_u(v[6]), as_u(v[7]));
}
__device__ __forceinline__ void store_any8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<u32x4_at2*>(p) =
      u32x4_at2{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7])};
}
__device__ __forceinline__ void store_any8(float* p, const float (&v)[8]) {
  reinterpret_cast<u32x4_at4*>(p)[0] = u32x4_at4{as_u(v[0]), as_u(v[1]), as_u(v[2]), as_u(v[3])};
  reinterpret_cast<u32x4_at4*>(p)[1] = u32x4_at4{as_u(v[4]), as_u(v[5]), as_u(v[6]), as_u(v[7])};
}

template <bool kVec, int kU, typename T>
__device__ __forceinline__ void store_row(T* __restrict__ p, int cols, Who t, const float (&v)[kU][8]) {
#pragma unroll
  for (int k = 0; k < kU; ++k) {
    const int e = elem_at(k, 0, t);
    if constexpr (kVec) {
      if (e < cols) store8(p + e, v[k]);
    } else if (e + 8 <= cols) {
      store_any8(p + e, v[k]);
    } else {
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (e + j < cols) store1(p + e + j, v[k][j]);
    }
  }
}

// Eight codes of unit v with scale s.
template <int kElem>
__device__ __forceinline__ uint2 pack_as(const float (&v)[8], float s) {
  return fp8_pack8<kElem>(v, s, recip_rn(s));
}
__device__ __forceinline__ uint2 pack_codes(int elem, const float (&v)[8], float s) {
  return elem == kI8 ? pack_as<kI8>(v, s) : elem == kE4M3 ? pack_as<kE4M3>(v, s) : pack_as<kE5M2>(v, s);
}
__device__ __forceinline__ float scale_of(int elem, uint32_t amax) {
  return elem == kI8 ? fp8_scale_bits<kI8>(amax)
                     : elem == kE4M3 ? fp8_scale_bits<kE4M3>(amax) : fp8_scale_bits<kE5M2>(amax);
}

template <bool kVec, int kU>
__device__ __forceinline__ void store_codes(uint8_t* __restrict__ p, int cols, Who t, int elem, float s,
                                            const float (&v)[kU][8]) {
#pragma unroll
  for (int k = 0; k < kU; ++k) {
    const uint2 w = pack_codes(elem, v[k], s);
    const int e = elem_at(k, 0, t);
    if constexpr (kVec) {
      if (e < cols) st_nt8(p + e, w.x, w.y);
    } else if (e + 8 <= cols) {
      *reinterpret_cast<u32x2_at1*>(p + e) = u32x2_at1{w.x, w.y};
    } else {
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (e + j < cols) p[e + j] = (uint8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
    }
  }
}

// ---------------------------------------------------------------------------
// Reductions over the threads of a row; every thread receives the result.
// ---------------------------------------------------------------------------
struct SumMax {
  float sum;
  uint32_t max;
};
constexpr int kWaves = 16;   // at most, of a workgroup

// The sum and the largest bit pattern at once.  `red` (kWaves entries) is free to be
// written when the call starts; a second call takes another one.  kLanes: of a row, 8 to 64, or
// more for the whole workgroup.
template <int kLanes>
__device__ __forceinline__ SumMax row_reduce(float sum, uint32_t most, SumMax* red) {
  sum += as_f(dpp<kDppXor1>(as_u(sum)));
  sum += as_f(dpp<kDppXor2>(as_u(sum)));
  sum += as_f(dpp<kDppHalfMirror>(as_u(sum)));
  if constexpr (kLanes > 8) sum += as_f(dpp<kDppMirror>(as_u(sum)));
  most = group_umax<(kLanes > 8 ? 16 : 8)>(most);
#pragma unroll
  for (int far = 16; far < 64 && far < kLanes; far *= 2) {
    sum += __shfl_xor(sum, far);
    most = max(most, (uint32_t)__shfl_xor((int)most, far));
  }
  if constexpr (kLanes > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = SumMax{sum, most};
    __syncthreads();
    sum = 0.0f;
    most = 0;
    for (int i = 0; i < (int)blockDim.x >> 6; ++i) {
      sum += red[i].sum;
      most = max(most, red[i].max);
    }
  }
  return SumMax{sum, most};
}

template <int kU>
__device__ __forceinline__ uint32_t amax_of(const float (&v)[kU][8]) {
  float m = 0.0f;
#pragma unroll
  for (int k = 0; k < kU; ++k) m = __builtin_fmaxf(m, absmax8(v[k]));
  return as_u(m);
}

// (mean, r) of a row; kinds: RMS (mean 0) or layer.  v keeps its values, centred for a
// layer norm (elements behind the row stay 0).
template <int kLanes, int kU>
__device__ __forceinline__ float norm_stats(bool layer, float eps, int cols, Who t, float (&v)[kU][8],
                                            SumMax* red) {
  if (layer) {
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[k][j];
    const float mean = row_reduce<kLanes>(s, 0, red).sum / (float)cols;
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[k][j] = elem_at(k, j, t) < cols ? v[k][j] - mean : 0.0f;
  }
  float q = 0.0f;
#pragma unroll
  for (int k = 0; k < kU; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) q = __builtin_fmaf(v[k][j], v[k][j], q);
  const float ms = row_reduce<kLanes>(q, 0, red + kWaves).sum / (float)cols;
  return 1.0f / sqrtf(ms + eps);
}

// How rows are taken: by 8 to 64 lanes each, as many as 256 threads hold, or one by up to
// kMost threads; kU units a thread.
template <int kUnits, int kMost>
struct Shape {
  static constexpr int kU = kUnits, lanes = kMost, threads = kMost > 64 ? kMost : 256;
  static constexpr int rows = kMost > 64 ? 1 : 256 / kMost;
};

// This thread's row and place in it.
template <typename S>
__device__ __forceinline__ int64_t row_of(Who& t) {
  t = S::rows > 1 ? Who{(int)threadIdx.x & (S::lanes - 1), S::lanes} : Who{(int)threadIdx.x, (int)blockDim.x};
  return (int64_t)blockIdx.x * S::rows + (S::rows > 1 ? threadIdx.x / S::lanes : 0);
}

template <typename T, bool kVec, typename S>
__global__ __launch_bounds__(S::threads) void k_norm(NormArgs a) {
  constexpr int kU = S::kU, kLanes = S::lanes;
  __shared__ SumMax red[5 * kWaves];
  Who t;
  const int64_t row = row_of<S>(t);
  if (row >= a.rows) return;   // all of a row's lanes; no barrier with several rows

  // The loads of x and residual are on their way before the first sum; where they fit the
  // registers, so are those of all others
  constexpr bool kEarly = kU == 1;
  const T* post = reinterpret_cast<const T*>(a.post);
  const T* gate = a.gate ? reinterpret_cast<const T*>(a.gate) + (int64_t)((uint32_t)row / a.per_gate) * a.gate_stride
                         : nullptr;
  const T* weight = reinterpret_cast<const T*>(a.weight);
  const T* bias = reinterpret_cast<const T*>(a.bias);
  const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_stride;
  Raw8 raw_x[kU], raw_res[kU], raw_post[kU], raw_gate[kU], raw_weight[kU], raw_bias[kU];
  fetch<kVec, kU, true>(x, a.cols, t, raw_x);
  if (a.residual) fetch<kVec, kU, true>(reinterpret_cast<const T*>(a.residual) + row * a.res_stride, a.cols, t, raw_res);
  if (kEarly && post) fetch<kVec, kU, false>(post, a.cols, t, raw_post);
  if (kEarly && gate) fetch<kVec, kU, false>(gate, a.cols, t, raw_gate);
  if (kEarly && weight) fetch<kVec, kU, false>(weight, a.cols, t, raw_weight);
  if (kEarly && bias) fetch<kVec, kU, false>(bias, a.cols, t, raw_bias);
  auto get = [&](const T* p, Raw8 (&raw)[kU], float (&to)[kU][8]) {
    if (!kEarly) fetch<kVec, kU, false>(p, a.cols, t, raw);
    widen<kVec, kU>(p, a.cols, t, raw, to);
  };
  float v[kU][8];
  widen<kVec, kU>(x, a.cols, t, raw_x, v);
  const bool layer = a.layer;
  if (post) {
    const float r = norm_stats<kLanes, kU>(layer, a.eps, a.cols, t, v, red + 3 * kWaves);
    float w[kU][8];
    get(post, raw_post, w);
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] = v[k][j] * r * w[k][j];
  }
  if (gate) {
    float g[kU][8];
    get(gate, raw_gate, g);
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] *= g[k][j];
  }
  if (a.residual) {
    float res[kU][8];
    widen<kVec, kU>(x, a.cols, t, raw_res, res);
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] += res[k][j] * a.res_scale;
  }
  if (a.h) {
    T* h = reinterpret_cast<T*>(a.h) + row * a.h_stride;
    store_row<kVec, kU>(h, a.cols, t, v);
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] = rounded(h, v[k][j]);
  }

  // u, and r where it is not in u
  float w[kU][8];
  if (weight) {
    get(weight, raw_weight, w);
  } else {
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) w[k][j] = 1.0f;
  }
  float r = 1.0f;
  uint32_t most = 0;
  if (layer) {
    const float rl = norm_stats<kLanes, kU>(true, a.eps, a.cols, t, v, red);
    float b[kU][8] = {};
    if (bias) get(bias, raw_bias, b);
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] = v[k][j] * rl * w[k][j] + b[k][j];
    if (a.form == kFormRow) most = row_reduce<kLanes>(0.0f, amax_of(v), red + 2 * kWaves).max;
  } else {
    float q = 0.0f;
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        q = __builtin_fmaf(v[k][j], v[k][j], q);
        v[k][j] *= w[k][j];
      }
    const SumMax m = row_reduce<kLanes>(q, amax_of(v), red);
    r = 1.0f / sqrtf(m.sum / (float)a.cols + a.eps);
    most = m.max;
  }

  if (a.form == kFormPlain) {
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] *= r;
    store_row<kVec, kU>(reinterpret_cast<T*>(a.out) + row * a.cols, a.cols, t, v);
  } else if (a.form == kFormRow) {
    const float s = scale_of(a.elem, most);
    store_codes<kVec, kU>(reinterpret_cast<uint8_t*>(a.out) + row * a.cols, a.cols, t, a.elem, s, v);
    if (t.t == 0) a.scales[row] = s * r;
  } else if constexpr (kVec) {   // 1x128 blocks: 16 threads each (cols % 128 == 0)
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int e = elem_at(k, 0, t);
      const float s = scale_of(a.elem, group_umax<16>(as_u(absmax8(v[k]))));
      const uint2 c = pack_codes(a.elem, v[k], s);
      if (e < a.cols) {
        st_nt8(reinterpret_cast<uint8_t*>(a.out) + row * a.cols + e, c.x, c.y);
        if ((t.t & 15) == 0) a.scales[row * (a.cols / 128) + e / 128] = s * r;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Activations.  Each takes a few float32 roundings (silu and tanh-gelu as
// g / (1 + 2^-z): the product with log2(e) carries its rounding error along, since 2^z
// turns an absolute error into a relative one; tanh-gelu's z itself is rounded, which costs its tail
// |z| 2^-24 a rounding: 52 units at g = -6).
// ---------------------------------------------------------------------------
__device__ __forceinline__ float sigmoid_times(float g, float z) {
  z = __builtin_fminf(__builtin_fmaxf(z, -150.0f), 150.0f);      // 2^t is 0 or inf there
  constexpr float kL2e = 1.44269504088896341f, kL2eLo = 1.92596299112661746887e-8f;
  const float t = -z * kL2e;
  const float lo = __builtin_fmaf(-z, kL2e, -t) - z * kL2eLo;
  const float p = __builtin_amdgcn_exp2f(t);                     // 2^t (1 + lo ln 2) = exp(-z)
  const float d = 1.0f + __builtin_fmaf(p, lo * 0.693147180559945309f, p);
  const float y = __builtin_amdgcn_rcpf(d);
  const float q = g * y;                                         // one correction of g / d
  const float off = __builtin_fmaxf(__builtin_fmaf(-q, d, g), -3.4e38f);   // (the maximum: not NaN for infinite g)
  const float c = __builtin_fmaf(off, y, q);
  return d < 0x1p126f ? c : 0.0f * g;                            // exp(-z) overflows: -0 for finite g
}

// 0.5 g erfc(z), z = -g / sqrt 2.  For z > 0, erfc turns the rounding of z into a relative error some
// 2 z^2 times as large (76 units of 2^-24 at z = 6), so z's low part d is carried along: erfc(z + d) =
// erfc(z) (1 - d h), h = -erfc'(z) / erfc(z).  h is taken as 2 z: it is more by at most 1 / z, which
// with |d| <= z 2^-24 or so makes one rounding.
__device__ __forceinline__ float gelu_erf(float g) {
  constexpr float kRs2 = 0.707106781186547524f, kRs2Lo = 1.21016171e-8f;
  const float x = __builtin_amdgcn_fmed3f(g, -20.0f, 20.0f);     // erfc is 0 or 2 there; keeps d and z d finite
  const float z = -x * kRs2;
  const float d = __builtin_fmaf(-x, kRs2Lo, __builtin_fmaf(-x, kRs2, -z));
  const float e = erfcf(z);
  return 0.5f * g * __builtin_fmaf(__builtin_fmaxf(z, 0.0f) * d, -2.0f * e, e);
}

__device__ __forceinline__ float activate(int act, float g) {
  if (act == kActSilu) return sigmoid_times(g, g);
  if (act == kActGeluTanh) {
    // (1 + tanh(z)) / 2 = 1 / (1 + exp(-2 z)), z = sqrt(2 / pi) (g + 0.044715 g^3)
    const float g2 = __builtin_fminf(g * g, 1e10f);
    return sigmoid_times(g, 1.59576912160573072f * __builtin_fmaf(0.044715f * g2, g, g));
  }
  if (act == kActGeluErf) return gelu_erf(g);
  const float p = __builtin_elementwise_maximum(g, 0.0f);        // squared relu (fmaxf drops NaN)
  return p * p;
}

template <typename T, bool kVec, int kU>
__device__ __forceinline__ void act_values(const ActArgs& a, int64_t row, int cols, int col0, Who t,
                                           float (&v)[kU][8]) {
  const T* gate = reinterpret_cast<const T*>(a.gate) + row * a.gate_stride + col0;
  const T* p = reinterpret_cast<const T*>(a.up) + row * a.up_stride + col0;
  Raw8 raw_gate[kU], raw_up[kU];
  fetch<kVec, kU, true>(gate, cols, t, raw_gate, col0);
  if (a.up) fetch<kVec, kU, true>(p, cols, t, raw_up, col0);
  widen<kVec, kU>(gate, cols, t, raw_gate, v, col0);
  float up[kU][8];
  if (a.up) widen<kVec, kU>(p, cols, t, raw_up, up, col0);
#pragma unroll
  for (int k = 0; k < kU; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[k][j] = activate(a.act, v[k][j]);
      if (a.up) v[k][j] *= up[k][j];
    }
}

// A scale per row.
template <typename T, bool kVec, typename S>
__global__ __launch_bounds__(S::threads) void k_act_row(ActArgs a) {
  constexpr int kU = S::kU, kLanes = S::lanes;
  __shared__ SumMax red[kWaves];
  Who t;
  const int64_t row = row_of<S>(t);
  if (row >= a.rows) return;
  float v[kU][8];
  act_values<T, kVec, kU>(a, row, a.cols, 0, t, v);
  const float s = scale_of(a.elem, row_reduce<kLanes>(0.0f, amax_of(v), red).max);
  store_codes<kVec, kU>(reinterpret_cast<uint8_t*>(a.out) + row * a.cols, a.cols, t, a.elem, s, v);
  if (t.t == 0) a.scales[row] = s;
}

// Plain values or 1x128 blocks: a workgroup takes 256 units of one row, or several narrow rows
// by 2^shift threads each (327680 rows of 128, bf16 SwiGLU 44 us, 330 with a workgroup each).
template <typename T, bool kVec, bool kNarrow>
__global__ __launch_bounds__(256) void k_act_flat(ActArgs a, uint32_t pieces, int shift) {
  const Who t{kNarrow ? (int)threadIdx.x & ((1 << shift) - 1) : (int)threadIdx.x, 256};
  int64_t row = blockIdx.x / pieces;
  if constexpr (kNarrow) row = (row << (8 - shift)) + (threadIdx.x >> shift);
  if (kNarrow && row >= a.rows) return;
  const int col0 = (int)(blockIdx.x % pieces) * 2048, cols = min(a.cols - col0, 2048);
  float v[1][8];
  act_values<T, kVec, 1>(a, row, cols, col0, t, v);
  if (a.form == kFormPlain) {
    store_row<kVec, 1>(reinterpret_cast<T*>(a.out) + row * a.cols + col0, cols, t, v);
  } else if constexpr (kVec) {
    const float s = scale_of(a.elem, group_umax<16>(as_u(absmax8(v[0]))));
    const uint2 c = pack_codes(a.elem, v[0], s);
    if (8 * t.t < cols) {
      st_nt8(reinterpret_cast<uint8_t*>(a.out) + row * a.cols + col0 + 8 * t.t, c.x, c.y);
      if ((t.t & 15) == 0) a.scales[row * (a.cols / 128) + (col0 + 8 * t.t) / 128] = s;
    }
  }
}

// f(shape, grid, threads) for rows of `cols` elements.  Up to 512, or 1024 of many rows, fit a
// wave, narrow ones a part of it (327680 heads of 128 29 us with 16 lanes each, 87 with 64; of 64
// 16 with 8, 24 with 16); wider ones get as many waves as they need.  Threads without an element cost as much
// as others (16384 rows of 1024: 21 us with 64 threads a row, 30 with 256), and fewer units a
// thread shorten a few rows (64 of 4096, launches in a loop: 3.2 / 3.9 / 4.0 us at 1 / 2 / 4 units) and cost
// many little (8192 of 4096: 41.7 / 39.8 / 39.8).  Many wide rows of an activation are
// faster with four units (8192 of 14336 118 us, 136 with two; 512 11.8 and 10.3), of a norm,
// which holds more arrays, with two (4096 of 12288 59 us, 79 with four).
template <typename F>
void with_row_shape(int64_t rows, int cols, bool light, F f) {
  auto go = [&](auto shape) {
    using S = decltype(shape);
    const int threads = S::rows > 1 ? S::threads : (cols + 512 * S::kU - 1) / (512 * S::kU) * 64;
    f(shape, (uint32_t)((rows + S::rows - 1) / S::rows), threads);
  };
  if (cols <= 64) go(Shape<1, 8>{});
  else if (cols <= 128) go(Shape<1, 16>{});
  else if (cols <= 256) go(Shape<1, 32>{});
  else if (cols <= 512) go(Shape<1, 64>{});
  else if (cols <= 1024 && rows >= 4096) go(Shape<2, 64>{});
  else if (cols <= 4096) go(Shape<1, 512>{});
  else if (cols <= 8192) go(Shape<2, 512>{});
  else if (cols <= 16384 && !(light && rows >= 2048)) go(Shape<2, 1024>{});
  else go(Shape<4, 1024>{});
}

// f(T, whether 16-byte accesses fit).
template <typename F>
void with_type(bool bf16, bool vec, F f) {
  if (bf16 && vec) f((const uint16_t*)nullptr, std::true_type{});
  else if (bf16) f((const uint16_t*)nullptr, std::false_type{});
  else if (vec) f((const float*)nullptr, std::true_type{});
  else f((const float*)nullptr, std::false_type{});
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, bool bf16, bool vec, hipStream_t st) {
  with_type(bf16, vec, [&](auto type, auto v) {
    with_row_shape(a.rows, a.cols, false, [&](auto shape, uint32_t grid, int threads) {
      using T = std::remove_const_t<std::remove_pointer_t<decltype(type)>>;
      k_norm<T, decltype(v)::value, decltype(shape)><<<grid, threads, 0, st>>>(a);
    });
  });
  return hipGetLastError();
}

hipError_t launch_act(const ActArgs& a, bool bf16, bool vec, hipStream_t st) {
  with_type(bf16, vec, [&](auto type, auto v) {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(type)>>;
    constexpr bool kVec = decltype(v)::value;
    if (a.form == kFormRow) {
      with_row_shape(a.rows, a.cols, true, [&](auto shape, uint32_t grid, int threads) {
        k_act_row<T, kVec, decltype(shape)><<<grid, threads, 0, st>>>(a);
      });
    } else {
      const uint32_t pieces = (uint32_t)(a.cols + 2047) / 2048;
      int shift = 3;
      while (shift < 8 && 8 << shift < a.cols) ++shift;
      const uint32_t grid = (uint32_t)((a.rows + (256 >> shift) - 1) >> (8 - shift)) * pieces;
      if (shift < 8) k_act_flat<T, kVec, true><<<grid, 256, 0, st>>>(a, pieces, shift);
      else k_act_flat<T, kVec, false><<<grid, 256, 0, st>>>(a, pieces, shift);
    }
  });
  return hipGetLastError();
}

}  // namespace pqb
