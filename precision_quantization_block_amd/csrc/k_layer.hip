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
// A row stays in registers (kTpr threads, kU units of 8 elements each) from its
// one read to its one write; the row's sums and maxima meet by DPP, two shuffles and
// one LDS exchange.  All of it is bound by HBM, and by latency where there are few rows.
#include "launch.h"
#include "quant.h"

namespace pqb {
namespace {

// ---------------------------------------------------------------------------
// A row in registers.  kVec: unit k of thread t is elements 8 (k kTpr + t) ..., by
// 16-byte accesses.  Otherwise (odd widths, strides or addresses) element j of
// unit k is (8 k + j) kTpr + t, so that neighbours still share a line.
// ---------------------------------------------------------------------------
template <bool kVec, int kTpr>
__device__ __forceinline__ int elem_at(int k, int j, int t) {
  return kVec ? 8 * (k * kTpr + t) + j : (8 * k + j) * kTpr + t;
}

__device__ __forceinline__ Raw8 load_cached8(const uint16_t* p) {
  return Raw8{*reinterpret_cast<const uint4*>(p), make_uint4(0, 0, 0, 0)};
}
__device__ __forceinline__ Raw8 load_cached8(const float* p) {
  return Raw8{*reinterpret_cast<const uint4*>(p), *reinterpret_cast<const uint4*>(p + 4)};
}

// kOnce: read by this thread only (non-temporal); else shared with other rows.
template <bool kVec, int kTpr, int kU, bool kOnce, typename T>
__device__ __forceinline__ void load_row(const T* __restrict__ p, int cols, int t, float (&v)[kU][8]) {
  if constexpr (kVec) {
    Raw8 raw[kU];
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int e = elem_at<true, kTpr>(k, 0, t);
      raw[k] = e < cols ? (kOnce ? load_raw8(p + e) : load_cached8(p + e)) : Raw8{};
    }
#pragma unroll
    for (int k = 0; k < kU; ++k) widen8(raw[k], p, v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = elem_at<false, kTpr>(k, j, t);
        v[k][j] = e < cols ? ld1(p + e) : 0.0f;
      }
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

template <bool kVec, int kTpr, int kU, typename T>
__device__ __forceinline__ void store_row(T* __restrict__ p, int cols, int t, const float (&v)[kU][8]) {
#pragma unroll
  for (int k = 0; k < kU; ++k) {
    if constexpr (kVec) {
      const int e = elem_at<true, kTpr>(k, 0, t);
      if (e < cols) store8(p + e, v[k]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = elem_at<false, kTpr>(k, j, t);
        if (e < cols) store1(p + e, v[k][j]);
      }
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

template <bool kVec, int kTpr, int kU>
__device__ __forceinline__ void store_codes(uint8_t* __restrict__ p, int cols, int t, int elem, float s,
                                            const float (&v)[kU][8]) {
#pragma unroll
  for (int k = 0; k < kU; ++k) {
    const uint2 w = pack_codes(elem, v[k], s);
    if constexpr (kVec) {
      const int e = elem_at<true, kTpr>(k, 0, t);
      if (e < cols) st_nt8(p + e, w.x, w.y);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = elem_at<false, kTpr>(k, j, t);
        if (e < cols) p[e] = (uint8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Reductions over the kTpr threads of a row; every thread receives the result.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float wave_sum(float v) {
  v += as_f(dpp<kDppXor1>(as_u(v)));
  v += as_f(dpp<kDppXor2>(as_u(v)));
  v += as_f(dpp<kDppHalfMirror>(as_u(v)));
  v += as_f(dpp<kDppMirror>(as_u(v)));
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}

struct SumMax {
  float sum;
  uint32_t max;
};

// The sum and the largest bit pattern at once.  `red` (kTpr / 64 entries) is free to be
// written when the call starts; a second call takes another one.
template <int kTpr>
__device__ __forceinline__ SumMax row_reduce(float sum, uint32_t most, SumMax* red) {
  sum = wave_sum(sum);
  most = wave_umax(most);
  if constexpr (kTpr > kWave) {
    constexpr int kWaves = kTpr / kWave;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = SumMax{sum, most};
    __syncthreads();
    sum = 0.0f;
    most = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
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
template <bool kVec, int kTpr, int kU>
__device__ __forceinline__ float norm_stats(bool layer, float eps, int cols, int t, float (&v)[kU][8],
                                            SumMax* red) {
  if (layer) {
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[k][j];
    const float mean = row_reduce<kTpr>(s, 0, red).sum / (float)cols;
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[k][j] = elem_at<kVec, kTpr>(k, j, t) < cols ? v[k][j] - mean : 0.0f;
  }
  float q = 0.0f;
#pragma unroll
  for (int k = 0; k < kU; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) q = __builtin_fmaf(v[k][j], v[k][j], q);
  const float ms = row_reduce<kTpr>(q, 0, red + kTpr / kWave).sum / (float)cols;
  return 1.0f / sqrtf(ms + eps);
}

constexpr int block_of(int tpr) { return tpr < 256 ? 256 : tpr; }

template <typename T, bool kVec, int kTpr, int kU>
__global__ __launch_bounds__(block_of(kTpr)) void k_norm(NormArgs a) {
  constexpr int kRows = block_of(kTpr) / kTpr, kRed = kTpr / kWave;
  __shared__ SumMax red[5 * kRed];
  const int t = threadIdx.x % kTpr;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kTpr;
  if (kRows > 1 && row >= a.rows) return;   // whole waves; no barrier with several rows

  float v[kU][8];
  load_row<kVec, kTpr, kU, true>(reinterpret_cast<const T*>(a.x) + row * a.x_stride, a.cols, t, v);
  const bool layer = a.layer;
  if (a.post) {
    const float r = norm_stats<kVec, kTpr, kU>(layer, a.eps, a.cols, t, v, red + 3 * kRed);
    float w[kU][8];
    load_row<kVec, kTpr, kU, false>(reinterpret_cast<const T*>(a.post), a.cols, t, w);
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] = v[k][j] * r * w[k][j];
  }
  if (a.gate) {
    float g[kU][8];
    load_row<kVec, kTpr, kU, false>(
        reinterpret_cast<const T*>(a.gate) + (int64_t)((uint32_t)row / a.per_gate) * a.gate_stride, a.cols, t, g);
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] *= g[k][j];
  }
  if (a.residual) {
    float g[kU][8];
    load_row<kVec, kTpr, kU, true>(reinterpret_cast<const T*>(a.residual) + row * a.res_stride, a.cols, t, g);
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] += g[k][j] * a.res_scale;
  }
  if (a.h) {
    T* h = reinterpret_cast<T*>(a.h) + row * a.h_stride;
    store_row<kVec, kTpr, kU>(h, a.cols, t, v);
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] = rounded(h, v[k][j]);
  }

  // u, and r where it is not in u
  float w[kU][8];
  if (a.weight) {
    load_row<kVec, kTpr, kU, false>(reinterpret_cast<const T*>(a.weight), a.cols, t, w);
  } else {
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) w[k][j] = 1.0f;
  }
  float r = 1.0f;
  uint32_t most = 0;
  if (layer) {
    const float rl = norm_stats<kVec, kTpr, kU>(true, a.eps, a.cols, t, v, red);
    float b[kU][8] = {};
    if (a.bias) load_row<kVec, kTpr, kU, false>(reinterpret_cast<const T*>(a.bias), a.cols, t, b);
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] = v[k][j] * rl * w[k][j] + b[k][j];
    if (a.form == kFormRow) most = row_reduce<kTpr>(0.0f, amax_of(v), red + 2 * kRed).max;
  } else {
    float q = 0.0f;
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        q = __builtin_fmaf(v[k][j], v[k][j], q);
        v[k][j] *= w[k][j];
      }
    const SumMax m = row_reduce<kTpr>(q, amax_of(v), red);
    r = 1.0f / sqrtf(m.sum / (float)a.cols + a.eps);
    most = m.max;
  }

  if (a.form == kFormPlain) {
#pragma unroll
    for (int k = 0; k < kU; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] *= r;
    store_row<kVec, kTpr, kU>(reinterpret_cast<T*>(a.out) + row * a.cols, a.cols, t, v);
  } else if (a.form == kFormRow) {
    const float s = scale_of(a.elem, most);
    store_codes<kVec, kTpr, kU>(reinterpret_cast<uint8_t*>(a.out) + row * a.cols, a.cols, t, a.elem, s, v);
    if (t == 0) a.scales[row] = s * r;
  } else if constexpr (kVec) {   // 1x128 blocks: 16 threads each (cols % 128 == 0)
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int e = elem_at<true, kTpr>(k, 0, t);
      const float s = scale_of(a.elem, group_umax<16>(as_u(absmax8(v[k]))));
      const uint2 c = pack_codes(a.elem, v[k], s);
      if (e < a.cols) {
        st_nt8(reinterpret_cast<uint8_t*>(a.out) + row * a.cols + e, c.x, c.y);
        if ((t & 15) == 0) a.scales[row * (a.cols / 128) + e / 128] = s * r;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Activations.  Each takes a few float32 roundings (silu and tanh-gelu as
// g / (1 + 2^-z): the product with log2(e) carries its rounding error along, since 2^z
// turns an absolute error into a relative one).
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
  const float c = __builtin_fmaf(__builtin_fmaf(-q, d, g), y, q);
  return d < 0x1p126f ? c : 0.0f * g;                            // exp(-z) overflows: -0 for finite g
}

__device__ __forceinline__ float activate(int act, float g) {
  if (act == kActSilu) return sigmoid_times(g, g);
  if (act == kActGeluTanh) {
    // (1 + tanh(z)) / 2 = 1 / (1 + exp(-2 z)), z = sqrt(2 / pi) (g + 0.044715 g^3)
    const float g2 = __builtin_fminf(g * g, 1e10f);
    return sigmoid_times(g, 1.59576912160573072f * __builtin_fmaf(0.044715f * g2, g, g));
  }
  if (act == kActGeluErf) return 0.5f * g * erfcf(-0.707106781186547524f * g);
  const float p = __builtin_fmaxf(g, 0.0f);                      // squared relu
  return p * p;
}

template <typename T, bool kVec, int kTpr, int kU>
__device__ __forceinline__ void act_values(const ActArgs& a, int64_t row, int cols, int col0, int t,
                                           float (&v)[kU][8]) {
  float up[kU][8];
  load_row<kVec, kTpr, kU, true>(reinterpret_cast<const T*>(a.gate) + row * a.gate_stride + col0, cols, t, v);
  if (a.up)
    load_row<kVec, kTpr, kU, true>(reinterpret_cast<const T*>(a.up) + row * a.up_stride + col0, cols, t, up);
#pragma unroll
  for (int k = 0; k < kU; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[k][j] = activate(a.act, v[k][j]);
      if (a.up) v[k][j] *= up[k][j];
    }
}

// A scale per row.
template <typename T, bool kVec, int kTpr, int kU>
__global__ __launch_bounds__(block_of(kTpr)) void k_act_row(ActArgs a) {
  constexpr int kRows = block_of(kTpr) / kTpr;
  __shared__ SumMax red[kTpr / kWave];
  const int t = threadIdx.x % kTpr;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kTpr;
  if (kRows > 1 && row >= a.rows) return;
  float v[kU][8];
  act_values<T, kVec, kTpr, kU>(a, row, a.cols, 0, t, v);
  const float s = scale_of(a.elem, row_reduce<kTpr>(0.0f, amax_of(v), red).max);
  store_codes<kVec, kTpr, kU>(reinterpret_cast<uint8_t*>(a.out) + row * a.cols, a.cols, t, a.elem, s, v);
  if (t == 0) a.scales[row] = s;
}

// Plain values or 1x128 blocks: a workgroup takes 256 units of one row.
template <typename T, bool kVec>
__global__ __launch_bounds__(256) void k_act_flat(ActArgs a, uint32_t pieces) {
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x / pieces;
  const int col0 = (int)(blockIdx.x % pieces) * 2048, cols = min(a.cols - col0, 2048);
  float v[1][8];
  act_values<T, kVec, 256, 1>(a, row, cols, col0, t, v);
  if (a.form == kFormPlain) {
    store_row<kVec, 256, 1>(reinterpret_cast<T*>(a.out) + row * a.cols + col0, cols, t, v);
  } else if constexpr (kVec) {
    const float s = scale_of(a.elem, group_umax<16>(as_u(absmax8(v[0]))));
    const uint2 c = pack_codes(a.elem, v[0], s);
    if (8 * t < cols) {
      st_nt8(reinterpret_cast<uint8_t*>(a.out) + row * a.cols + col0 + 8 * t, c.x, c.y);
      if ((t & 15) == 0) a.scales[row * (a.cols / 128) + (col0 + 8 * t) / 128] = s;
    }
  }
}

// f(threads per row, units per thread) for the smallest row shape that holds `cols`.
template <typename F>
void with_row_shape(int cols, F f) {
  if (cols <= 512) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  else if (cols <= 1024) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
  else if (cols <= 2048) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
  else if (cols <= 4096) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  else if (cols <= 8192) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
  else if (cols <= 16384) f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
  else f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 4>{});
}

// f(T, whether 16-byte accesses fit).
template <typename F>
void with_type(bool bf16, bool vec, F f) {
  if (bf16 && vec) f((const uint16_t*)nullptr, std::true_type{});
  else if (bf16) f((const uint16_t*)nullptr, std::false_type{});
  else if (vec) f((const float*)nullptr, std::true_type{});
  else f((const float*)nullptr, std::false_type{});
}

template <typename K>
uint32_t row_grid(int64_t rows, K tpr) {
  constexpr int kRows = block_of(K::value) / K::value;
  return (uint32_t)((rows + kRows - 1) / kRows);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, bool bf16, bool vec, hipStream_t st) {
  with_type(bf16, vec, [&](auto type, auto v) {
    with_row_shape(a.cols, [&](auto tpr, auto units) {
      using T = std::remove_const_t<std::remove_pointer_t<decltype(type)>>;
      k_norm<T, decltype(v)::value, decltype(tpr)::value, decltype(units)::value>
          <<<row_grid(a.rows, tpr), block_of(tpr), 0, st>>>(a);
    });
  });
  return hipGetLastError();
}

hipError_t launch_act(const ActArgs& a, bool bf16, bool vec, hipStream_t st) {
  with_type(bf16, vec, [&](auto type, auto v) {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(type)>>;
    constexpr bool kVec = decltype(v)::value;
    if (a.form == kFormRow) {
      with_row_shape(a.cols, [&](auto tpr, auto units) {
        k_act_row<T, kVec, decltype(tpr)::value, decltype(units)::value>
            <<<row_grid(a.rows, tpr), block_of(tpr), 0, st>>>(a);
      });
    } else {
      const uint32_t pieces = (uint32_t)(a.cols + 2047) / 2048;
      k_act_flat<T, kVec><<<(uint32_t)a.rows * pieces, 256, 0, st>>>(a, pieces);
    }
  });
  return hipGetLastError();
}

}  // namespace pqb
