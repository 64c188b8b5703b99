// Rotary positions: the pair (x0, x1) of values i of a head's first `rot` becomes
//   (x0 c - x1 s, x1 c + x0 s),   c, s = A cos, A sin of pos * angles[i],
// pairs being (i, i + rot / 2), or (2 i, 2 i + 1) when interleaved; the rest of the head is
// copied.  The angle of a far position loses its fraction of a turn in float32
// (at position 2^20 a whole 2^-4 radians), so it is formed in float64 as
// turns, less the nearest quarter turn; only the remainder, at most pi / 4, goes on
// in float32, to Taylor's polynomials of degree 9 and 10 (the next terms are below
// 2^-29 there).
//
// A workgroup takes one token, or up to four of small heads: its threads form each cosine and sine once, into
// LDS, and every head of q and k is then turned from there.  Reading and writing q and k
// is all that costs: bound by HBM, by latency for few tokens.
#include "launch.h"
#include "quant.h"

namespace pqb {
namespace {

constexpr int kThreads = 256, kTokens = 4;   // (tokens of a workgroup at most)

__device__ __forceinline__ float2 cos_sin(double turns, float amp) {
  turns -= __builtin_rint(turns);
  const double quarter = __builtin_rint(turns * 4.0);
  const float x = (float)((turns - quarter * 0.25) * 6.28318530717958647692);
  const float z = x * x;
  // sum (-1)^n x^(2n) / (2n)! and x^(2n + 1) / (2n + 1)!
  float c = -1.0f / 3628800.0f, s = 1.0f / 362880.0f;
  c = __builtin_fmaf(c, z, 1.0f / 40320.0f);
  s = __builtin_fmaf(s, z, -1.0f / 5040.0f);
  c = __builtin_fmaf(c, z, -1.0f / 720.0f);
  s = __builtin_fmaf(s, z, 1.0f / 120.0f);
  c = __builtin_fmaf(c, z, 1.0f / 24.0f);
  s = __builtin_fmaf(s, z, -1.0f / 6.0f);
  c = __builtin_fmaf(c, z, -0.5f);
  s = __builtin_fmaf(s * z, x, x);
  c = __builtin_fmaf(c, z, 1.0f);
  const int k = (int)quarter & 3;
  const float cc = (k & 1) ? s : c, ss = (k & 1) ? c : s;
  return make_float2(amp * ((k == 1 || k == 2) ? -cc : cc), amp * (k >= 2 ? -ss : ss));
}

// The position of token t, or false where no request owns it.
__device__ __forceinline__ bool position_of(const RopeArgs& a, int64_t t, int& pos) {
  if (a.positions) {
    pos = a.positions[t];
    return true;
  }
  if (t < a.starts[0] || t >= a.starts[a.batch]) return false;
  int64_t lo = 0, hi = a.batch;              // starts[lo] <= t < starts[hi]
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    (a.starts[mid] <= t ? lo : hi) = mid;
  }
  pos = a.kv_lens[lo] - a.starts[lo + 1] + (int)t;
  return true;
}

// kV values: 16 bytes (8 of bf16, 4 of float32), or fewer one by one.
template <int kV>
__device__ __forceinline__ void load_v(const uint16_t* p, float (&v)[kV]) {
  if constexpr (kV == 8) widen8(load_raw8(p), p, v);
  else for (int j = 0; j < kV; ++j) v[j] = ld1(p + j);
}
template <int kV>
__device__ __forceinline__ void load_v(const float* p, float (&v)[kV]) {
  if constexpr (kV == 4) {
    const uint4 w = ld_nt16(p);
    v[0] = as_f(w.x), v[1] = as_f(w.y), v[2] = as_f(w.z), v[3] = as_f(w.w);
  } else {
    for (int j = 0; j < kV; ++j) v[j] = ld1(p + j);
  }
}
template <int kV>
__device__ __forceinline__ void store_v(uint16_t* p, const float (&v)[kV]) {
  if constexpr (kV == 8)
    st_nt16(p, bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7]));
  else
    for (int j = 0; j < kV; ++j) p[j] = (uint16_t)(bf16x2_rne(v[j], 0.0f) & 0xFFFFu);
}
template <int kV>
__device__ __forceinline__ void store_v(float* p, const float (&v)[kV]) {
  if constexpr (kV == 4) st_nt16(p, as_u(v[0]), as_u(v[1]), as_u(v[2]), as_u(v[3]));
  else for (int j = 0; j < kV; ++j) p[j] = v[j];
}

// Parts of a head, one a thread: kV values of each half, kV / 2 pairs of an interleaved head, or
// kV values behind `rot`.  kV is 16 bytes' worth, or 1 (2 if interleaved) for any even
// dim, stride and address.
template <typename T, int kV, bool kInterleaved>
__global__ __launch_bounds__(kThreads) void k_rope(RopeArgs a, int tokens) {
  __shared__ float2 cs[kTokens * kRopeMaxRot / 2];
  __shared__ int owned[kTokens];
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  const int nt = (int)min((int64_t)tokens, a.tokens - t0);
  const int half = a.rot / 2;
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int t = i / half, p = i - t * half;
    int pos = 0;
    const bool own = position_of(a, t0 + t, pos);
    cs[i] = cos_sin((double)pos * (a.angles[p] * 0.15915494309189533577), a.amplitude);
    if (p == 0) owned[t] = own;
  }
  __syncthreads();

  const int turned = kInterleaved ? a.rot / kV : half / kV;
  const int parts = turned + (a.dim - a.rot) / kV, heads = a.heads[0] + a.heads[1];
  for (int i = threadIdx.x; i < nt * heads * parts; i += kThreads) {
    const int th = i / parts, p = i - th * parts, t = th / heads;
    int h = th - t * heads;
    if (!owned[t]) continue;
    const int which = h >= a.heads[0];
    h -= which ? a.heads[0] : 0;
    const T* x = reinterpret_cast<const T*>(a.x[which]) + (t0 + t) * a.stride[which] + (int64_t)h * a.dim;
    T* out = reinterpret_cast<T*>(a.out[which]) + (t0 + t) * a.out_stride[which] + (int64_t)h * a.dim;
    float u[kV], v[kV];
    if (p >= turned) {
      const int e = a.rot + (p - turned) * kV;
      load_v<kV>(x + e, u);
      store_v<kV>(out + e, u);
    } else if constexpr (kInterleaved) {
      load_v<kV>(x + p * kV, u);
#pragma unroll
      for (int j = 0; j < kV; j += 2) {
        const float2 w = cs[t * half + (p * kV + j) / 2];
        v[j] = __builtin_fmaf(u[j], w.x, -(u[j + 1] * w.y));
        v[j + 1] = __builtin_fmaf(u[j + 1], w.x, u[j] * w.y);
      }
      store_v<kV>(out + p * kV, v);
    } else {
      load_v<kV>(x + p * kV, u);
      load_v<kV>(x + half + p * kV, v);
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        const float2 w = cs[t * half + p * kV + j];
        const float x0 = u[j], x1 = v[j];
        u[j] = __builtin_fmaf(x0, w.x, -(x1 * w.y));
        v[j] = __builtin_fmaf(x1, w.x, x0 * w.y);
      }
      store_v<kV>(out + p * kV, u);
      store_v<kV>(out + half + p * kV, v);
    }
  }
}

template <typename T>
void launch(const RopeArgs& a, bool vec, hipStream_t st) {
  constexpr int kV = 16 / sizeof(T);
  // As many tokens as give each thread a part (8192 tokens of 32 + 8 heads of 128, bf16: 29.0,
  // 30.6 and 31.7 us with 1, 2 and 4; of 8 + 1 heads of 64: 8.6, 7.0 and 6.1)
  const int64_t parts = (int64_t)(a.heads[0] + a.heads[1]) * ((a.interleaved ? a.rot : a.rot / 2) + a.dim - a.rot) /
                        (vec ? kV : a.interleaved ? 2 : 1);
  const int tokens = parts >= kThreads ? 1 : parts >= kThreads / 2 ? 2 : kTokens;
  const uint32_t grid = (uint32_t)((a.tokens + tokens - 1) / tokens);
  if (a.interleaved) {
    if (vec) k_rope<T, kV, true><<<grid, kThreads, 0, st>>>(a, tokens);
    else k_rope<T, 2, true><<<grid, kThreads, 0, st>>>(a, tokens);
  } else {
    if (vec) k_rope<T, kV, false><<<grid, kThreads, 0, st>>>(a, tokens);
    else k_rope<T, 1, false><<<grid, kThreads, 0, st>>>(a, tokens);
  }
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, bool bf16, bool vec, hipStream_t st) {
  if (bf16) launch<uint16_t>(a, vec, st);
  else launch<float>(a, vec, st);
  return hipGetLastError();
}

}  // namespace pqb
