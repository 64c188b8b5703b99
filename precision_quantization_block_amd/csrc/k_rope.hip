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
// is all that costs: bound by HBM (8192 tokens of 40 heads of 128, bf16, 29 us, 5.8 TB/s), by
// latency for few tokens (64 3.6 us).
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

// kV consecutive values by one access of up to 16 bytes, aligned to its size; kOnce: with
// non-temporal hints, for heads that are whole 16-byte parts (where narrow parts share
// lines with others, the hints write lines twice: 20 of 128 turned, bf16, 69 us with them, 49
// without).
template <int kBytes>
struct Words {
  typedef uint32_t type __attribute__((ext_vector_type(kBytes / 4)));
};
template <>
struct Words<4> {
  typedef uint32_t type;
};
template <>
struct Words<2> {
  typedef uint16_t type;
};

template <bool kOnce, int kV, typename T>
__device__ __forceinline__ void load_v(const T* p, float (&v)[kV]) {
  using words = typename Words<kV * sizeof(T)>::type;
  if constexpr (kV == 1) {
    v[0] = ld1(p);
  } else {
    const words* q = reinterpret_cast<const words*>(p);
    const words w = kOnce ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      if constexpr (kV * sizeof(T) == 4) v[j] = as_f(j ? w & 0xFFFF0000u : w << 16);
      else if constexpr (sizeof(T) == 2) v[j] = as_f(j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
      else v[j] = as_f(w[j]);
    }
  }
}
template <bool kOnce, int kV, typename T>
__device__ __forceinline__ void store_v(T* p, const float (&v)[kV]) {
  using words = typename Words<kV * sizeof(T)>::type;
  if constexpr (kV == 1) {
    if constexpr (sizeof(T) == 2) *p = (uint16_t)(bf16x2_rne(v[0], 0.0f) & 0xFFFFu);
    else *p = v[0];
  } else {
    words w;
    if constexpr (kV * sizeof(T) == 4) w = bf16x2_rne(v[0], v[1]);
    else
#pragma unroll
      for (int j = 0; j < (int)(kV * sizeof(T) / 4); ++j) {
        if constexpr (sizeof(T) == 2) w[j] = bf16x2_rne(v[2 * j], v[2 * j + 1]);
        else w[j] = as_u(v[j]);
      }
    words* q = reinterpret_cast<words*>(p);
    if (kOnce) __builtin_nontemporal_store(w, q);
    else *q = w;
  }
}

// Parts of a head, one a thread: kV values of each half or kV / 2 pairs of an interleaved
// head; behind `rot`, which are copied, kV values up to `wide` and 16 bytes from there on.  kV
// is the most that rot, dim, strides and addresses allow.
template <typename T, int kV, bool kInterleaved>
__global__ __launch_bounds__(kThreads) void k_rope(RopeArgs a, int tokens, int wide) {
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

  // f(x, out, part, the token's cosines and sines) for each of `parts` parts of every head: the
  // parts of a kind together, so that a wave's threads do the same, and their places by
  // steps, not by a division each.
  const int heads = a.heads[0] + a.heads[1];
  auto each = [&](int parts, auto f) {
    if (parts == 0) return;
    int h = (int)threadIdx.x / parts, p = (int)threadIdx.x - h * parts, t = 0;
    const int step_h = kThreads / parts, step_p = kThreads - step_h * parts;
    for (;;) {
      while (h >= heads) h -= heads, ++t;
      if (t >= nt) return;
      if (owned[t]) {
        const int which = h >= a.heads[0], head = h - (which ? a.heads[0] : 0);
        f(reinterpret_cast<const T*>(a.x[which]) + (t0 + t) * a.stride[which] + (int64_t)head * a.dim,
          reinterpret_cast<T*>(a.out[which]) + (t0 + t) * a.out_stride[which] + (int64_t)head * a.dim, p, cs + t * half);
      }
      h += step_h;
      p += step_p;
      if (p >= parts) p -= parts, ++h;
    }
  };
  constexpr int kPairs = kInterleaved ? (kV > 1 ? kV / 2 : 1) : kV;   // of a turned part
  constexpr int kWide = 16 / sizeof(T);
  constexpr bool kOnce = kV == kWide;
  each(half / kPairs, [&](const T* x, T* out, int p, const float2* c) {
    c += kPairs * p;
    if constexpr (kInterleaved) {
      float y[2 * kPairs];
      x += 2 * kPairs * p;
      out += 2 * kPairs * p;
      if constexpr (kV > 1) load_v<kOnce, kV>(x, y);
      else y[0] = ld1(x), y[1] = ld1(x + 1);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        const float x0 = y[2 * j], x1 = y[2 * j + 1];
        y[2 * j] = __builtin_fmaf(x0, c[j].x, -(x1 * c[j].y));
        y[2 * j + 1] = __builtin_fmaf(x1, c[j].x, x0 * c[j].y);
      }
      if constexpr (kV > 1) {
        store_v<kOnce, kV>(out, y);
      } else {
        store_v<kOnce, 1>(out, {y[0]});
        store_v<kOnce, 1>(out + 1, {y[1]});
      }
    } else {
      float u[kV], v[kV];
      load_v<kOnce, kV>(x + p * kV, u);
      load_v<kOnce, kV>(x + half + p * kV, v);
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        const float x0 = u[j], x1 = v[j];
        u[j] = __builtin_fmaf(x0, c[j].x, -(x1 * c[j].y));
        v[j] = __builtin_fmaf(x1, c[j].x, x0 * c[j].y);
      }
      store_v<kOnce, kV>(out + p * kV, u);
      store_v<kOnce, kV>(out + half + p * kV, v);
    }
  });
  each((wide - a.rot) / kV, [&](const T* x, T* out, int p, const float2*) {
    float u[kV];
    load_v<kOnce, kV>(x + a.rot + p * kV, u);
    store_v<kOnce, kV>(out + a.rot + p * kV, u);
  });
  each((a.dim - wide) / kWide, [&](const T* x, T* out, int p, const float2*) {
    float u[kWide];
    load_v<kOnce, kWide>(x + wide + p * kWide, u);
    store_v<kOnce, kWide>(out + wide + p * kWide, u);
  });
}

template <typename T, int kV>
void launch(const RopeArgs& a, int wide, hipStream_t st) {
  // As many tokens as give each thread a part (8192 tokens of 32 + 8 heads of 128, bf16: 29.0,
  // 30.6 and 31.7 us with 1, 2 and 4; of 8 + 1 heads of 64: 8.6, 7.0 and 6.1)
  const int pairs = a.interleaved && kV > 1 ? kV / 2 : kV;
  const int64_t parts = (int64_t)(a.heads[0] + a.heads[1]) *
                        (a.rot / 2 / pairs + (wide - a.rot) / kV + (a.dim - wide) * (int)sizeof(T) / 16);
  const int tokens = parts >= kThreads ? 1 : parts >= kThreads / 2 ? 2 : kTokens;
  const uint32_t grid = (uint32_t)((a.tokens + tokens - 1) / tokens);
  if (a.interleaved) k_rope<T, kV, true><<<grid, kThreads, 0, st>>>(a, tokens, wide);
  else k_rope<T, kV, false><<<grid, kThreads, 0, st>>>(a, tokens, wide);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, bool bf16, int unit, bool aligned, hipStream_t st) {
  const int most = bf16 ? 8 : 4, wide = aligned ? (a.rot + most - 1) / most * most : a.dim;
  if (bf16) {
    if (unit >= 8) launch<uint16_t, 8>(a, wide, st);
    else if (unit == 4) launch<uint16_t, 4>(a, wide, st);
    else if (unit == 2) launch<uint16_t, 2>(a, wide, st);
    else launch<uint16_t, 1>(a, wide, st);
  } else {
    if (unit >= 4) launch<float, 4>(a, wide, st);
    else if (unit == 2) launch<float, 2>(a, wide, st);
    else launch<float, 1>(a, wide, st);
  }
  return hipGetLastError();
}

}  // namespace pqb
