// Paged 8-bit KV cache: page planning and appends (layouts in paged.h).
//
// Plan.  Request b holds c_b tokens and gets n_b more; pages have ps tokens.
//   need_b = ceil((c_b + n_b) / ps) - ceil(c_b / ps),
//   S = exclusive sum of n, R = exclusive sum of need,
//   table[b, ceil(c_b / ps) + j] = free[used + R_b + j]          0 <= j < need_b,
//   slots[S_b + i] = table[b, (c_b + i) / ps] ps + (c_b + i) % ps   0 <= i < n_b.
// A few hundred bytes to a few hundred kilobytes move, so the time is launch and
// dependent-load latency: one workgroup takes both sums in one scan (a 64-bit
// word holds n below and need above) and fills the slots too, each thread finding
// its slot's request by bisection of S in LDS.  More than kPlanOneMax slots take a
// workgroup for each kPlanOneMax: every one repeats the sums rather than wait for
// them, and the first writes them.  That needs inputs that no output overlaps;
// a step in place, or more requests than LDS holds, fills its slots in a
// second launch.
// In a captured graph 64 requests' tokens take 5.5 us, where an empty launch takes
// 4; 777 requests with 49,000 slots 7.4 us, and 9.9 us with the second launch.
//
// Append.  One workgroup per run (consecutive slots inside one page), head and
// tensor.  The page's exponent is X = the smallest integer with
// max(amax, 1e-12) <= 448 2^X over the run, raised to the held exponent unless the
// run starts the page; codes are E4M3(x 2^-X), round to nearest even, and the
// product is exact (a power of two, far from float32's ends).  If X rose, the
// codes before the run are decoded, scaled and encoded again.  The input is
// read once (the first 64 tokens of a run stay in registers between the maximum
// and the codes) and V goes through LDS to be written along its tokens.
// Bound by HBM: prompts of 28,160 tokens (8 heads x 128, bf16) take 38 us, 4.6 TB/s
// of input and codes, where a copy reaches 5.1; with V turned a byte at a time they
// took 57.  64 single tokens take 5.9 us, 4 of them the launch.
#include <algorithm>

#include "../../include/pqb.h"
#include "launch.h"
#include "paged.h"

namespace pqb {
namespace {

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------

constexpr int kPlanThreads = 1024, kPlanWaves = kPlanThreads / kWave;
constexpr int64_t kPlanOneMax = 1024;  // slots that a planning workgroup fills
constexpr int kPlanOneBatch = 2048;    // requests whose sums it then keeps in LDS

__device__ __forceinline__ uint64_t wave_incl_sum(uint64_t v) {
  const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const uint64_t o = (uint64_t)__shfl_up((unsigned long long)v, d);
    if (lane >= d) v += o;
  }
  return v;
}

__device__ __forceinline__ int32_t pages_of(int32_t tokens, int shift) {
  return (int32_t)(((int64_t)tokens + (1 << shift) - 1) >> shift);
}

// The slot of new token t, of request b with first row s0, c cached tokens and
// first own free entry `base`; writes the table entry of a page that t starts.
__device__ __forceinline__ int32_t plan_slot(const PlanArgs& a, int64_t t, int64_t b, int32_t s0,
                                             int32_t c, int32_t base) {
  const int32_t pos = c + (int32_t)(t - s0), j = pos >> a.shift, held = pages_of(c, a.shift);
  int32_t* row = a.table + b * a.width;
  int32_t page;
  if (j < held) {
    page = row[j];
  } else {
    page = a.free_pages[base + (j - held)];
    if ((pos & ((1 << a.shift) - 1)) == 0) row[j] = page;
  }
  const int64_t slot = ((int64_t)page << a.shift) + (pos & ((1 << a.shift) - 1));
  return page < 0 || slot > INT32_MAX ? -1 : (int32_t)slot;
}

// The last b with S[b] <= t, for 0 <= t < S[n].
template <typename P>
__device__ __forceinline__ int64_t find_row(P S, int64_t n, int64_t t) {
  int64_t lo = 0, hi = n;
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (S[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

template <bool kFill>
__global__ __launch_bounds__(kPlanThreads) void k_plan(const PlanArgs a) {
  __shared__ int64_t part[kPlanWaves][2];
  __shared__ uint32_t flags;
  __shared__ uint64_t wsum[kPlanWaves];
  __shared__ int32_t first[kFill ? kPlanOneBatch + 1 : 1], held[kFill ? kPlanOneBatch : 1],
      base[kFill ? kPlanOneBatch : 1];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const bool writer = blockIdx.x == 0;
  if (tid == 0) flags = 0;
  __syncthreads();
  const int64_t used = *a.free_used, room = a.width << a.shift;
  int64_t tokens = 0, need = 0;
  uint32_t bad = (used < 0 || used > a.free_total) ? PQB_PLAN_NEGATIVE : 0u;
  for (int64_t b = tid; b < a.batch; b += kPlanThreads) {
    const int32_t c = a.cached[b], n = a.added[b];
    if (c < 0 || n < 0) {
      bad |= PQB_PLAN_NEGATIVE;
    } else {
      const int64_t end = (int64_t)c + n;
      if (end > room) bad |= PQB_PLAN_TABLE;
      tokens += n;
      need += ((end + (1 << a.shift) - 1) >> a.shift) - pages_of(c, a.shift);
    }
  }
#pragma unroll
  for (int d = kWave / 2; d; d >>= 1) {
    tokens += (int64_t)__shfl_xor((long long)tokens, d);
    need += (int64_t)__shfl_xor((long long)need, d);
  }
  if (bad) atomicOr(&flags, bad);
  if (lane == 0) {
    part[wave][0] = tokens;
    part[wave][1] = need;
  }
  __syncthreads();
  tokens = need = 0;
#pragma unroll
  for (int w = 0; w < kPlanWaves; ++w) {
    tokens += part[w][0];
    need += part[w][1];
  }
  bad = flags;
  if (tokens > a.max_new) bad |= PQB_PLAN_SLOTS;
  if (used >= 0 && need > a.free_total - used) bad |= PQB_PLAN_PAGES;
  if (tid == 0) {
    if (writer) {
      a.status[0] = (int32_t)bad;
      a.status[1] = (int32_t)min(need, (int64_t)INT32_MAX);
      a.status[2] = (int32_t)min(tokens, (int64_t)INT32_MAX);
      a.status[3] = 0;
      *a.free_used_out = (int32_t)(bad ? used : used + need);
      a.starts[a.batch] = bad ? 0 : (int32_t)tokens;
    }
    if constexpr (kFill) first[a.batch] = bad ? 0 : (int32_t)tokens;
  }
  uint64_t run = 0;  // sums of the chunks before this one: tokens below, pages above
  for (int64_t b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
    const int64_t b = b0 + tid;
    int32_t c = 0, n = 0;
    if (b < a.batch) {
      c = a.cached[b];
      n = bad ? 0 : a.added[b];
    }
    const uint32_t mine = bad ? 0u : (uint32_t)(pages_of(c + n, a.shift) - pages_of(c, a.shift));
    const uint64_t v = (uint64_t)(uint32_t)n | ((uint64_t)mine << 32);
    const uint64_t incl = wave_incl_sum(v);
    if (lane == kWave - 1) wsum[wave] = incl;
    __syncthreads();
    uint64_t before = run, all = 0;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
      if (w < wave) before += wsum[w];
      all += wsum[w];
    }
    run += all;
    if (b < a.batch) {
      const uint64_t ex = before + incl - v;
      const int32_t s0 = (int32_t)(uint32_t)ex, p0 = (int32_t)used + (int32_t)(ex >> 32);
      if (writer) {
        a.starts[b] = s0;
        a.kv_lens[b] = c + n;
      }
      if constexpr (kFill) {
        first[b] = s0;
        held[b] = c;
        base[b] = p0;
      } else {
        a.base[b] = p0;
      }
    }
    __syncthreads();
  }
  if constexpr (kFill) {
    const int64_t total = bad ? 0 : tokens;
    const int64_t t0 = (int64_t)blockIdx.x * kPlanOneMax, t1 = min(t0 + kPlanOneMax, a.max_new);
    for (int64_t t = t0 + tid; t < t1; t += kPlanThreads) {
      int32_t slot = -1;
      if (t < total) {
        const int64_t b = find_row(first, a.batch, t);
        slot = plan_slot(a, t, b, first[b], held[b], base[b]);
      }
      a.slots[t] = slot;
    }
  }
}

__global__ __launch_bounds__(kBlockThreads) void k_plan_slots(const PlanArgs a) {
  const int64_t t = (int64_t)blockIdx.x * kBlockThreads + threadIdx.x;
  if (t >= a.max_new) return;
  int32_t slot = -1;
  if (t < a.starts[a.batch]) {
    const int64_t b = find_row(a.starts, a.batch, t);
    const int32_t s0 = a.starts[b], n = a.starts[b + 1] - s0;
    slot = plan_slot(a, t, b, s0, a.kv_lens[b] - n, a.base[b]);
  }
  a.slots[t] = slot;
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------

constexpr int kAppThreads = 256;
constexpr int kAppRows = 64;  // tokens of a run taken at a time (V's LDS tile)

// The smallest X with max(amax, 1e-12) <= 448 2^X (448 = 1.75 2^8), from amax's bits.
__device__ __forceinline__ int page_exponent(uint32_t amax_bits) {
  const uint32_t b = max(amax_bits, kAmaxFloorBits) & 0x7FFFFFFFu;
  return (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
}

__device__ __forceinline__ float pow2(int e) { return as_f((uint32_t)(e + 127) << 23); }

// Four codes, each times f (a power of two <= 1), encoded again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  const f32x2 lo = e4m3x2_decode<false>(w), hi = e4m3x2_decode<true>(w);
  return e4m3_bytes4(lo[0] * f, lo[1] * f, hi[0] * f, hi[1] * f);
}

// Rows r0 .. r3 of four bytes -> columns c0 .. c3.
__device__ __forceinline__ void transpose4(const uint32_t r[4], uint32_t c[4]) {
  const uint32_t a = __builtin_amdgcn_perm(r[1], r[0], 0x05010400u), b = __builtin_amdgcn_perm(r[1], r[0], 0x07030602u);
  const uint32_t d = __builtin_amdgcn_perm(r[3], r[2], 0x05010400u), e = __builtin_amdgcn_perm(r[3], r[2], 0x07030602u);
  c[0] = __builtin_amdgcn_perm(d, a, 0x05040100u);
  c[1] = __builtin_amdgcn_perm(d, a, 0x07060302u);
  c[2] = __builtin_amdgcn_perm(e, b, 0x05040100u);
  c[3] = __builtin_amdgcn_perm(e, b, 0x07060302u);
}

// Eight values times inv, as codes.
template <typename T>
__device__ __forceinline__ uint2 codes8(const Raw8& raw, const T* tag, float inv) {
  float v[8];
  widen8(raw, tag, v);
  return make_uint2(e4m3_bytes4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    e4m3_bytes4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}

// One workgroup: a window of tokens, one head of K or V; every run that starts in
// the window, to its end.  Its loads come in two rounds, the slots of the window
// and of one page behind it, then the values and the held scale.
template <typename T, int kD>
__global__ __launch_bounds__(kAppThreads) void k_append(const AppendArgs a) {
  constexpr int kUnits = kD / 8;                             // 8-channel units of a token
  constexpr int kKeep = kAppRows * kUnits / kAppThreads;     // units a thread keeps
  constexpr int kLd = kD + 8;                                // LDS row: 8-byte steps, spread banks
  constexpr int kMaxPage = 256;
  __shared__ int run_at[kMaxPage], nruns;
  __shared__ int32_t slot[2 * kMaxPage + 1];                 // of tokens t0 - 1, t0, ...
  __shared__ uint32_t red[kAppThreads / kWave];
  __shared__ int red_n[kAppThreads / kWave], held_x;
  __shared__ __align__(16) uint8_t tile[kAppRows * kLd];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int head = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const int ps = 1 << a.shift;
  const int64_t t0 = (int64_t)blockIdx.x * a.window, nslots = (int64_t)a.pages << a.shift;
  const T* x = reinterpret_cast<const T*>(is_v ? a.v : a.k) + (int64_t)head * kD;
  const int64_t ld = is_v ? a.v_stride : a.k_stride;
  uint8_t* codes = is_v ? a.v_codes : a.k_codes;
  uint8_t* scales = is_v ? a.v_scales : a.k_scales;

  // a slot of -2 follows nothing and is followed by nothing
  for (int i = tid; i < a.window + ps + 1; i += kAppThreads) {
    const int64_t t = t0 - 1 + i;
    slot[i] = t >= 0 && t < a.tokens ? a.slots[t] : -2;
  }
  if (tid == 0) nruns = 0;
  __syncthreads();
  if (tid < a.window) {
    const int32_t s = slot[tid + 1];
    const bool starts = (s & (ps - 1)) == 0 || (int64_t)slot[tid] + 1 != s;
    if (s >= 0 && s < nslots && starts) run_at[atomicAdd(&nruns, 1)] = tid;
  }
  __syncthreads();
  const int runs = nruns;
  for (int r = 0; r < runs; ++r) {
    const int first = run_at[r];
    const int32_t s = slot[first + 1];
    const int64_t t = t0 + first;
    const int off = s & (ps - 1);
    // the run's length: the first i >= 1 whose slot does not follow
    const uint64_t m = __ballot(tid < ps - off && (int64_t)slot[first + 1 + tid] == (int64_t)s + tid);
    if (lane == 0) red_n[wave] = m == ~0ull ? kWave : __builtin_ctzll(~m);
    __syncthreads();
    int n = 0;
#pragma unroll
    for (int w = 0; w < kAppThreads / kWave; ++w) {
      n += red_n[w];
      if (red_n[w] < kWave) break;
    }
    const int64_t tile_id = (int64_t)(s >> a.shift) * a.heads + head;
    uint8_t* dst = codes + tile_id * ((int64_t)kD << a.shift);
    const T* src = x + t * ld;
    // tokens of the run up to the next multiple of kAppRows in the page are kept
    const int n0 = min(n, kAppRows - (off & (kAppRows - 1)));
    if (tid == 0) held_x = (int)scales[tile_id] - kE8m0Bias;
    Raw8 keep[kKeep];
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      const int u = tid + i * kAppThreads, row = u / kUnits, col = u % kUnits;
      keep[i] = Raw8{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
      if (row < n0) keep[i] = load_raw8(src + row * ld + col * 8);
    }
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      float v[8];
      widen8(keep[i], src, v);
      amax = max(amax, as_u(absmax8(v)));
    }
    for (int u = n0 * kUnits + tid; u < n * kUnits; u += kAppThreads) {
      float v[8];
      widen8(load_raw8(src + (u / kUnits) * ld + (u % kUnits) * 8), src, v);
      amax = max(amax, as_u(absmax8(v)));
    }
    amax = wave_umax(amax);
    if (lane == 0) red[wave] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAppThreads / kWave; ++w) amax = max(amax, red[w]);
    const int xold = held_x;
    int xp = page_exponent(amax);
    if (off) xp = max(xp, xold);
    const bool grown = off && xp > xold;
    const float f = pow2(max(xold - xp, -20));  // 448 2^-20 already rounds to 0
    const float inv = pow2(-max(min(xp, 126), -126));
    if (tid == 0) scales[tile_id] = (uint8_t)(xp + kE8m0Bias);

    if (!is_v) {
      if (grown)
        for (int i = tid; i < off * kD / 16; i += kAppThreads) {
          uint4* p = reinterpret_cast<uint4*>(dst) + i;
          const uint4 w = *p;
          *p = make_uint4(rescale4(w.x, f), rescale4(w.y, f), rescale4(w.z, f), rescale4(w.w, f));
        }
      uint2* out = reinterpret_cast<uint2*>(dst + (int64_t)off * kD);
#pragma unroll
      for (int i = 0; i < kKeep; ++i) {
        const int u = tid + i * kAppThreads;
        if (u / kUnits < n0) out[u] = codes8(keep[i], src, inv);
      }
      for (int u = n0 * kUnits + tid; u < n * kUnits; u += kAppThreads)
        out[u] = codes8(load_raw8(src + (u / kUnits) * ld + (u % kUnits) * 8), src, inv);
    } else {
      // kAppRows page offsets at a time: the run's codes into LDS by token, then
      // blocks of four tokens by four channels turned and written along the tokens.
      // A dword is written by one thread, which keeps the bytes of tokens outside
      // the run (held before it, rescaled if the exponent rose; untouched behind it).
      for (int c0 = grown ? 0 : off & -kAppRows; c0 < off + n; c0 += kAppRows) {
        const int lo = max(off, c0), hi = min(off + n, c0 + kAppRows);
        if (lo == off && hi > lo) {
#pragma unroll
          for (int i = 0; i < kKeep; ++i) {
            const int u = tid + i * kAppThreads, row = u / kUnits;
            if (row < hi - lo) *reinterpret_cast<uint2*>(tile + row * kLd + (u % kUnits) * 8) = codes8(keep[i], src, inv);
          }
        } else {
          for (int u = tid; u < (hi - lo) * kUnits; u += kAppThreads)
            *reinterpret_cast<uint2*>(tile + (u / kUnits) * kLd + (u % kUnits) * 8) =
                codes8(load_raw8(src + (int64_t)(lo - off + u / kUnits) * ld + (u % kUnits) * 8), src, inv);
        }
        __syncthreads();
        const int from = (grown ? c0 : lo) >> 2, groups = ((hi + 3) >> 2) - from;
        for (int i = tid; i < groups * (kD / 4); i += kAppThreads) {
          const int d = i / groups * 4, o = (from + i % groups) * 4;
          uint32_t* p = reinterpret_cast<uint32_t*>(dst + (d << a.shift) + o);
          uint32_t rows[4], cols[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            rows[k] = o + k >= lo && o + k < hi ? *reinterpret_cast<const uint32_t*>(tile + (o + k - lo) * kLd + d) : 0;
          transpose4(rows, cols);
          if (o < lo || o + 4 > hi) {
            // bytes of the run, and of what is held before it
            const int b0 = min(max(lo - o, 0), 4), b1 = min(max(hi - o, 0), 4);
            const uint32_t below = b0 == 4 ? ~0u : (1u << (8 * b0)) - 1;
            const uint32_t fresh = (b1 == 4 ? ~0u : (1u << (8 * b1)) - 1) & ~below;
            uint32_t was[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) was[k] = p[(k << a.shift) / 4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t held = grown ? (rescale4(was[k], f) & below) | (was[k] & ~below) : was[k];
              cols[k] = (cols[k] & fresh) | (held & ~fresh);
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) p[(k << a.shift) / 4] = cols[k];
        }
        __syncthreads();
      }
    }
    __syncthreads();  // red, red_n, held_x and the tile are free for the next run
  }
}

template <typename T>
void append_d(const AppendArgs& a, int head_dim, dim3 grid, hipStream_t st) {
  switch (head_dim) {
    case 64: hipLaunchKernelGGL((k_append<T, 64>), grid, dim3(kAppThreads), 0, st, a); break;
    case 128: hipLaunchKernelGGL((k_append<T, 128>), grid, dim3(kAppThreads), 0, st, a); break;
    case 192: hipLaunchKernelGGL((k_append<T, 192>), grid, dim3(kAppThreads), 0, st, a); break;
    default: hipLaunchKernelGGL((k_append<T, 256>), grid, dim3(kAppThreads), 0, st, a); break;
  }
}

// About this many workgroups before a window takes more than one token.
constexpr int64_t kAppendGroups = 4096;

}  // namespace

// Whether the second launch is what fills the slots.
static bool plan_two_launches(int64_t batch, int64_t max_new, bool in_place) {
  return batch > kPlanOneBatch || (in_place && max_new > kPlanOneMax);
}

size_t plan_workspace_bytes(int64_t batch, int64_t max_new) {
  return plan_two_launches(batch, max_new, true) ? 4 * (size_t)batch : 0;
}

hipError_t launch_plan(const PlanArgs& a, hipStream_t st) {
  const bool in_place = a.kv_lens == a.cached || a.free_used_out == a.free_used;
  if (!plan_two_launches(a.batch, a.max_new, in_place)) {
    const int64_t groups = std::max<int64_t>(1, (a.max_new + kPlanOneMax - 1) / kPlanOneMax);
    hipLaunchKernelGGL((k_plan<true>), dim3((unsigned)groups), dim3(kPlanThreads), 0, st, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((k_plan<false>), dim3(1), dim3(kPlanThreads), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.max_new == 0) return e;
  hipLaunchKernelGGL(k_plan_slots, dim3((unsigned)((a.max_new + kBlockThreads - 1) / kBlockThreads)),
                     dim3(kBlockThreads), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_append(AppendArgs a, bool bf16, int head_dim, hipStream_t st) {
  // A window is one workgroup's tokens.  Single tokens of many requests are a
  // run each and want a workgroup each; a prompt's run is a page, and windows of
  // one token would be almost all empty workgroups.
  a.window = 1;
  const int most = 1 << a.shift;
  while (a.window < most && (a.tokens + a.window - 1) / a.window * a.heads * 2 > kAppendGroups)
    a.window *= 2;
  const dim3 grid((unsigned)((a.tokens + a.window - 1) / a.window), (unsigned)(2 * a.heads));
  if (bf16)
    append_d<uint16_t>(a, head_dim, grid, st);
  else
    append_d<float>(a, head_dim, grid, st);
  return hipGetLastError();
}

}  // namespace pqb
