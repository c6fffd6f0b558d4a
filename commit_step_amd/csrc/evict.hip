// dllm_evict_select: the tokens of each cache that an eviction keeps.
//
// One workgroup per sequence, each wave a run of it.  The weights' order-
// preserving keys (best first, common.h; a protected token's key is 0, before
// every weight's) are read once, into registers up to 32768 tokens.  Three
// histograms of 11, 11 and 10 bits find the budget-th smallest key; then each
// wave counts and places its kept positions in order, with one prefix over the
// waves between.  One workgroup's instructions and latency bound it: 31 us for
// 32768 tokens, where sweeps that read the weights again each time took 59 us.
#include <algorithm>

#include "common.h"

namespace dllm {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;
constexpr int kSelList = 8192;           // keys of one first digit held in LDS

struct SelectArgs {
  const float *weights;
  int64_t weights_stride, T, budget, sink, recent, new_T;
  const int32_t *lens;
  int32_t *kept, *new_lens;
  float *new_weights;
};

// R keys per thread in registers (n <= R * 1024), or, with R = 0, read again in
// every sweep.
template <int R>
__global__ __launch_bounds__(kSelThreads) void evict_select_kernel(SelectArgs a) {
  __shared__ uint32_t hist[2048];
  __shared__ uint32_t list_key[kSelList];
  __shared__ uint8_t list_wave[kSelList];
  __shared__ uint32_t s_digit, s_below, s_count;
  __shared__ int s_listed;
  __shared__ int s_wave[kSelWaves], s_less[kSelWaves], s_same[kSelWaves];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t b = blockIdx.x;
  const float *w = a.weights + b * a.weights_stride;
  const int n = (int)(a.lens[b] < 0 ? 0 : min((int64_t)a.lens[b], a.T));
  const int keep = (int)min((int64_t)n, a.budget);
  int32_t *kept = a.kept + b * a.budget;
  float *nw = a.new_weights ? a.new_weights + b * a.new_T : nullptr;
  if (tid == 0) a.new_lens[b] = keep;
  for (int64_t j = keep + tid; j < a.budget; j += kSelThreads) kept[j] = -1;
  if (nw)
    for (int64_t j = keep + tid; j < a.new_T; j += kSelThreads) nw[j] = 0.f;
  if (n <= a.budget) {
    for (int j = tid; j < keep; j += kSelThreads) {
      kept[j] = j;
      if (nw) nw[j] = w[j];
    }
    return;
  }
  // this wave's tokens: 64 i + lane of [lo, hi)
  const int sink = (int)a.sink, tail = n - (int)a.recent;
  const int run = ((n + kSelWaves - 1) / kSelWaves + 63) / 64 * 64;
  const int lo = min(wave * run, n), hi = min(lo + run, n);
  auto key_at = [&](int t, float x) -> uint32_t { return t < sink || t >= tail ? 0u : conf_key(x); };
  uint32_t key[R > 0 ? R : 1];                // ~0 past the end: no weight's key
  if constexpr (R > 0) {
    float x[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {              // every load in flight before the first is used
      const int t = lo + 64 * i + lane;
      x[i] = w[t < hi ? t : 0];
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int t = lo + 64 * i + lane;
      key[i] = t < hi ? key_at(t, x[i]) : ~0u;
    }
  }
  // calls f(first token, key) for every 64 of the wave's tokens
  auto sweep = [&](auto f) {
    if constexpr (R > 0) {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (lo + 64 * i < hi) f(lo + 64 * i, key[i]);
    } else {
      for (int t0 = lo; t0 < hi; t0 += 64 * 8) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int t = t0 + 64 * i + lane;
          x[i] = w[t < hi ? t : 0];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int t = t0 + 64 * i + lane;
          if (t0 + 64 * i < hi) f(t0 + 64 * i, t < hi ? key_at(t, x[i]) : ~0u);
        }
      }
    }
  };

  // The keep-th smallest key, digit by digit from the top.  The keys of the
  // first digit's bin (some percent of them) go into a list, and the other two
  // digits and the waves' counts come from that; a bin that the list cannot
  // hold (many equal weights) is swept again instead.
  uint32_t prefix = 0, mask = 0;
  uint32_t want = (uint32_t)keep;             // still to find among keys matching prefix
  int listed = -1;                            // keys in the list, -1: none built
  int less = 0, same = 0;                     // of this wave: keys below, equal to the threshold
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t bits = pass == 2 ? 0x3ffu : 0x7ffu;
    for (int i = tid; i < 2048; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    if (listed >= 0) {
      for (int i = tid; i < listed; i += kSelThreads) {
        const uint32_t k = list_key[i];
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & bits], 1u);
      }
    } else {
      sweep([&](int, uint32_t k) {
        const bool in = k != ~0u && (k & mask) == prefix;
        const uint32_t bin = (k >> shift) & bits;
        // one count for a wave of one bin (equal weights would queue for it)
        const uint64_t m = __builtin_amdgcn_ballot_w64(in);
        if (m == 0) return;
        const int first = __builtin_amdgcn_readlane((int)bin, __builtin_ctzll(m));
        if (__builtin_amdgcn_ballot_w64(in && bin != (uint32_t)first) == 0) {
          if (lane == 0) atomicAdd(&hist[first], (uint32_t)__builtin_popcountll(m));
        } else if (in) {
          atomicAdd(&hist[bin], 1u);
        }
      });
    }
    __syncthreads();
    // inclusive prefix over the bins, two per thread; the digit's bin is the
    // first whose prefix reaches want
    const uint32_t h0 = hist[2 * tid], h1 = hist[2 * tid + 1];
    int sum = (int)(h0 + h1);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(sum, o);
      if (lane >= o) sum += u;
    }
    if (lane == 63) s_wave[wave] = sum;
    __syncthreads();
    int before = 0;
    for (int i = 0; i < wave; ++i) before += s_wave[i];
    const uint32_t incl = (uint32_t)(before + sum), excl = incl - h0 - h1;
    if (excl < want && want <= incl) {
      const bool first = want <= excl + h0;
      s_digit = (uint32_t)(2 * tid + (first ? 0 : 1));
      s_below = first ? excl : excl + h0;
      s_count = first ? h0 : h1;
      s_listed = 0;
    }
    __syncthreads();
    prefix |= s_digit << shift;
    mask |= bits << shift;
    want -= s_below;
    if (pass == 0 && s_count <= (uint32_t)kSelList) {
      const uint32_t digit = prefix >> 21;
      sweep([&](int, uint32_t k) {
        const bool in = k != ~0u && k >> 21 == digit;
        less += __builtin_popcountll(__builtin_amdgcn_ballot_w64(k >> 21 < digit));
        if (in) {
          const int at = atomicAdd(&s_listed, 1);
          list_key[at] = k;
          list_wave[at] = (uint8_t)wave;
        }
      });
      __syncthreads();
      listed = s_listed;
    }
    __syncthreads();
  }

  // keys below the threshold all stay, and the first `want` equal to it
  if (tid < kSelWaves) { s_less[tid] = 0; s_same[tid] = 0; }
  __syncthreads();
  if (listed >= 0) {
    for (int i = tid; i < listed; i += kSelThreads) {
      if (list_key[i] < prefix) atomicAdd(&s_less[list_wave[i]], 1);
      if (list_key[i] == prefix) atomicAdd(&s_same[list_wave[i]], 1);
    }
  } else {
    less = 0;
    sweep([&](int, uint32_t k) {
      less += __builtin_popcountll(__builtin_amdgcn_ballot_w64(k < prefix));
      same += __builtin_popcountll(__builtin_amdgcn_ballot_w64(k == prefix));
    });
  }
  if (lane == 0) { atomicAdd(&s_less[wave], less); atomicAdd(&s_same[wave], same); }
  __syncthreads();
  int at_less = 0, at_same = 0;
  for (int i = 0; i < wave; ++i) { at_less += s_less[i]; at_same += s_same[i]; }
  const uint64_t below = (1ull << lane) - 1ull;
  sweep([&](int t0, uint32_t k) {
    const int t = t0 + lane;
    const bool is_less = k < prefix, is_same = k == prefix;
    const uint64_t ml = __builtin_amdgcn_ballot_w64(is_less);
    const uint64_t ms = __builtin_amdgcn_ballot_w64(is_same);
    const int rl = at_less + __builtin_popcountll(ml & below);
    const int rs = at_same + __builtin_popcountll(ms & below);
    if (is_less || (is_same && rs < (int)want)) kept[rl + min(rs, (int)want)] = t;
    at_less += __builtin_popcountll(ml);
    at_same += __builtin_popcountll(ms);
  });
  if (nw) {
    // the kept tokens' weights, from the positions the workgroup has just stored
    // (a load beside each store above would wait for memory 64 tokens at a time)
    __syncthreads();
    for (int j0 = 0; j0 < keep; j0 += 8 * kSelThreads) {
      int t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = kept[min(j0 + i * kSelThreads + tid, keep - 1)];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = j0 + i * kSelThreads + tid;
        if (j < keep) nw[j] = w[t[i]];
      }
    }
  }
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" int dllm_evict_select(const float *weights, int64_t B, int64_t T,
                                 int64_t weights_stride, const int32_t *kv_lens, int64_t budget,
                                 int64_t sink, int64_t recent, int32_t *kept, int32_t *new_lens,
                                 float *new_weights, int64_t new_T, hipStream_t stream) {
  const char *who = "dllm_evict_select";
  if (B < 0 || T < 0 || T > 0x7fffffffLL - kSelThreads * 64)
    return fail(DLLM_ERR_ARG, "%s: B must be >= 0 and T in [0, 2^31 - 2^16)", who);
  if (budget < 1 || budget > 0x7fffffffLL)
    return fail(DLLM_ERR_ARG, "%s: budget must be in [1, 2^31)", who);
  if (sink < 0 || recent < 0 || sink > budget || recent > budget - sink)
    return fail(DLLM_ERR_ARG, "%s: sink and recent must be >= 0 and at most budget together", who);
  if (weights_stride < T) return fail(DLLM_ERR_ARG, "%s: weights_stride < T", who);
  if (new_weights && new_T < budget) return fail(DLLM_ERR_ARG, "%s: new_T < budget", who);
  if (B > 0xffffffffLL / kSelThreads)
    return fail(DLLM_ERR_UNSUPPORTED, "%s: too many sequences in one call", who);
  if (B == 0) return ok();
  if ((!weights && T > 0) || !kv_lens || !kept || !new_lens)
    return fail(DLLM_ERR_ARG, "%s: weights, kv_lens, kept and new_lens must be non-NULL", who);
  if (weights && (const void *)new_weights == (const void *)weights)
    return fail(DLLM_ERR_ARG, "%s: new_weights aliases weights", who);
  const SelectArgs a{weights, weights_stride, T, budget, sink, recent, new_T,
                     kv_lens, kept, new_lens, new_weights};
  const dim3 grid((uint32_t)B), block(kSelThreads);
  // keys per thread for the longest sequence there can be
  if (T <= 4 * kSelThreads) hipLaunchKernelGGL(evict_select_kernel<4>, grid, block, 0, stream, a);
  else if (T <= 32 * kSelThreads)
    hipLaunchKernelGGL(evict_select_kernel<32>, grid, block, 0, stream, a);
  else hipLaunchKernelGGL(evict_select_kernel<0>, grid, block, 0, stream, a);
  return check_launch(who);
}
