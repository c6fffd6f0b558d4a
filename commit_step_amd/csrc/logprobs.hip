// dllm_token_logprobs and dllm_token_logprobs_grad: scores of given tokens.
//
// Forward, per scored position: one pass over V logits keeps, per wave, the
// running maximum M, z- and S of token_stats_dev.h (chunk_update), and the
// candidates for the K largest logits.  Then
//   log p_t = (x_t - M) / T - log1p(z-),   H = log1p(z-) - ln2 S / (1 + z-).
// Bound by reading the logits once from HBM: 1024 rows of 151936 bfloat16 with 5
// alternatives take 69.5 us (4.5 TB/s), 2048 of 126464 without any 108 us
// (4.8 TB/s); one row, split over 30 workgroups, 14 us with 20 alternatives.
//
// Backward, per scored position: p_v from the logits and the forward pass's
// (M, log z), one read and one write of the row; nothing is summed.  Rows that
// are not scored are written without being read.  4096 rows of 126464, half of
// them scored, take 316 us (4.9 TB/s, the rate of a large copy).
#include <string.h>

#include <algorithm>

#include "token_stats_dev.h"

namespace dllm {
namespace {

constexpr int kTopThreads = 256;
constexpr int kTopWaves = kTopThreads / 64;
constexpr int kMaxTopSlices = 64;
constexpr uint64_t kNoKey = ~0ull;

struct LogprobArgs {
  const void *logits;
  int64_t row_stride;
  int64_t V;
  int64_t slice_len;
  const int32_t *targets;
  int slices;
  int top;
  int n_suppress;
  float c;                 // log2 e / T
  float inv_t;             // 1 / T
  float *logprob;
  float *entropy;
  float *norm;
  int32_t *top_ids;
  float *top_logprobs;
  uint32_t *row_count;     // workspace: [rows] arrived slices
  uint64_t *parts;         // workspace: [rows][slices][2 + top]
  int32_t suppress[DLLM_MAX_SUPPRESS];   // sorted ascending
};

struct GradArgs {
  const void *logits;
  void *grad;
  int64_t row_stride, grad_stride;
  int64_t V;
  int64_t chunk;           // elements per workgroup
  int64_t chunks;          // workgroups per row
  const int32_t *targets;
  const float *norm, *entropy, *g_logprob, *g_entropy;
  float c, inv_t;
  int n_suppress;
  int32_t suppress[DLLM_MAX_SUPPRESS];
};

template <typename A>
__device__ __forceinline__ bool suppressed(const A &a, int64_t v) {
  for (int i = 0; i < a.n_suppress; ++i)
    if (a.suppress[i] == v) return true;
  return false;
}

// ---------------------------------------------------------------- the K largest
// Every wave collects candidates, elements that reach a bound below which the
// row's K largest cannot lie, unsorted in LDS; the few that are left at the end
// are ranked by counting.  The bound is the K-th largest of 64 groups' maxima
// (4 lanes each, over everything they have seen): K elements reach it.  It is
// taken in iterations 0, 1, 3 and 7 (one barrier each), so the candidates of a
// row are about K (2 + log2 of its iterations).  A sorted list per wave with
// one insertion after another measured 32 us for one token's 20 alternatives
// over 126464 ids, this 14 us; 8 us without alternatives.
//
// A candidate is a 64-bit key: the value's order-preserving bits, best first,
// then the id, so ascending keys are decreasing logits, equal ones by id.

constexpr int kCap = 256;            // candidates of a wave

__device__ __forceinline__ uint64_t top_key(float v, int id) {
  return ((uint64_t)conf_key(v) << 32) | (uint32_t)id;
}

// The K-th largest of the 64 groups' maxima (-inf when fewer groups hold
// anything).  Every thread calls it; gm is one of two buffers used in turn.
__device__ __forceinline__ float group_bound(float tmax, int K, float *gm) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float q = fmaxf(tmax, dpp_f<kQuadSwap1>(tmax, tmax));
  q = fmaxf(q, dpp_f<kQuadSwap2>(q, q));
  if ((lane & 3) == 0) gm[wave * 16 + (lane >> 2)] = q;
  __syncthreads();
  const float v = gm[lane];
  int above = 0;
#pragma unroll
  for (int j = 0; j < 64; j += 4) {
    const float4 o = *reinterpret_cast<const float4 *>(gm + j);
    above += (o.x > v) + (o.y > v) + (o.z > v) + (o.w > v);
  }
  // the smallest value with fewer than K above it
  return -wave_max(above < K ? -v : -kInf);
}

// A wave's candidates: n (wave-uniform) keys in buf, and the key that a new one
// has to stay below (kNoKey until a full buffer was cut to its K best).
struct Candidates {
  uint64_t *buf;
  int n;
  uint64_t kth;
};

// Cut the wave's buffer to its K smallest keys.
__device__ __forceinline__ void cut_to_best(Candidates &c, int K) {
  const int lane = threadIdx.x & 63;
  uint64_t k[kCap / 64];
#pragma unroll
  for (int j = 0; j < kCap / 64; ++j) k[j] = lane + 64 * j < c.n ? c.buf[lane + 64 * j] : kNoKey;
  uint64_t mine = kNoKey;
  for (int i = 0; i < K; ++i) {
    uint64_t m = k[0];
#pragma unroll
    for (int j = 1; j < kCap / 64; ++j) m = k[j] < m ? k[j] : m;
    const uint64_t best = wave_min_u64(m);
    if (lane == i) mine = best;
#pragma unroll
    for (int j = 0; j < kCap / 64; ++j) k[j] = k[j] == best ? kNoKey : k[j];
    c.kth = best;
  }
  // the reads above are complete in every lane: a wave's LDS operations are in order
  if (lane < K) c.buf[lane] = mine;
  c.n = K;
}

// Lanes with `pass` offer (v, id).
__device__ __forceinline__ void offer(Candidates &c, int K, bool pass, float v, int id) {
  const uint64_t key = top_key(v, id);
  uint64_t m = __builtin_amdgcn_ballot_w64(pass && key < c.kth);
  if (m == 0) return;
  if (c.n + __builtin_popcountll(m) > kCap) {
    cut_to_best(c, K);
    m = __builtin_amdgcn_ballot_w64(pass && key < c.kth);
  }
  const int lane = threadIdx.x & 63;
  const int at = c.n + __builtin_popcountll(m & ((1ull << lane) - 1ull));
  if ((m >> lane) & 1ull) c.buf[at] = key;
  c.n += __builtin_popcountll(m);
}

// The smallest value that is a candidate: the bound itself where elements equal
// to it count (a chunk that is part of the bound, or whose ids come before
// others'), else the next float (ids ascend from chunk to chunk, and K elements
// of lower id reach the bound); never -inf.
__device__ __forceinline__ float least_candidate(float bound, bool equal) {
  if (bound == -kInf) return -3.40282347e38f;
  if (equal) return bound;
  if (bound == 0.f) return 1.4e-45f;
  const uint32_t u = __float_as_uint(bound);
  return __uint_as_float(bound > 0.f ? u + 1u : u - 1u);      // above +inf: NaN, which nothing reaches
}

// One chunk of the sweep: every lane holds U loads of VEC elements, element j
// of load k at id idx_of(k, j); those of at least `least` are offered, the
// lanes' first ones together, then their second ones.
template <int U, int VEC, typename IdxF>
__device__ __forceinline__ void collect(Candidates &c, int K, const float (&x)[U * VEC], float least,
                                        IdxF idx_of) {
#pragma unroll
  for (int k = 0; k < U; ++k) {
    uint32_t bits = 0;
#pragma unroll
    for (int j = 0; j < VEC; ++j) bits |= x[k * VEC + j] >= least ? 1u << j : 0u;
    while (__builtin_amdgcn_ballot_w64(bits != 0) != 0) {
      const int j = bits ? __builtin_ctz(bits) : 0;
      float v = x[k * VEC];
#pragma unroll
      for (int e = 1; e < VEC; ++e) v = j == e ? x[k * VEC + e] : v;
      offer(c, K, bits != 0, v, idx_of(k, j));
      bits &= bits - 1u;
    }
  }
}

// The K smallest of the workgroup's keys, each thread holding N (kNoKey: none),
// in order into out[0 .. K-1] (kNoKey past the last): the K-th best group's
// value bounds them again, and what reaches it is ranked by counting.  Every
// thread calls it; cand has room for all keys.
template <int N>
__device__ __forceinline__ void select_keys(const uint64_t (&key)[N], int K, float *gm, uint64_t *cand,
                                            int *n_cand, uint64_t *out) {
  const int tid = threadIdx.x;
  float best = -kInf;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (key[i] != kNoKey) best = fmaxf(best, conf_from_key((uint32_t)(key[i] >> 32)));
  if (tid == 0) *n_cand = 0;
  if (tid < K) out[tid] = kNoKey;
  const float bound = group_bound(best, K, gm);
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (key[i] != kNoKey && conf_from_key((uint32_t)(key[i] >> 32)) >= bound)
      cand[atomicAdd(n_cand, 1)] = key[i];
  __syncthreads();
  const int m = *n_cand;
  for (int i = tid; i < m; i += kTopThreads) {
    const uint64_t k = cand[i];
    int rank = 0;
    for (int j = 0; j < m; ++j) rank += cand[j] < k;
    if (rank < K) out[rank] = k;
  }
  __syncthreads();
}

// ---------------------------------------------------------------- degenerate rows

struct RowSums {
  float M;     // largest logit, NaN as -inf
  float z, S;  // against M, without one maximal element (finite M)
  int n;       // M = +-inf: the ids the row is uniform over
};

// Two plain passes over a row that holds NaN or +inf, or no finite
// unsuppressed logit, or whose M log2 e overflows.  Valid in every thread.
template <typename T>
__device__ RowSums plain_row(const LogprobArgs &a, const T *row, float *fs, int *is) {
  const int tid = threadIdx.x;
  float m = -kInf;
  int n = 0, first = kIdxNone;
  for (int64_t v = tid; v < a.V; v += kTopThreads) {
    if (suppressed(a, v)) continue;
    const float x = ElemT<T>::load1(row + v);
    if (x == kInf) ++n;
    if (x > m) { m = x; first = (int)v; }
  }
  __syncthreads();
  fs[tid] = m;
  is[tid] = first;
  __syncthreads();
  for (int o = kTopThreads / 2; o > 0; o >>= 1) {
    if (tid < o && (fs[tid + o] > fs[tid] || (fs[tid + o] == fs[tid] && is[tid + o] < is[tid]))) {
      fs[tid] = fs[tid + o];
      is[tid] = is[tid + o];
    }
    __syncthreads();
  }
  RowSums r;
  r.M = fs[0];
  const int at = is[0];
  __syncthreads();
  is[tid] = n;
  float z = 0.f, S = 0.f;
  if (bits_finite(__float_as_uint(r.M))) {
    for (int64_t v = tid; v < a.V; v += kTopThreads) {
      if (v == at || suppressed(a, v)) continue;
      const float x = ElemT<T>::load1(row + v);
      if (!(x > -kInf)) continue;
      const float d = clamp_d((x - r.M) * a.c);
      const float t = __builtin_amdgcn_exp2f(d);
      z += t;
      S = fmaf(t, d, S);
    }
  }
  fs[tid] = z;
  __syncthreads();
  for (int o = kTopThreads / 2; o > 0; o >>= 1) {
    if (tid < o) { fs[tid] += fs[tid + o]; is[tid] += is[tid + o]; }
    __syncthreads();
  }
  r.z = fs[0];
  r.n = r.M == -kInf ? (int)a.V - a.n_suppress : is[0];
  __syncthreads();
  fs[tid] = S;
  __syncthreads();
  for (int o = kTopThreads / 2; o > 0; o >>= 1) {
    if (tid < o) fs[tid] += fs[tid + o];
    __syncthreads();
  }
  r.S = fs[0];
  __syncthreads();
  return r;
}

// ---------------------------------------------------------------- forward

template <typename T, bool TOP>
__global__ __launch_bounds__(kTopThreads, 4) void logprob_kernel(LogprobArgs a) {
  using E = ElemT<T>;
  constexpr int VEC = E::VEC, U = E::U, CH = U * VEC, STEP = kTopThreads * CH;
  constexpr int kKeys = kMaxTopSlices * DLLM_MAX_TOP;         // of a row's slices
  static_assert(kKeys >= kTopWaves * kCap, "room for every wave's candidates");
  __shared__ Partial wave_parts[kTopWaves];
  __shared__ uint64_t wave_cand[TOP ? kTopWaves : 1][kCap];
  __shared__ uint64_t cand[TOP ? kKeys : kTopThreads];
  __shared__ uint64_t best[DLLM_MAX_TOP];
  __shared__ __align__(16) float gm[2][64];
  __shared__ int s_ncand, s_last;
  __shared__ Partial s_part;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row_id = blockIdx.x / (uint32_t)a.slices;
  const int slice = (int)(blockIdx.x % (uint32_t)a.slices);
  const int K = a.top;

  const int64_t target = a.targets[row_id];
  if (target < 0 || target >= a.V) {
    if (slice == 0) {
      if (tid == 0) {
        a.logprob[row_id] = 0.f;
        a.entropy[row_id] = 0.f;
        if (a.norm) { a.norm[2 * row_id] = 0.f; a.norm[2 * row_id + 1] = 0.f; }
      }
      if (tid < K) {
        a.top_ids[row_id * K + tid] = -1;
        a.top_logprobs[row_id * K + tid] = -kInf;
      }
    }
    return;
  }
  const T *row = reinterpret_cast<const T *>(a.logits) + row_id * a.row_stride;
  const int64_t lo = (int64_t)slice * a.slice_len;
  const int64_t hi = min(lo + a.slice_len, a.V);

  WaveState st;
  st.c = a.c;
  st.M = -kInf; st.R = -kInf; st.idx = kIdxNone; st.zx = 0.f; st.Sx = 0.f; st.z = 0.f; st.S = 0.f;
  st.sb = -kInf; st.ib = kIdxNone; st.xb = -kInf; st.m2 = -kInf; st.m2x = -kInf;
  Candidates tc{TOP ? wave_cand[wave] : nullptr, 0, kNoKey};
  float tmax = -kInf, bound = -kInf;
  int sp = 0;

  // The slice's 16-byte-aligned body [blo, bhi); its head and tail, fewer than
  // VEC elements each, are one more chunk of wave 0.
  const uint32_t mis = (uint32_t)reinterpret_cast<uintptr_t>(row + lo) & 15u;
  const int64_t blo = min(lo + (int64_t)(((16u - mis) & 15u) / sizeof(T)), hi);
  const int64_t bhi = blo + (hi - blo) / VEC * VEC;

  // The next iteration's loads are in flight while one is reduced.  A lane past
  // the end reads the body's first word (in bounds, its value unused).
  const int n_it = (int)((bhi - blo + STEP - 1) / STEP);
  uint4 r[U], rn[U];
  auto load = [&](uint4 (&w)[U], int it) {
    const int64_t base = blo + (int64_t)it * STEP;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t v0 = base + (int64_t)(k * kTopThreads + tid) * VEC;
      w[k] = load_stream(reinterpret_cast<const uint4 *>(row + (v0 < bhi ? v0 : blo)));
    }
  };
  if (n_it > 0) load(rn, 0);
  for (int it = 0; it < n_it; ++it) {
    const int64_t base = blo + (int64_t)it * STEP;
#pragma unroll
    for (int k = 0; k < U; ++k) r[k] = rn[k];
    if (it + 1 < n_it) load(rn, it + 1);
    float x[CH];
    if (base + STEP <= bhi) {
#pragma unroll
      for (int k = 0; k < U; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[k * VEC + e] = E::at(r[k], e);
    } else {
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const bool ok = base + (int64_t)(k * kTopThreads + tid) * VEC < bhi;
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[k * VEC + e] = ok ? E::at(r[k], e) : -kInf;
      }
    }
    // suppressed ids of this iteration (rare, workgroup-uniform)
    while (sp < a.n_suppress && a.suppress[sp] < base) ++sp;
    for (int q = sp; q < a.n_suppress && a.suppress[q] < base + STEP; ++q) {
      const int off = (int)(a.suppress[q] - base);
      const int ks = off / (kTopThreads * VEC), rs = off - ks * (kTopThreads * VEC);
      const int owner = rs / VEC, es = rs - owner * VEC;
      if (tid == owner) {
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (k == ks && e == es) x[k * VEC + e] = -kInf;
      }
    }
    chunk_update<U, VEC, false, false>(st, x, [&](int k, int j, int ln) -> int {
      return (int)(base + (int64_t)(k * kTopThreads + wave * 64 + ln) * VEC + j);
    });
    if constexpr (TOP) {
      float cm = x[0];
#pragma unroll
      for (int e = 1; e < CH; ++e) cm = fmaxf(cm, x[e]);
      tmax = fmaxf(tmax, cm);
      const bool renew = it < 8 && (it & (it + 1)) == 0;
      if (renew) bound = group_bound(tmax, K, gm[__builtin_popcount(it) & 1]);
      const float least = least_candidate(bound, renew);
      if (__builtin_amdgcn_ballot_w64(cm >= least) != 0)
        collect<U, VEC>(tc, K, x, least, [&](int k, int j) -> int {
          return (int)(base + (int64_t)(k * kTopThreads + tid) * VEC + j);
        });
    }
  }
  const int nh = (int)(blo - lo), nq = (int)(hi - bhi);
  if (wave == 0 && nh + nq > 0) {
    float x1[1] = {-kInf};
    const int64_t v = lane < nh ? lo + lane : bhi + (lane - nh);
    if (lane < nh + nq && !suppressed(a, v)) x1[0] = E::load1(row + v);
    chunk_update<1, 1, true, false>(st, x1, [&](int, int, int ln) -> int {
      return (int)(ln < nh ? lo + ln : bhi + (ln - nh));
    });
    if constexpr (TOP)
      collect<1, 1>(tc, K, x1, least_candidate(bound, true), [&](int, int) -> int { return (int)v; });
  }

  // wave partials -> the workgroup's
  Partial p = empty_partial();
  p.M = st.M;
  p.idx = st.idx;
  p.z = wave_sum(st.z) + st.zx;
  p.S = wave_sum(st.S) + st.Sx;
  to_max_relative(st, p.z, p.S);
  if (lane == 0) wave_parts[wave] = p;
  __syncthreads();
  if (wave == 0) {
    const Partial q =
        butterfly_merge<false>(lane < kTopWaves ? wave_parts[lane] : empty_partial(), kTopWaves, a.c);
    if (lane == 0) s_part = q;
  }
  if constexpr (TOP) {
    uint64_t mine[kCap / 64];
#pragma unroll
    for (int j = 0; j < kCap / 64; ++j) mine[j] = lane + 64 * j < tc.n ? tc.buf[lane + 64 * j] : kNoKey;
    select_keys(mine, K, gm[0], cand, &s_ncand, best);
  } else {
    __syncthreads();
    if (K > 0 && tid == 0) best[0] = s_part.idx == kIdxNone ? kNoKey : top_key(s_part.M, s_part.idx);
    __syncthreads();
  }

  if (a.slices > 1) {
    // publish this slice; the row's last slice merges them in slice order
    const int words = 2 + K;
    uint64_t *mine = a.parts + ((int64_t)row_id * a.slices + slice) * words;
    if (tid == 0) {
      store_coherent(&mine[0], pack2(__float_as_uint(s_part.M), (uint32_t)s_part.idx));
      store_coherent(&mine[1], pack2(__float_as_uint(s_part.z), __float_as_uint(s_part.S)));
    }
    if (tid < K) store_coherent(&mine[2 + tid], best[tid]);
    wait_stores_complete();
    __syncthreads();
    if (tid == 0) {
      const uint32_t prev = atomicAdd(&a.row_count[row_id], 1u);
      s_last = prev == (uint32_t)(a.slices - 1);
    }
    __syncthreads();
    if (!s_last) return;
    uint64_t *all = a.parts + (int64_t)row_id * a.slices * words;
    if (wave == 0) {
      Partial q = empty_partial();
      if (lane < a.slices) {
        const uint64_t w0 = load_coh(&all[(int64_t)lane * words]);
        const uint64_t w1 = load_coh(&all[(int64_t)lane * words + 1]);
        q.M = __uint_as_float((uint32_t)w0);
        q.idx = (int)(uint32_t)(w0 >> 32);
        q.z = __uint_as_float((uint32_t)w1);
        q.S = __uint_as_float((uint32_t)(w1 >> 32));
      }
      q = butterfly_merge<false>(q, 64, a.c);
      if (lane == 0) s_part = q;
    }
    if constexpr (TOP) {
      constexpr int N = kKeys / kTopThreads;
      uint64_t mine[N];
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int i = tid + j * kTopThreads;
        mine[j] = i < a.slices * K ? load_coh(&all[(int64_t)(i / K) * words + 2 + i % K]) : kNoKey;
      }
      select_keys(mine, K, gm[1], cand, &s_ncand, best);
    } else {
      __syncthreads();
      if (K > 0 && tid == 0) best[0] = s_part.idx == kIdxNone ? kNoKey : top_key(s_part.M, s_part.idx);
      __syncthreads();
    }
    // leave the workspace zeroed
    for (int i = tid; i < a.slices * words; i += kTopThreads) all[i] = 0;
    if (tid == 0) a.row_count[row_id] = 0u;
  }

  float M = s_part.M, z = s_part.z, S = s_part.S;
  float logz, ent, each = 0.f;
  const bool fine = bits_finite(__float_as_uint(M)) && bits_finite(__float_as_uint(z)) &&
                    bits_finite(__float_as_uint(S));
  if (!fine) {
    const RowSums r = plain_row(a, row, reinterpret_cast<float *>(cand),
                                reinterpret_cast<int *>(cand) + kTopThreads);
    M = r.M; z = r.z; S = r.S;
    each = logf((float)r.n);
  }
  const bool finite = bits_finite(__float_as_uint(M));
  if (finite) {
    logz = log1p_nonneg(z);
    ent = logz - kLn2 * S / (1.0f + z);
  } else {
    logz = each;
    ent = each;
  }
  // log p of a logit of this row
  auto log_p = [&](float x) {
    if (!finite) return x == M || M == -kInf ? -each : -kInf;
    return (x - M) * a.inv_t - logz;
  };
  if (tid == 0) {
    float x = E::load1(row + target);
    if (x != x) x = -kInf;
    a.logprob[row_id] = suppressed(a, target) ? -kInf : log_p(x);
    a.entropy[row_id] = ent;
    if (a.norm) { a.norm[2 * row_id] = M; a.norm[2 * row_id + 1] = logz; }
    if (M == -kInf && K > 0) {
      // uniform: the lowest unsuppressed ids
      int id = 0, q = 0;
      for (int i = 0; i < K; ++i, ++id) {
        while (q < a.n_suppress && a.suppress[q] == id) { ++q; ++id; }
        a.top_ids[row_id * K + i] = id < a.V ? id : -1;
        a.top_logprobs[row_id * K + i] = id < a.V ? -each : -kInf;
      }
    }
  }
  if (tid < K && M != -kInf) {
    const uint64_t k = best[tid];
    float lp = -kInf;
    if (k != kNoKey) lp = log_p(conf_from_key((uint32_t)(k >> 32)));
    a.top_ids[row_id * K + tid] = lp > -kInf ? (int)(uint32_t)k : -1;
    a.top_logprobs[row_id * K + tid] = lp;
  }
}

// ---------------------------------------------------------------- backward

template <typename T> __device__ __forceinline__ T round_to(float x);
template <> __device__ __forceinline__ float round_to<float>(float x) { return x; }
template <> __device__ __forceinline__ uint16_t round_to<uint16_t>(float x) {
  return __builtin_bit_cast(uint16_t, (__bf16)x);      // to nearest, ties to even
}

template <typename T>
__global__ __launch_bounds__(256) void logprob_grad_kernel(GradArgs a) {
  using E = ElemT<T>;
  constexpr int VEC = E::VEC;
  const int64_t row_id = blockIdx.x / (uint32_t)a.chunks;
  const int64_t lo = (int64_t)(blockIdx.x % (uint32_t)a.chunks) * a.chunk;
  const int64_t hi = min(lo + a.chunk, a.V);
  const int tid = threadIdx.x;
  const T *row = reinterpret_cast<const T *>(a.logits) + row_id * a.row_stride;
  T *out = reinterpret_cast<T *>(a.grad) + row_id * a.grad_stride;
  const int64_t target = a.targets[row_id];
  const bool scored = target >= 0 && target < a.V;
  float g = 0.f, h = 0.f, M = 0.f, logz2 = 0.f, H = 0.f;
  if (scored) {
    if (a.g_logprob) g = a.g_logprob[row_id];
    if (a.g_entropy) h = a.g_entropy[row_id];
    M = a.norm[2 * row_id];
    logz2 = a.norm[2 * row_id + 1] * kLog2e;
    H = a.entropy[row_id];
  }
  const bool plain = a.n_suppress == 0;
  auto one = [&](float x, int64_t v) -> float {
    if (!plain && suppressed(a, v)) return 0.f;
    x = x != x ? -kInf : x;
    // log2 p; below -200 the probability is 0 in float32, and 0 * -inf never arises
    const float d = x == M ? 0.f : (x - M) * a.c;
    const float lp2 = fmaxf(d - logz2, -200.f);
    const float p = __builtin_amdgcn_exp2f(lp2);
    const float r = v == target ? g : 0.f;
    return (r - p * fmaf(h, fmaf(lp2, kLn2, H), g)) * a.inv_t;
  };
  const uint32_t mis = (uint32_t)reinterpret_cast<uintptr_t>(out + lo) & 15u;
  const bool same = !scored || ((uint32_t)reinterpret_cast<uintptr_t>(row + lo) & 15u) == mis;
  const int64_t blo = min(lo + (int64_t)(((16u - mis) & 15u) / sizeof(T)), hi);
  const int64_t bhi = same ? blo + (hi - blo) / VEC * VEC : blo;
  for (int64_t v0 = blo + tid * VEC; v0 < bhi; v0 += 256 * VEC) {
    uint4 o = make_uint4(0, 0, 0, 0);
    if (scored) {
      const uint4 r = load_stream(reinterpret_cast<const uint4 *>(row + v0));
      T y[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) y[e] = round_to<T>(one(E::at(r, e), v0 + e));
      o = __builtin_bit_cast(uint4, y);
    }
    *reinterpret_cast<uint4 *>(out + v0) = o;
  }
  // head and tail (the whole chunk where the two rows are aligned differently)
  const int64_t nh = blo - lo, n = nh + (hi - bhi);
  for (int64_t i = tid; i < n; i += 256) {
    const int64_t v = i < nh ? lo + i : bhi + (i - nh);
    out[v] = scored ? round_to<T>(one(E::load1(row + v), v)) : round_to<T>(0.f);
  }
}

// ---------------------------------------------------------------- host side

struct TopPlan { int slices; int64_t slice_len; };

// Fewer rows than CUs: split each into slices of at least 4096 elements.
TopPlan top_plan(int64_t rows, int64_t V) {
  const int cus = device_cu_count();
  int64_t s = 1;
  if (rows > 0 && rows < cus && V >= 8192) {
    s = std::min<int64_t>((cus + rows - 1) / rows, V / 4096);
    s = std::max<int64_t>(1, std::min<int64_t>(s, kMaxTopSlices));
  }
  int64_t len = (V + s - 1) / s;
  len = (len + 7) / 8 * 8;
  return {(int)((V + len - 1) / len), len};
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

size_t top_workspace(int64_t rows, int slices, int top) {
  if (slices <= 1) return 0;
  return align256((size_t)rows * 4) + (size_t)rows * slices * (2 + top) * 8;
}

// Checks common to both passes; fills the sorted suppress list.
int check_common(const char *who, const void *logits, int dtype, int64_t B, int64_t L, int64_t V,
                 int64_t row_stride, float temperature, const int32_t *suppress_ids,
                 int n_suppress, int32_t *sorted) {
  if (dtype != DLLM_F32 && dtype != DLLM_BF16)
    return fail(DLLM_ERR_DTYPE, "%s: dtype %d is neither DLLM_F32 nor DLLM_BF16", who, dtype);
  if (B < 0 || L < 0) return fail(DLLM_ERR_ARG, "%s: B and L must be >= 0", who);
  if (V < 1 || V > 0x7fffffffLL)
    return fail(DLLM_ERR_ARG, "%s: V = %lld must be in [1, 2^31)", who, (long long)V);
  if (row_stride < V) return fail(DLLM_ERR_ARG, "%s: row_stride < V", who);
  if (!(temperature >= 0x1p-126f) || temperature == __builtin_inff())
    return fail(DLLM_ERR_ARG, "%s: temperature must be finite and at least 2^-126", who);
  if (n_suppress < 0 || n_suppress > DLLM_MAX_SUPPRESS)
    return fail(DLLM_ERR_ARG, "%s: n_suppress must be in [0, %d]", who, DLLM_MAX_SUPPRESS);
  if (n_suppress > 0 && !suppress_ids)
    return fail(DLLM_ERR_ARG, "%s: suppress_ids is NULL", who);
  for (int i = 0; i < n_suppress; ++i) {
    const int32_t s = suppress_ids[i];
    if (s < 0 || s >= V)
      return fail(DLLM_ERR_ARG, "%s: suppress id %d is outside [0, V)", who, s);
    int j = i;
    while (j > 0 && sorted[j - 1] > s) { sorted[j] = sorted[j - 1]; --j; }
    sorted[j] = s;
  }
  for (int i = 1; i < n_suppress; ++i)
    if (sorted[i] == sorted[i - 1])
      return fail(DLLM_ERR_ARG, "%s: suppress id %d appears twice", who, sorted[i]);
  if (n_suppress >= V) return fail(DLLM_ERR_ARG, "%s: every id is suppressed", who);
  if (B > 0x7fffffffLL || L > 0x7fffffffLL || (L > 0 && B > (int64_t)(0xffffffffu / 1024u) / L))
    return fail(DLLM_ERR_UNSUPPORTED, "%s: more than %u positions", who, 0xffffffffu / 1024u);
  if (B > 0 && L > 0 && logits &&
      (uintptr_t)logits % (dtype == DLLM_BF16 ? 2 : 4) != 0)
    return fail(DLLM_ERR_ARG, "%s: logits are not aligned to their element", who);
  return DLLM_OK;
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" size_t dllm_token_logprobs_workspace_size(int dtype, int64_t B, int64_t L, int64_t V,
                                                     int top) {
  if ((dtype != DLLM_F32 && dtype != DLLM_BF16) || B < 0 || L < 0 || V < 1 || top < 0 ||
      top > DLLM_MAX_TOP || (L > 0 && B > (int64_t)(0xffffffffu / 1024u) / L))
    return 0;
  const TopPlan p = top_plan(B * L, V);
  return top_workspace(B * L, p.slices, top);
}

extern "C" int dllm_token_logprobs(const void *logits, int dtype, int64_t B, int64_t L, int64_t V,
                                   int64_t row_stride, float temperature,
                                   const int32_t *suppress_ids, int n_suppress,
                                   const int32_t *targets, int top, float *logprob, float *entropy,
                                   float *norm, int32_t *top_ids, float *top_logprobs,
                                   void *workspace, size_t workspace_bytes, hipStream_t stream) {
  const char *who = "dllm_token_logprobs";
  LogprobArgs a;
  memset(&a, 0, sizeof(a));
  const int rc = check_common(who, logits, dtype, B, L, V, row_stride, temperature, suppress_ids,
                              n_suppress, a.suppress);
  if (rc != DLLM_OK) return rc;
  if (top < 0 || top > DLLM_MAX_TOP)
    return fail(DLLM_ERR_ARG, "%s: top must be in [0, %d]", who, DLLM_MAX_TOP);
  if (B == 0 || L == 0) return ok();
  if (!logits || !targets || !logprob || !entropy)
    return fail(DLLM_ERR_ARG, "%s: logits, targets, logprob and entropy must be non-NULL", who);
  if (top > 0 && (!top_ids || !top_logprobs))
    return fail(DLLM_ERR_ARG, "%s: top_ids and top_logprobs must be non-NULL", who);
  const int64_t rows = B * L;
  const TopPlan p = top_plan(rows, V);
  const size_t need = top_workspace(rows, p.slices, top);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(DLLM_ERR_SHAPE, "%s: workspace has %zu bytes, needs %zu", who, workspace_bytes,
                need);
  if (need > 0 && (uintptr_t)workspace % 16 != 0)
    return fail(DLLM_ERR_ARG, "%s: workspace must be 16-byte aligned", who);
  a.logits = logits;
  a.row_stride = row_stride;
  a.V = V;
  a.slice_len = p.slice_len;
  a.targets = targets;
  a.slices = p.slices;
  a.top = top;
  a.n_suppress = n_suppress;
  a.c = (float)(1.4426950408889634 / (double)temperature);
  a.inv_t = (float)(1.0 / (double)temperature);
  a.logprob = logprob;
  a.entropy = entropy;
  a.norm = norm;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  if (need > 0) {
    a.row_count = reinterpret_cast<uint32_t *>(workspace);
    a.parts = reinterpret_cast<uint64_t *>(reinterpret_cast<char *>(workspace) +
                                           align256((size_t)rows * 4));
  }
  const dim3 grid((uint32_t)(rows * p.slices));
  // one alternative is the maximum that the statistics keep anyway
  const dim3 block(kTopThreads);
  if (dtype == DLLM_BF16) {
    if (top > 1) hipLaunchKernelGGL((logprob_kernel<uint16_t, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((logprob_kernel<uint16_t, false>), grid, block, 0, stream, a);
  } else {
    if (top > 1) hipLaunchKernelGGL((logprob_kernel<float, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((logprob_kernel<float, false>), grid, block, 0, stream, a);
  }
  return check_launch(who);
}

extern "C" int dllm_token_logprobs_grad(const void *logits, int dtype, int64_t B, int64_t L,
                                        int64_t V, int64_t row_stride, float temperature,
                                        const int32_t *suppress_ids, int n_suppress,
                                        const int32_t *targets, const float *norm,
                                        const float *entropy, const float *grad_logprob,
                                        const float *grad_entropy, void *grad,
                                        int64_t grad_stride, hipStream_t stream) {
  const char *who = "dllm_token_logprobs_grad";
  GradArgs a;
  memset(&a, 0, sizeof(a));
  const int rc = check_common(who, logits, dtype, B, L, V, row_stride, temperature, suppress_ids,
                              n_suppress, a.suppress);
  if (rc != DLLM_OK) return rc;
  if (grad_stride < V) return fail(DLLM_ERR_ARG, "%s: grad_stride < V", who);
  if (B == 0 || L == 0) return ok();
  if (!logits || !targets || !norm || !entropy || !grad)
    return fail(DLLM_ERR_ARG, "%s: logits, targets, norm, entropy and grad must be non-NULL", who);
  if ((uintptr_t)grad % (dtype == DLLM_BF16 ? 2 : 4) != 0)
    return fail(DLLM_ERR_ARG, "%s: grad is not aligned to its element", who);
  if (grad == logits && grad_stride != row_stride)
    return fail(DLLM_ERR_ARG, "%s: grad is the logits with another row stride", who);
  const int64_t rows = B * L;
  a.logits = logits;
  a.grad = grad;
  a.row_stride = row_stride;
  a.grad_stride = grad_stride;
  a.V = V;
  // 8 loads of 16 bytes per thread and workgroup
  a.chunk = 256 * 8 * (dtype == DLLM_BF16 ? 8 : 4);
  a.chunks = (V + a.chunk - 1) / a.chunk;
  if (rows * a.chunks > (int64_t)(0xffffffffu / 256u)) {
    // the grid's limit: longer chunks
    a.chunks = std::max<int64_t>(1, (int64_t)(0xffffffffu / 256u) / rows);
    a.chunk = ((V + a.chunks - 1) / a.chunks + 7) / 8 * 8;
    a.chunks = (V + a.chunk - 1) / a.chunk;
  }
  a.targets = targets;
  a.norm = norm;
  a.entropy = entropy;
  a.g_logprob = grad_logprob;
  a.g_entropy = grad_entropy;
  a.c = (float)(1.4426950408889634 / (double)temperature);
  a.inv_t = (float)(1.0 / (double)temperature);
  a.n_suppress = n_suppress;
  const dim3 grid((uint32_t)(rows * a.chunks));
  if (dtype == DLLM_BF16)
    hipLaunchKernelGGL(logprob_grad_kernel<uint16_t>, grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL(logprob_grad_kernel<float>, grid, dim3(256), 0, stream, a);
  return check_launch(who);
}
