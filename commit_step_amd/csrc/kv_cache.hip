// dllm_kv_write, dllm_kv_read, dllm_kv_gather: the 8-bit key/value cache.
//
// All three move data: one workgroup per page and head, 16-byte loads and
// stores, the transposition between tokens-by-channels and the values' layout
// through LDS.  Bound by HBM bandwidth (a write reads 4 D bytes per token and
// head and stores 2 D; a read the reverse) and, for a few tokens, by the launch
// and two dependent fetches.  Measured at 32000 tokens of 8 heads of 128
// channels: a write 49 us (4.0 TB/s: two sweeps over a page in LDS between load
// and store, the second after the page's maximum is known), a read 31 us
// (6.4 TB/s); 8 tokens of 4 heads: 5.4 and 3.8 us.
#include <string.h>

#include <algorithm>

#include "kv_dev.h"

namespace dllm {
namespace {

constexpr int kKvThreads = 256;

struct CacheArgs {
  uint8_t *k, *v;
  float *k_scale, *v_scale;
  int64_t num_pages;
  int H;
};

struct WriteArgs {
  CacheArgs c;
  const uint16_t *k, *v;               // bf16 bits
  int64_t ks[3], vs[3];                // element strides (B, L, head)
  int64_t L, max_pages, table_stride;
  int64_t touched;                     // pages per sequence in the grid
  const int32_t *table, *start, *lens;
  int vec;                             // rows are 16-byte aligned
};

// Largest value over the workgroup (>= 0); `red` holds one float per wave.
__device__ __forceinline__ float group_max(float v, float *red) {
  const float w = wave_max(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = w;
  __syncthreads();
  float m = red[0];
#pragma unroll
  for (int i = 1; i < kKvThreads / 64; ++i) m = fmaxf(m, red[i]);
  return m;
}

// NaN to 0 and |x| for the page's maximum (infinities do not count).
__device__ __forceinline__ uint16_t clean(uint16_t b, float &amax) {
  const uint32_t mag = b & 0x7fffu;
  if (mag > 0x7f80u) return 0;
  if (mag < 0x7f80u) amax = fmaxf(amax, __uint_as_float(mag << 16));
  return b;
}

template <int D>
__global__ __launch_bounds__(kKvThreads) void kv_write_kernel(WriteArgs a) {
  constexpr int ROW = D + 8;                       // LDS row, off the bank period
  __shared__ __align__(16) uint16_t kt[kPage * ROW], vt[kPage * ROW];
  __shared__ float red[kKvThreads / 64];
  const int tid = threadIdx.x;
  const uint32_t unit = blockIdx.x / (uint32_t)a.c.H;
  const int h = (int)(blockIdx.x - unit * (uint32_t)a.c.H);
  const int64_t b = unit / (uint32_t)a.touched;
  const int64_t j = unit - (uint32_t)b * (uint32_t)a.touched;
  const int64_t s0 = a.start[b];
  const int64_t n = a.lens ? min((int64_t)a.lens[b], a.L) : a.L;
  if (s0 < 0 || n <= 0) return;
  const int64_t p = s0 / kPage + j;
  if (p >= a.max_pages || p * kPage >= s0 + n) return;
  const int64_t page = page_of(a.table + b * a.table_stride, p, a.c.num_pages);
  if (page < 0) return;
  const int lo = (int)max((int64_t)0, s0 - p * kPage);         // new tokens: slots [lo, hi)
  const int hi = (int)min((int64_t)kPage, s0 + n - p * kPage);
  const int64_t l0 = p * kPage - s0;                           // token of slot 0

  float ka = 0.f, va = 0.f;
  const uint16_t *kp = a.k + b * a.ks[0] + h * a.ks[2];
  const uint16_t *vp = a.v + b * a.vs[0] + h * a.vs[2];
  if (a.vec) {
    constexpr int PER = D / 8;                                 // 16-byte pieces per token
    for (int i = tid; i < kPage * PER; i += kKvThreads) {
      const int t = i / PER, d = i % PER * 8;
      if (t < lo || t >= hi) continue;
      u32x4 kw = *reinterpret_cast<const u32x4 *>(kp + (l0 + t) * a.ks[1] + d);
      u32x4 vw = *reinterpret_cast<const u32x4 *>(vp + (l0 + t) * a.vs[1] + d);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        kw[q] = (uint32_t)clean((uint16_t)kw[q], ka) | (uint32_t)clean((uint16_t)(kw[q] >> 16), ka) << 16;
        vw[q] = (uint32_t)clean((uint16_t)vw[q], va) | (uint32_t)clean((uint16_t)(vw[q] >> 16), va) << 16;
      }
      *reinterpret_cast<u32x4 *>(&kt[t * ROW + d]) = kw;
      *reinterpret_cast<u32x4 *>(&vt[t * ROW + d]) = vw;
    }
  } else {
    for (int i = tid; i < kPage * D; i += kKvThreads) {
      const int t = i / D, d = i % D;
      if (t < lo || t >= hi) continue;
      kt[t * ROW + d] = clean(kp[(l0 + t) * a.ks[1] + d], ka);
      vt[t * ROW + d] = clean(vp[(l0 + t) * a.vs[1] + d], va);
    }
  }
  const int64_t ph = page * a.c.H + h;
  const int ke_old = stored_exp(a.c.k_scale[ph]), ve_old = stored_exp(a.c.v_scale[ph]);
  int ke = scale_exp(group_max(ka, red));
  int ve = scale_exp(group_max(va, red));
  if (lo > 0) {                                    // older tokens stay
    ke = max(ke, ke_old);
    ve = max(ve, ve_old);
  }
  const bool k_grew = lo > 0 && ke > ke_old, v_grew = lo > 0 && ve > ve_old;

  // keys: item (piece c, token t), 16 channels
  uint8_t *kc = a.c.k + ph * (kPage * D);
  for (int i = tid; i < D / 16 * kPage; i += kKvThreads) {
    const int c = i / kPage, t = i % kPage;
    u32x4 *dst = reinterpret_cast<u32x4 *>(kc + i * 16);
    if (t >= lo && t < hi) {
      const uint16_t *src = &kt[t * ROW + c * 16];
      u32x4 w;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          f[e] = __builtin_amdgcn_ldexpf(__uint_as_float((uint32_t)src[q * 4 + e] << 16), -ke);
        w[q] = encode4(f[0], f[1], f[2], f[3]);
      }
      *dst = w;
    } else if (t < lo && k_grew) {
      u32x4 w = *dst;
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q] = recode4(w[q], ke_old - ke);
      *dst = w;
    }
  }
  // values: item (32 channels, half, channel), 16 tokens
  uint8_t *vc = a.c.v + ph * (kPage * D);
  const bool whole = lo == 0 && hi == kPage;
  for (int i = tid; i < D * 2; i += kKvThreads) {
    const int d = i / 64 * 32 + i % 32, hh = i / 32 % 2;
    u32x4 *dst = reinterpret_cast<u32x4 *>(vc + i * 16);
    u32x4 old = {0, 0, 0, 0};
    if (!whole) old = *dst;
    u32x4 w;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int t0 = 8 * g + 4 * hh;
      float f[4];
      uint32_t fresh = 0, older = 0;               // byte masks
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = t0 + e;
        const bool in = t >= lo && t < hi;
        f[e] = in ? __builtin_amdgcn_ldexpf(__uint_as_float((uint32_t)vt[t * ROW + d] << 16), -ve)
                  : 0.f;
        fresh |= in ? 0xffu << (8 * e) : 0u;
        older |= t < lo ? 0xffu << (8 * e) : 0u;
      }
      const uint32_t moved = v_grew ? recode4(old[g], ve_old - ve) : old[g];
      w[g] = (encode4(f[0], f[1], f[2], f[3]) & fresh) | (moved & older) | (old[g] & ~(fresh | older));
    }
    *dst = w;
  }
  if (tid == 0) {
    a.c.k_scale[ph] = pow2(ke);
    a.c.v_scale[ph] = pow2(ve);
  }
}

struct ReadArgs {
  CacheArgs c;
  int64_t max_pages, table_stride;
  const int32_t *table, *lens;
  uint16_t *k, *v;
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  // exact: a code times a power of two has 4 significant bits
  return (__float_as_uint(a) >> 16) | (__float_as_uint(b) & 0xffff0000u);
}

template <int D>
__global__ __launch_bounds__(kKvThreads) void kv_read_kernel(ReadArgs a) {
  constexpr int ROW = D + 2;
  __shared__ __align__(16) uint16_t vt[kPage * ROW];
  const int tid = threadIdx.x;
  const uint32_t unit = blockIdx.x / (uint32_t)a.c.H;
  const int h = (int)(blockIdx.x - unit * (uint32_t)a.c.H);
  const int64_t b = unit / (uint32_t)a.max_pages;
  const int64_t p = unit - (uint32_t)b * (uint32_t)a.max_pages;
  const int64_t n = cut_len(a.lens[b], a.max_pages);
  const int64_t page = page_of(a.table + b * a.table_stride, p, a.c.num_pages);
  const int live = page < 0 ? 0 : (int)min(max(n - p * kPage, (int64_t)0), (int64_t)kPage);
  const int64_t ph = (page < 0 ? 0 : page) * a.c.H + h;
  uint16_t *ko = a.k + ((b * a.max_pages + p) * kPage * a.c.H + h) * D;
  uint16_t *vo = a.v + ((b * a.max_pages + p) * kPage * a.c.H + h) * D;
  const int64_t tok = (int64_t)a.c.H * D;          // elements from token to token
  const float ks = live ? pow2(stored_exp(a.c.k_scale[ph])) : 0.f;
  const float vs = live ? pow2(stored_exp(a.c.v_scale[ph])) : 0.f;
  for (int i = tid; i < D / 16 * kPage; i += kKvThreads) {
    const int c = i % (D / 16), t = i / (D / 16);
    u32x4 o0 = {0, 0, 0, 0}, o1 = {0, 0, 0, 0};
    if (t < live) {
      const u32x4 w = *reinterpret_cast<const u32x4 *>(a.c.k + ph * (kPage * D) + (c * kPage + t) * 16);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[q], false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[q], true);
        const uint32_t x = pack_bf16(lo.x * ks, lo.y * ks), y = pack_bf16(hi.x * ks, hi.y * ks);
        if (q < 2) { o0[2 * q] = x; o0[2 * q + 1] = y; }
        else { o1[2 * q - 4] = x; o1[2 * q - 3] = y; }
      }
    }
    u32x4 *dst = reinterpret_cast<u32x4 *>(ko + t * tok + c * 16);
    dst[0] = o0;
    dst[1] = o1;
  }
  if (live) {
    for (int i = tid; i < D * 2; i += kKvThreads) {
      const int d = i / 64 * 32 + i % 32, hh = i / 32 % 2;
      const u32x4 w = *reinterpret_cast<const u32x4 *>(a.c.v + ph * (kPage * D) + i * 16);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[g], false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[g], true);
        const int t = 8 * g + 4 * hh;
        vt[t * ROW + d] = (uint16_t)(__float_as_uint(lo.x * vs) >> 16);
        vt[(t + 1) * ROW + d] = (uint16_t)(__float_as_uint(lo.y * vs) >> 16);
        vt[(t + 2) * ROW + d] = (uint16_t)(__float_as_uint(hi.x * vs) >> 16);
        vt[(t + 3) * ROW + d] = (uint16_t)(__float_as_uint(hi.y * vs) >> 16);
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < D / 8 * kPage; i += kKvThreads) {
    const int d = i % (D / 8) * 8, t = i / (D / 8);
    u32x4 o = {0, 0, 0, 0};
    if (t < live) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        o[q] = *reinterpret_cast<const uint32_t *>(&vt[t * ROW + d + 2 * q]);
    }
    *reinterpret_cast<u32x4 *>(vo + t * tok + d) = o;
  }
}

struct GatherArgs {
  CacheArgs c;
  int64_t max_pages, table_stride, kept_stride, new_pages, new_stride;
  const int32_t *table, *kept, *counts, *new_table;
};

// One workgroup per new page and head.  Keys: every lane fetches the 16-byte
// pieces of its token from that token's old page.  Values: a token's channels
// lie one byte in every 16-byte piece, so each old page that a kept token comes
// from is read whole (its other kept tokens are neighbours) and the lane picks
// its bytes; kept positions increase, so an old page is met once per new page.
// The values' layout, which makes attention's loads contiguous, is paid for
// here: a quarter of 106496 tokens of 8 heads of 128 channels takes 77 us, for
// 134 MB that have to move and about 335 MB that do.
template <int D>
__global__ __launch_bounds__(kKvThreads) void kv_gather_kernel(GatherArgs a) {
  constexpr int KI = (D / 16 * kPage + kKvThreads - 1) / kKvThreads;   // key items per thread
  constexpr int VI = (D * 2 + kKvThreads - 1) / kKvThreads;            // value items per thread
  __shared__ int32_t s_pos[kPage];        // old position, -1: none
  __shared__ int64_t s_page[kPage];       // old page, -1: none
  __shared__ int s_ke[kPage], s_ve[kPage];
  __shared__ float red[kKvThreads / 64];
  const int tid = threadIdx.x;
  const uint32_t unit = blockIdx.x / (uint32_t)a.c.H;
  const int h = (int)(blockIdx.x - unit * (uint32_t)a.c.H);
  const int64_t b = unit / (uint32_t)a.new_pages;
  const int64_t p = unit - (uint32_t)b * (uint32_t)a.new_pages;
  const int64_t count = min(cut_len(a.counts[b], a.new_pages), a.kept_stride);
  if (p * kPage >= count) return;
  const int64_t page = page_of(a.new_table + b * a.new_stride, p, a.c.num_pages);
  if (page < 0) return;
  if (tid < kPage) {
    const int64_t jj = p * kPage + tid;
    int64_t pos = jj < count ? a.kept[b * a.kept_stride + jj] : -1;
    if (pos < 0 || pos >= a.max_pages * kPage) pos = -1;
    const int64_t src = pos < 0 ? -1 : page_of(a.table + b * a.table_stride, pos / kPage, a.c.num_pages);
    s_pos[tid] = src < 0 ? -1 : (int32_t)(pos % kPage);
    s_page[tid] = src;
    s_ke[tid] = src < 0 ? 0 : stored_exp(a.c.k_scale[src * a.c.H + h]);
    s_ve[tid] = src < 0 ? 0 : stored_exp(a.c.v_scale[src * a.c.H + h]);
  }
  __syncthreads();

  float ka = 0.f, va = 0.f;
  u32x4 kw[KI], vw[VI];
#pragma unroll
  for (int q = 0; q < KI; ++q) {
    const int i = tid + q * kKvThreads;
    kw[q] = u32x4{0, 0, 0, 0};
    if (i >= D / 16 * kPage) continue;
    const int c = i / kPage, t = i % kPage;
    if (s_pos[t] < 0) continue;
    kw[q] = *reinterpret_cast<const u32x4 *>(a.c.k + (s_page[t] * a.c.H + h) * (kPage * D) +
                                             (c * kPage + s_pos[t]) * 16);
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) m = fmaxf(m, amax4(kw[q][e]));
    ka = fmaxf(ka, __builtin_amdgcn_ldexpf(m, s_ke[t]));
  }
#pragma unroll
  for (int q = 0; q < VI; ++q) {
    const int i = tid + q * kKvThreads;
    vw[q] = u32x4{0, 0, 0, 0};
    if (i >= D * 2) continue;
    const int hh = i / 32 % 2;
    const int dpart = (i - hh * 32) * 16;            // the channel's piece of half 0
    int64_t held = -1;
    u32x4 w0 = {0, 0, 0, 0}, w1 = {0, 0, 0, 0};      // the old page's two halves
#pragma unroll
    for (int g = 0; g < 4; ++g) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 8 * g + 4 * hh + e;
        const int pos = s_pos[t];
        if (pos < 0) continue;
        if (s_page[t] != held) {
          held = s_page[t];
          const uint8_t *src = a.c.v + (held * a.c.H + h) * (kPage * D) + dpart;
          w0 = *reinterpret_cast<const u32x4 *>(src);
          w1 = *reinterpret_cast<const u32x4 *>(src + 512);
        }
        const int og = pos / 8, oe = pos % 4;
        const u32x4 w = (pos / 4 % 2) ? w1 : w0;
        const uint32_t word = og == 0 ? w[0] : og == 1 ? w[1] : og == 2 ? w[2] : w[3];
        const uint32_t byte = (word >> (8 * oe)) & 0xffu;
        vw[q][g] |= byte << (8 * e);
        const f32x2 f = __builtin_amdgcn_cvt_pk_f32_fp8((int)byte, false);
        va = fmaxf(va, __builtin_amdgcn_ldexpf(fabsf(f.x), s_ve[t]));
      }
    }
  }
  const int ke = scale_exp(group_max(ka, red));
  const int ve = scale_exp(group_max(va, red));
  const int64_t ph = page * a.c.H + h;
#pragma unroll
  for (int q = 0; q < KI; ++q) {
    const int i = tid + q * kKvThreads;
    if (i >= D / 16 * kPage) continue;
    const int t = i % kPage;
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = recode4(kw[q][e], s_ke[t] - ke);
    *reinterpret_cast<u32x4 *>(a.c.k + ph * (kPage * D) + i * 16) = w;
  }
#pragma unroll
  for (int q = 0; q < VI; ++q) {
    const int i = tid + q * kKvThreads;
    if (i >= D * 2) continue;
    const int hh = i / 32 % 2;
    u32x4 w;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int t = 8 * g + 4 * hh;
      const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)vw[q][g], false);
      const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)vw[q][g], true);
      w[g] = encode4(__builtin_amdgcn_ldexpf(lo.x, s_ve[t] - ve),
                     __builtin_amdgcn_ldexpf(lo.y, s_ve[t + 1] - ve),
                     __builtin_amdgcn_ldexpf(hi.x, s_ve[t + 2] - ve),
                     __builtin_amdgcn_ldexpf(hi.y, s_ve[t + 3] - ve));
    }
    *reinterpret_cast<u32x4 *>(a.c.v + ph * (kPage * D) + i * 16) = w;
  }
  if (tid == 0) {
    a.c.k_scale[ph] = pow2(ke);
    a.c.v_scale[ph] = pow2(ve);
  }
}

}  // namespace

// Host side of every call that takes a cache (also attention.hip): checks the
// descriptor.
int check_cache(const char *who, const dllm_kv_cache *c) {
  if (!c) return fail(DLLM_ERR_ARG, "%s: cache is NULL", who);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(DLLM_ERR_UNSUPPORTED, "%s: head_dim = %d is not 64, 128 or 256", who, c->head_dim);
  if (c->kv_heads < 1 || c->kv_heads > 4096)
    return fail(DLLM_ERR_ARG, "%s: kv_heads = %d must be in [1, 4096]", who, c->kv_heads);
  if (c->num_pages < 1 || c->num_pages > 0x7fffffffLL)
    return fail(DLLM_ERR_ARG, "%s: num_pages must be in [1, 2^31)", who);
  if (!c->k || !c->v || !c->k_scale || !c->v_scale)
    return fail(DLLM_ERR_ARG, "%s: the cache's k, v, k_scale and v_scale must be non-NULL", who);
  if ((uintptr_t)c->k % 16 != 0 || (uintptr_t)c->v % 16 != 0 || (uintptr_t)c->k_scale % 4 != 0 ||
      (uintptr_t)c->v_scale % 4 != 0)
    return fail(DLLM_ERR_ARG, "%s: the cache's k and v must be 16-byte aligned, its scales 4-byte",
                who);
  return DLLM_OK;
}

int check_table(const char *who, const char *name, const int32_t *table, int64_t B,
                int64_t max_pages, int64_t stride) {
  if (max_pages < 0 || max_pages > (0x7fffffffLL / kPage))
    return fail(DLLM_ERR_ARG, "%s: %s has %lld pages per sequence, must be in [0, 2^26)", who, name,
                (long long)max_pages);
  if (stride < max_pages) return fail(DLLM_ERR_ARG, "%s: %s row stride < its pages", who, name);
  if (B > 0 && max_pages > 0 && (!table || (uintptr_t)table % 4 != 0))
    return fail(DLLM_ERR_ARG, "%s: %s is NULL or unaligned", who, name);
  return DLLM_OK;
}

namespace {

CacheArgs cache_args(const dllm_kv_cache &c) {
  return CacheArgs{c.k, c.v, c.k_scale, c.v_scale, c.num_pages, c.kv_heads};
}

// One workgroup per unit; DLLM_ERR_UNSUPPORTED beyond the grid's limit.
int check_units(const char *who, int64_t B, int64_t pages, int64_t H) {
  const int64_t lim = 0xffffffffLL / kKvThreads;
  if (pages > 0 && (B > lim / H || B * H > lim / pages))
    return fail(DLLM_ERR_UNSUPPORTED, "%s: more than %lld pages and heads in one call", who,
                (long long)lim);
  return DLLM_OK;
}

#define DLLM_BY_DIM(dim, kernel, grid, stream, args)                                          \
  do {                                                                                        \
    if ((dim) == 64) hipLaunchKernelGGL(kernel<64>, grid, dim3(kKvThreads), 0, stream, args); \
    else if ((dim) == 128)                                                                    \
      hipLaunchKernelGGL(kernel<128>, grid, dim3(kKvThreads), 0, stream, args);               \
    else hipLaunchKernelGGL(kernel<256>, grid, dim3(kKvThreads), 0, stream, args);            \
  } while (0)

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" int dllm_kv_write(const dllm_kv_cache *cache, const void *k, const int64_t *k_strides,
                             const void *v, const int64_t *v_strides, int64_t B, int64_t L,
                             const int32_t *page_table, int64_t max_pages, int64_t table_stride,
                             const int32_t *start, const int32_t *lens, hipStream_t stream) {
  const char *who = "dllm_kv_write";
  int rc = check_cache(who, cache);
  if (rc != DLLM_OK) return rc;
  if (B < 0 || L < 0 || B > 0x7fffffffLL || L > 0x7fffffffLL)
    return fail(DLLM_ERR_ARG, "%s: B and L must be in [0, 2^31)", who);
  rc = check_table(who, "page_table", page_table, B, max_pages, table_stride);
  if (rc != DLLM_OK) return rc;
  if (B == 0 || L == 0 || max_pages == 0) return ok();
  if (!k || !v || !k_strides || !v_strides || !start)
    return fail(DLLM_ERR_ARG, "%s: k, v, their strides and start must be non-NULL", who);
  if ((uintptr_t)k % 2 != 0 || (uintptr_t)v % 2 != 0)
    return fail(DLLM_ERR_ARG, "%s: k and v must be aligned to their element", who);
  WriteArgs a;
  memset(&a, 0, sizeof(a));
  a.c = cache_args(*cache);
  a.k = (const uint16_t *)k;
  a.v = (const uint16_t *)v;
  a.vec = (uintptr_t)k % 16 == 0 && (uintptr_t)v % 16 == 0;
  for (int i = 0; i < 3; ++i) {
    a.ks[i] = k_strides[i];
    a.vs[i] = v_strides[i];
    if (a.ks[i] % 8 != 0 || a.vs[i] % 8 != 0) a.vec = 0;
  }
  a.L = L;
  a.max_pages = max_pages;
  a.table_stride = table_stride;
  a.table = page_table;
  a.start = start;
  a.lens = lens;
  // a run of L tokens touches at most this many pages, wherever it starts
  a.touched = std::min<int64_t>((L + 2 * kPage - 2) / kPage, max_pages);
  rc = check_units(who, B, a.touched, cache->kv_heads);
  if (rc != DLLM_OK) return rc;
  const dim3 grid((uint32_t)(B * a.touched * cache->kv_heads));
  DLLM_BY_DIM(cache->head_dim, kv_write_kernel, grid, stream, a);
  return check_launch(who);
}

extern "C" int dllm_kv_read(const dllm_kv_cache *cache, int64_t B, const int32_t *page_table,
                            int64_t max_pages, int64_t table_stride, const int32_t *lens,
                            void *k_out, void *v_out, hipStream_t stream) {
  const char *who = "dllm_kv_read";
  int rc = check_cache(who, cache);
  if (rc != DLLM_OK) return rc;
  if (B < 0 || B > 0x7fffffffLL) return fail(DLLM_ERR_ARG, "%s: B must be in [0, 2^31)", who);
  rc = check_table(who, "page_table", page_table, B, max_pages, table_stride);
  if (rc != DLLM_OK) return rc;
  if (B == 0 || max_pages == 0) return ok();
  if (!lens || !k_out || !v_out)
    return fail(DLLM_ERR_ARG, "%s: lens, k_out and v_out must be non-NULL", who);
  if ((uintptr_t)k_out % 16 != 0 || (uintptr_t)v_out % 16 != 0)
    return fail(DLLM_ERR_ARG, "%s: k_out and v_out must be 16-byte aligned", who);
  rc = check_units(who, B, max_pages, cache->kv_heads);
  if (rc != DLLM_OK) return rc;
  ReadArgs a;
  memset(&a, 0, sizeof(a));
  a.c = cache_args(*cache);
  a.max_pages = max_pages;
  a.table_stride = table_stride;
  a.table = page_table;
  a.lens = lens;
  a.k = (uint16_t *)k_out;
  a.v = (uint16_t *)v_out;
  const dim3 grid((uint32_t)(B * max_pages * cache->kv_heads));
  DLLM_BY_DIM(cache->head_dim, kv_read_kernel, grid, stream, a);
  return check_launch(who);
}

extern "C" int dllm_kv_gather(const dllm_kv_cache *cache, int64_t B, const int32_t *page_table,
                              int64_t max_pages, int64_t table_stride, const int32_t *kept,
                              int64_t kept_stride, const int32_t *counts,
                              const int32_t *new_table, int64_t new_pages, int64_t new_stride,
                              hipStream_t stream) {
  const char *who = "dllm_kv_gather";
  int rc = check_cache(who, cache);
  if (rc != DLLM_OK) return rc;
  if (B < 0 || B > 0x7fffffffLL) return fail(DLLM_ERR_ARG, "%s: B must be in [0, 2^31)", who);
  rc = check_table(who, "page_table", page_table, B, max_pages, table_stride);
  if (rc != DLLM_OK) return rc;
  rc = check_table(who, "new_table", new_table, B, new_pages, new_stride);
  if (rc != DLLM_OK) return rc;
  if (kept_stride < 0) return fail(DLLM_ERR_ARG, "%s: kept_stride must be >= 0", who);
  if (B == 0 || new_pages == 0) return ok();
  if ((!kept && kept_stride > 0) || !counts || (max_pages > 0 && page_table == new_table))
    return fail(DLLM_ERR_ARG, "%s: kept and counts must be non-NULL, and new_table another table",
                who);
  rc = check_units(who, B, new_pages, cache->kv_heads);
  if (rc != DLLM_OK) return rc;
  GatherArgs a;
  memset(&a, 0, sizeof(a));
  a.c = cache_args(*cache);
  a.max_pages = max_pages;
  a.table_stride = table_stride;
  a.kept_stride = kept_stride;
  a.new_pages = new_pages;
  a.new_stride = new_stride;
  a.table = page_table;
  a.kept = kept;
  a.counts = counts;
  a.new_table = new_table;
  const dim3 grid((uint32_t)(B * new_pages * cache->kv_heads));
  DLLM_BY_DIM(cache->head_dim, kv_gather_kernel, grid, stream, a);
  return check_launch(who);
}
