// dllm_block_attention and dllm_attention_weights: attention over the 8-bit
// key/value cache.
//
// Columns: the L * G queries of one sequence and key/value head (G query heads
// share a key/value head); a wave works on 32 of them at a time.  Per page of
// 32 tokens, on the 32x32x16 matrix instructions:
//   S^T (tokens x columns) = K Q^T   keys decoded to bfloat16 (exactly: 4
//                                    significant bits times a power of two),
//   online softmax in base 2 down each column, which one lane pair holds: the
//     running maximum m, the sum l, and the weights p = 2^(s - m),
//   O^T (channels x columns) += V^T P^T   values decoded to float16 without
//     their scale, p in float16.
// The accumulator layout of S^T is the operand layout that P^T needs, since the
// cache keeps a page's values in that token order (kv_dev.h): no weight
// crosses lanes and no tile goes through LDS.
//
// p is biased by 2^14, so float16 keeps 11 bits of it down to 2^-28 and
// counts weights down to 2^-39; pages whose value scale is smaller than the largest seen
// (exponent E) have their p scaled by the difference, so the accumulator is in
// units of 2^E.
//
// The cache is split along its tokens over workgroups when there are few
// columns; a second kernel joins the parts.
#include <string.h>

#include <algorithm>

#include "kv_dev.h"

namespace dllm {

int check_cache(const char *who, const dllm_kv_cache *c);
int check_table(const char *who, const char *name, const int32_t *table, int64_t B,
                int64_t max_pages, int64_t stride);

namespace {

constexpr float kNegInf = -__builtin_inff();
constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = kAttnThreads / 64;
constexpr float kBias = 14.0f;          // weights are held as 2^14 p

struct AttnArgs {
  const uint16_t *q;
  int64_t qs[3];
  uint16_t *out;
  int64_t os[3];
  const uint8_t *k, *v;
  const float *k_scale, *v_scale;
  int64_t num_pages;
  int64_t max_pages, table_stride;
  const int32_t *table, *kv_lens, *q_start, *q_lens;
  int64_t block_len;
  int64_t B;
  int H, G, L;
  int ncols;                // L * G
  int groups;               // column groups (workgroups per sequence, head and split)
  int splits;
  int vec;                  // query rows are 16-byte aligned
  int out_vec;              // output rows are 8-byte aligned
  float c;                  // scale * log2 e
  float *lse;
  float *part_o;            // [B * H * ncols][splits][D]
  float *part_ml;           // [B * H * ncols][splits][2]
  float *weights;           // dllm_attention_weights
};

// The columns of one wave tile: lane i of each half is column c0 + i.
struct Column {
  int l, g;        // query and query head within the group
  bool on;         // a real query
  int lim;         // it attends to tokens t < lim
};

__device__ __forceinline__ Column column(const AttnArgs &a, int64_t b, int64_t c, int n,
                                         int64_t q_len) {
  Column r;
  const int cc = c < a.ncols ? (int)c : 0;
  r.l = cc / a.G;
  r.g = cc - r.l * a.G;
  r.on = c < a.ncols && r.l < q_len;
  r.lim = r.on ? n : 0;
  if (a.block_len > 0 && r.on) {
    const int64_t s = a.q_start ? max((int64_t)a.q_start[b], (int64_t)0) : 0;
    r.lim = (int)min((int64_t)n, ((s + r.l) / a.block_len + 1) * a.block_len);
  }
  return r;
}

// The column's query as D / 16 operand pieces: piece s of half h holds
// channels 32 (s / 2) + 16 h + 8 (s % 2) .. + 7, as the keys' pieces do.
template <int D>
__device__ __forceinline__ void load_query(const AttnArgs &a, int64_t b, int64_t head,
                                           const Column &col, bf16x8 (&q)[D / 16]) {
  const int h = (threadIdx.x & 63) >> 5;
  const uint16_t *row = a.q + b * a.qs[0] + col.l * a.qs[1] + head * a.qs[2];
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
    const int d = 32 * (s / 2) + 16 * h + 8 * (s % 2);
    u32x4 w = {0, 0, 0, 0};
    if (col.on) {
      if (a.vec) {
        w = *reinterpret_cast<const u32x4 *>(row + d);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = (uint32_t)row[d + 2 * e] | (uint32_t)row[d + 2 * e + 1] << 16;
      }
    }
    q[s] = __builtin_bit_cast(bf16x8, w);
  }
}

// 8 codes times a power of two, exactly.
__device__ __forceinline__ bf16x8 decode_bf16(uint32_t w0, uint32_t w1, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, scale, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, scale, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, scale, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, scale, true);
  return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}
__device__ __forceinline__ f16x8 decode_f16(uint32_t w0, uint32_t w1) {
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, false);
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, true);
  const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, false);
  const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, true);
  return f16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// Maximum and sum of the two lanes of a column (v_permlane32_swap: both lanes
// get the lower half's value in one register and the upper half's in another).
__device__ __forceinline__ float halves_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float halves_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// A page's pieces of this lane, as stored (keys or values).
template <int D>
__device__ __forceinline__ void load_pieces(const uint8_t *base, int64_t ph, u32x4 (&w)[D / 32]) {
  const u32x4 *p = reinterpret_cast<const u32x4 *>(base + ph * (kPage * D)) + (threadIdx.x & 63);
#pragma unroll
  for (int c = 0; c < D / 32; ++c) w[c] = p[c * 64];
}

// State of one tile of 32 columns.
template <int D>
struct Tile {
  f32x16 o[D / 32];     // O^T: channel 32 c + 8 (r / 4) + 4 h + r % 4 of the lane's column
  float m, l;           // base-2 maximum; biased sum over this half's tokens
};

// S^T of one page: tokens x columns, in the keys' own unit.
template <int D, int QT>
__device__ __forceinline__ void score_page(const u32x4 (&kw)[D / 32], float ks,
                                           const bf16x8 (&q)[QT][D / 16], f32x16 (&s)[QT]) {
#pragma unroll
  for (int x = 0; x < QT; ++x)
#pragma unroll
    for (int r = 0; r < 16; ++r) s[x][r] = 0.f;
#pragma unroll
  for (int st = 0; st < D / 16; ++st) {
    const bf16x8 k = decode_bf16(kw[st / 2][2 * (st % 2)], kw[st / 2][2 * (st % 2) + 1], ks);
#pragma unroll
    for (int x = 0; x < QT; ++x)
      s[x] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, q[x][st], s[x], 0, 0, 0);
  }
}

// The weights of one page (tokens t0 ..) and the running maximum and sum.
template <int D>
__device__ __forceinline__ void weigh_page(float c, int t0, int lim, bool masked, int ve, int E,
                                           f32x16 &s, Tile<D> &tile, f16x8 (&p)[2]) {
  const int h = (threadIdx.x & 63) >> 5;
  if (masked) {
    const int left = lim - t0 - 4 * h;
#pragma unroll
    for (int r = 0; r < 16; ++r)
      if (8 * (r / 4) + r % 4 >= left) s[r] = kNegInf;
  }
  float mx = s[0];
#pragma unroll
  for (int r = 1; r < 16; ++r) mx = fmaxf(mx, s[r]);
  mx = halves_max(mx) * c;
  const float m1 = fmaxf(tile.m, mx);
  if (__builtin_amdgcn_ballot_w64(m1 > tile.m) != 0) {
    // (-inf) - (-inf) never arises: m1 is above -inf where it rose
    const float f = m1 > tile.m ? __builtin_amdgcn_exp2f(tile.m - m1) : 1.0f;
    tile.l *= f;
#pragma unroll
    for (int cc = 0; cc < D / 32; ++cc) tile.o[cc] *= f;
    tile.m = m1;
  }
  // a column that has met no token yet has m = -inf: weights 0
  const float sub = m1 == kNegInf ? 0.f : m1 - kBias;
  float w[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) w[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -sub));
  float l = 0.f;
#pragma unroll
  for (int r = 0; r < 16; ++r) l += w[r];
  tile.l += l;
  if (ve < E) {
    const float f = __builtin_amdgcn_ldexpf(1.0f, ve - E);
#pragma unroll
    for (int r = 0; r < 16; ++r) w[r] *= f;
  }
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int r = 0; r < 8; ++r) p[e][r] = (_Float16)w[8 * e + r];
}

// Columns' results: the output itself, or this split's part.
template <int D>
__device__ __forceinline__ void store_tile(const AttnArgs &a, int64_t b, int hkv, int64_t c, int split,
                                           const Column &col, const Tile<D> &t, int E) {
  const int h = (threadIdx.x & 63) >> 5;
  const float l = halves_sum(t.l);
  if (!col.on) return;
  const float unit = pow2(E);
  if (a.splits == 1) {
    const float inv = l > 0.f ? 1.0f / l : (l == l ? 0.f : l);
    const int64_t head = (int64_t)hkv * a.G + col.g;
    uint16_t *o = a.out + b * a.os[0] + col.l * a.os[1] + head * a.os[2];
#pragma unroll
    for (int cc = 0; cc < D / 32; ++cc)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint16_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          y[e] = __builtin_bit_cast(uint16_t, (__bf16)(t.o[cc][4 * g + e] * inv * unit));
        const int d = 32 * cc + 8 * g + 4 * h;
        if (a.out_vec) {
          *reinterpret_cast<uint2 *>(o + d) = __builtin_bit_cast(uint2, y);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) o[d + e] = y[e];
        }
      }
    if (h == 0)
      a.lse[(b * a.H * a.G + head) * a.L + col.l] =
          (t.m + __builtin_amdgcn_logf(l) - kBias) * kLn2;      // -inf when it met nothing
    return;
  }
  const int64_t row = ((b * a.H + hkv) * a.ncols + c) * a.splits + split;
  float *po = a.part_o + row * D;
#pragma unroll
  for (int cc = 0; cc < D / 32; ++cc)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      f32x4 y;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = t.o[cc][4 * g + e] * unit;
      *reinterpret_cast<f32x4 *>(po + 32 * cc + 8 * g + 4 * h) = y;
    }
  if (h == 0) {
    a.part_ml[2 * row] = t.m;
    a.part_ml[2 * row + 1] = l;
  }
}

// WIDE: the four waves take different columns and the same pages; else they
// share QT column tiles and take every fourth page, joined through LDS.
template <int D, int QT, bool WIDE>
__global__ __launch_bounds__(kAttnThreads) void attention_kernel(AttnArgs a) {
  constexpr int REGS = D / 2;                      // accumulator registers of a tile
  __shared__ float s_o[WIDE ? 1 : 2 * REGS * 64];
  __shared__ float s_ml[WIDE ? 1 : 2 * 3 * 64];
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t unit = blockIdx.x;
  const int group = (int)(unit % a.groups);
  unit /= a.groups;
  const int split = (int)(unit % a.splits);
  unit /= a.splits;
  const int hkv = (int)(unit % a.H);
  const int64_t b = unit / a.H;
  const int64_t c0 = WIDE ? ((int64_t)group * kAttnWaves + wave) * (32 * QT) : (int64_t)group * (32 * QT);
  if (WIDE && c0 >= a.ncols) return;
  const int n = (int)cut_len(a.kv_lens[b], a.max_pages);
  const int64_t q_len = a.q_lens ? min((int64_t)a.q_lens[b], (int64_t)a.L) : a.L;

  Column col[QT];
  bf16x8 q[QT][D / 16];
  Tile<D> tile[QT];
  int max_lim = 0, min_lim = 0x7fffffff;
#pragma unroll
  for (int x = 0; x < QT; ++x) {
    col[x] = column(a, b, c0 + 32 * x + (lane & 31), n, q_len);
    load_query<D>(a, b, (int64_t)hkv * a.G + col[x].g, col[x], q[x]);
    max_lim = max(max_lim, col[x].lim);
    min_lim = min(min_lim, col[x].lim);
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
#pragma unroll
      for (int r = 0; r < 16; ++r) tile[x].o[c][r] = 0.f;
    tile[x].m = kNegInf;
    tile[x].l = 0.f;
  }
  max_lim = -wave_min_i(-max_lim);
  min_lim = wave_min_i(min_lim);
  int E = kScaleMin;
  const int64_t pages = (max_lim + kPage - 1) / kPage;
  const int lo = (int)(pages * split / a.splits), hi = (int)(pages * (split + 1) / a.splits);
  const int32_t *row = a.table + b * a.table_stride;
  constexpr int STEP = WIDE ? 1 : kAttnWaves;
  int t = WIDE ? lo : lo + wave;
  if (t < hi) {
    // One buffer each for keys and values: the next page's keys are fetched
    // when this page's scores are done with them, its values after the
    // products, so each load has the other half of a page's work to arrive.
    u32x4 kw[D / 32], vw[D / 32];
    int64_t id = page_of(row, t, a.num_pages);
    int64_t ph = max(id, (int64_t)0) * a.H + hkv;     // a missing page reads page 0, unused
    load_pieces<D>(a.k, ph, kw);
    load_pieces<D>(a.v, ph, vw);
    float ks = pow2(stored_exp(a.k_scale[ph]));
    int ve = stored_exp(a.v_scale[ph]);
    for (;;) {
      const bool here = id >= 0;
      const int next = t + STEP < hi ? t + STEP : t;
      const int64_t id1 = page_of(row, next, a.num_pages);
      const int64_t ph1 = max(id1, (int64_t)0) * a.H + hkv;
      f32x16 s[QT];
      if (here) score_page<D, QT>(kw, ks, q, s);
      load_pieces<D>(a.k, ph1, kw);
      const float ks1 = pow2(stored_exp(a.k_scale[ph1]));
      const int ve1 = stored_exp(a.v_scale[ph1]);
      if (here) {
        const int t0 = t * kPage;
        if (t0 + kPage > n) {
          // the cache ends inside this page: what lies behind may be any bits,
          // and 0 * NaN is NaN, so the values there become 0
          const int live = n - t0 - 4 * h;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int m = min(max(live - 8 * g, 0), 4);
            const uint32_t keep = m == 4 ? ~0u : (1u << (8 * m)) - 1u;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) vw[c][g] &= keep;
          }
        }
        if (ve > E) {
          // the accumulators' unit 2^E follows the largest value scale
          const float f = __builtin_amdgcn_ldexpf(1.0f, E - ve);
#pragma unroll
          for (int x = 0; x < QT; ++x)
#pragma unroll
            for (int c = 0; c < D / 32; ++c) tile[x].o[c] *= f;
          E = ve;
        }
        f16x8 p[QT][2];
#pragma unroll
        for (int x = 0; x < QT; ++x)
          weigh_page<D>(a.c, t0, col[x].lim, t0 + kPage > min_lim, ve, E, s[x], tile[x], p[x]);
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const f16x8 v = decode_f16(vw[c][2 * e], vw[c][2 * e + 1]);
#pragma unroll
            for (int x = 0; x < QT; ++x)
              tile[x].o[c] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, p[x][e], tile[x].o[c], 0, 0, 0);
          }
      }
      if (next == t) break;
      load_pieces<D>(a.v, ph1, vw);
      t = next;
      id = id1;
      ks = ks1;
      ve = ve1;
    }
  }
  if constexpr (!WIDE) {
    // waves 2, 3 into 0, 1, then 1 into 0: every lane its own column's rows
#pragma unroll
    for (int x = 0; x < QT; ++x) {
#pragma unroll
      for (int step = 2; step >= 1; step >>= 1) {
        __syncthreads();
        if (wave >= step && wave < 2 * step) {
          const int slot = wave - step;
#pragma unroll
          for (int c = 0; c < D / 32; ++c)
#pragma unroll
            for (int r = 0; r < 16; ++r) s_o[(slot * REGS + c * 16 + r) * 64 + lane] = tile[x].o[c][r];
          s_ml[(slot * 3 + 0) * 64 + lane] = tile[x].m;
          s_ml[(slot * 3 + 1) * 64 + lane] = tile[x].l;
          s_ml[(slot * 3 + 2) * 64 + lane] = __int_as_float(E);
        }
        __syncthreads();
        if (wave < step) {
          const float om = s_ml[(wave * 3 + 0) * 64 + lane], ol = s_ml[(wave * 3 + 1) * 64 + lane];
          const int oe = __float_as_int(s_ml[(wave * 3 + 2) * 64 + lane]);
          const float m1 = fmaxf(tile[x].m, om);
          const float fa = tile[x].m == kNegInf ? 0.f : __builtin_amdgcn_exp2f(tile[x].m - m1);
          const float fb = om == kNegInf ? 0.f : __builtin_amdgcn_exp2f(om - m1);
          // a NaN column stays NaN: its sum is
          tile[x].l = tile[x].l * fa + ol * fb;
          // units: the larger exponent for this column tile
          const int e1 = max(E, oe);
          const float ga = fa * __builtin_amdgcn_ldexpf(1.0f, E - e1);
          const float gb = fb * __builtin_amdgcn_ldexpf(1.0f, oe - e1);
#pragma unroll
          for (int c = 0; c < D / 32; ++c)
#pragma unroll
            for (int r = 0; r < 16; ++r)
              tile[x].o[c][r] = tile[x].o[c][r] * ga + s_o[(wave * REGS + c * 16 + r) * 64 + lane] * gb;
          tile[x].m = m1;
          // the other tiles of this wave are still in the old unit
#pragma unroll
          for (int y = 0; y < QT; ++y)
            if (y != x) {
              const float f = __builtin_amdgcn_ldexpf(1.0f, E - e1);
#pragma unroll
              for (int c = 0; c < D / 32; ++c) tile[y].o[c] *= f;
            }
          E = e1;
        }
      }
    }
    if (wave != 0) return;
  }
#pragma unroll
  for (int x = 0; x < QT; ++x)
    store_tile<D>(a, b, hkv, c0 + 32 * x + (lane & 31), split, col[x], tile[x], E);
}

// One wave per query and head: joins the splits' parts in split order.
template <int D>
__global__ __launch_bounds__(kAttnThreads) void attention_join_kernel(AttnArgs a) {
  constexpr int PER = D / 64;
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * kAttnWaves + (threadIdx.x >> 6);
  if (row >= a.B * a.H * a.ncols) return;
  const int64_t c = row % a.ncols, bh = row / a.ncols;
  const int hkv = (int)(bh % a.H);
  const int64_t b = bh / a.H;
  const int l = (int)(c / a.G), g = (int)(c % a.G);
  const int64_t q_len = a.q_lens ? min((int64_t)a.q_lens[b], (int64_t)a.L) : a.L;
  if (l >= q_len) return;
  const float *ml = a.part_ml + row * a.splits * 2;
  float m = kNegInf;
  for (int s = lane; s < a.splits; s += 64) m = fmaxf(m, ml[2 * s]);
  m = wave_max(m);
  const float *po = a.part_o + row * a.splits * D + lane * PER;
  float acc[PER], sum = 0.f;
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
  for (int s = 0; s < a.splits; ++s) {
    const float ms = ml[2 * s];
    const float f = ms == kNegInf ? 0.f : __builtin_amdgcn_exp2f(ms - m);
    sum = fmaf(ml[2 * s + 1], f, sum);
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = fmaf(po[(int64_t)s * D + e], f, acc[e]);
  }
  const float inv = sum > 0.f ? 1.0f / sum : (sum == sum ? 0.f : sum);
  const int64_t head = (int64_t)hkv * a.G + g;
  uint16_t *o = a.out + b * a.os[0] + l * a.os[1] + head * a.os[2] + lane * PER;
#pragma unroll
  for (int e = 0; e < PER; ++e) o[e] = __builtin_bit_cast(uint16_t, (__bf16)(acc[e] * inv));
  if (lane == 0)
    a.lse[(b * a.H * a.G + head) * a.L + l] =
        (m + __builtin_amdgcn_logf(sum) - kBias) * kLn2;
}

// Attention weights: one workgroup per sequence and page.  Each wave takes every
// fourth (head, column tile), recomputes S^T, and adds 2^(s - lse) into one
// register per token of its lane's columns; the lanes and waves meet in LDS
// once, in a fixed order.
template <int D>
__global__ __launch_bounds__(kAttnThreads) void attention_weights_kernel(AttnArgs a) {
  __shared__ float s_w[kAttnWaves * 64 * 17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5;
  const int64_t t = blockIdx.x % a.max_pages, b = blockIdx.x / a.max_pages;
  const int64_t n = cut_len(a.kv_lens[b], a.max_pages);
  const int64_t t0 = t * kPage;
  if (t0 >= n) return;
  const int64_t id = page_of(a.table + b * a.table_stride, t, a.num_pages);
  if (id < 0) return;
  const int64_t q_len = a.q_lens ? min((int64_t)a.q_lens[b], (int64_t)a.L) : a.L;
  const int tiles = (a.ncols + 31) / 32;
  float w[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) w[r] = 0.f;
  int held = -1;
  bf16x8 k[D / 16];
  for (int64_t u = wave; u < (int64_t)a.H * tiles; u += kAttnWaves) {
    const int hkv = (int)(u / tiles);
    const int64_t c0 = u % tiles * 32;
    const Column col = column(a, b, c0 + (lane & 31), n, q_len);
    if (__builtin_amdgcn_ballot_w64(col.lim > t0) == 0) continue;
    if (hkv != held) {
      held = hkv;
      const int64_t ph = id * a.H + hkv;
      const u32x4 *kp = reinterpret_cast<const u32x4 *>(a.k + ph * (kPage * D)) + lane;
      const float ks = pow2(stored_exp(a.k_scale[ph]));
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        const u32x4 x = kp[c * 64];
        k[2 * c] = decode_bf16(x[0], x[1], ks);
        k[2 * c + 1] = decode_bf16(x[2], x[3], ks);
      }
    }
    const int64_t head = (int64_t)hkv * a.G + col.g;
    bf16x8 q[D / 16];
    load_query<D>(a, b, head, col, q);
    f32x16 s;
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = 0.f;
#pragma unroll
    for (int st = 0; st < D / 16; ++st)
      s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[st], q[st], s, 0, 0, 0);
    const float z = col.on ? a.lse[(b * a.H * a.G + head) * a.L + col.l] : kNegInf;
    const float sub = z * kLog2e;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const bool in = t0 + 8 * (r / 4) + 4 * h + r % 4 < col.lim && z != kNegInf;
      w[r] += in ? __builtin_amdgcn_exp2f(fmaf(s[r], a.c, -sub)) : 0.f;
    }
  }
#pragma unroll
  for (int r = 0; r < 16; ++r) s_w[(wave * 64 + lane) * 17 + r] = w[r];
  __syncthreads();
  // thread (token, eighth): 16 of the 128 (wave, lane) columns, then a fold
  const int tok = threadIdx.x >> 3, part = threadIdx.x & 7;
  const int r = tok / 8 * 4 + tok % 4, half = tok / 4 % 2;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int j = part * 16 + i;                 // wave j / 32, column j % 32
    sum += s_w[((j / 32) * 64 + half * 32 + j % 32) * 17 + r];
  }
  sum += __shfl_xor(sum, 1);
  sum += __shfl_xor(sum, 2);
  sum += __shfl_xor(sum, 4);
  if (part == 0 && t0 + tok < n) a.weights[b * a.max_pages * kPage + t0 + tok] += sum;
}

// ---------------------------------------------------------------- host side

struct AttnPlan {
  int qt;          // column tiles per wave
  bool wide;
  int groups, splits;
};

// Up to 64 columns: the waves of a workgroup share them and take turns at the
// pages (more bytes in flight per column); above, each wave has its own
// columns and the four read the same pages from the CU's cache.
AttnPlan attn_plan(int64_t B, int64_t ncols, int64_t H, int64_t D, int64_t max_pages) {
  AttnPlan p;
  p.qt = D == 256 || ncols <= 32 ? 1 : 2;
  p.wide = ncols > 32 * p.qt;
  const int64_t per = 32 * p.qt * (p.wide ? kAttnWaves : 1);
  p.groups = (int)((ncols + per - 1) / per);
  // workgroups for two rounds of the CUs, of at least 4 pages (wide) or 2
  // pages a wave
  const int64_t want = 2LL * device_cu_count();
  const int64_t units = std::max<int64_t>(1, B * H * p.groups);
  int64_t s = (want + units - 1) / units;
  s = std::min<int64_t>(s, std::max<int64_t>(1, max_pages / (p.wide ? 4 : 2 * kAttnWaves)));
  p.splits = (int)std::min<int64_t>(std::max<int64_t>(1, s), 128);
  return p;
}

size_t attn_workspace(int64_t rows, int splits, int64_t D) {
  return splits <= 1 ? 0 : (size_t)rows * splits * (D + 2) * 4;
}

int check_attention(const char *who, const dllm_kv_cache *cache, const void *q,
                    const int64_t *q_strides, int64_t B, int64_t L, int64_t q_heads,
                    const int32_t *page_table, int64_t max_pages, int64_t table_stride,
                    const int32_t *kv_lens, int64_t block_len, float scale) {
  int rc = check_cache(who, cache);
  if (rc != DLLM_OK) return rc;
  if (B < 0 || L < 0 || B > 0x7fffffffLL)
    return fail(DLLM_ERR_ARG, "%s: B and L must be in [0, 2^31)", who);
  if (q_heads < 1 || q_heads % cache->kv_heads != 0 || q_heads > 0x7fffffLL)
    return fail(DLLM_ERR_ARG, "%s: q_heads = %lld must be a positive multiple of kv_heads = %d", who,
                (long long)q_heads, cache->kv_heads);
  if (L > 0x7fffff00LL / q_heads || (B > 0 && L > 0 && L * q_heads > (1LL << 40) / B))
    return fail(DLLM_ERR_UNSUPPORTED, "%s: too many queries in one call", who);
  rc = check_table(who, "page_table", page_table, B, max_pages, table_stride);
  if (rc != DLLM_OK) return rc;
  if (block_len < 0 || block_len > 0x7fffffffLL)
    return fail(DLLM_ERR_ARG, "%s: block_len must be in [0, 2^31)", who);
  if (!(scale > 0.0f) || scale == __builtin_inff())
    return fail(DLLM_ERR_ARG, "%s: scale must be finite and > 0", who);
  if (B == 0 || L == 0) return DLLM_OK;
  if (!q || !q_strides || !kv_lens)
    return fail(DLLM_ERR_ARG, "%s: q, q_strides and kv_lens must be non-NULL", who);
  if ((uintptr_t)q % 2 != 0) return fail(DLLM_ERR_ARG, "%s: q must be aligned to its element", who);
  return DLLM_OK;
}

AttnArgs attn_args(const dllm_kv_cache &c, const void *q, const int64_t *q_strides, int64_t B,
                   int64_t L, int64_t q_heads, const int32_t *page_table, int64_t max_pages,
                   int64_t table_stride, const int32_t *kv_lens, const int32_t *q_start,
                   const int32_t *q_lens, int64_t block_len, float scale) {
  AttnArgs a;
  memset(&a, 0, sizeof(a));
  a.q = (const uint16_t *)q;
  a.vec = (uintptr_t)q % 16 == 0;
  for (int i = 0; i < 3; ++i) {
    a.qs[i] = q_strides[i];
    if (a.qs[i] % 8 != 0) a.vec = 0;
  }
  a.k = c.k;
  a.v = c.v;
  a.k_scale = c.k_scale;
  a.v_scale = c.v_scale;
  a.num_pages = c.num_pages;
  a.max_pages = max_pages;
  a.table_stride = table_stride;
  a.table = page_table;
  a.kv_lens = kv_lens;
  a.q_start = q_start;
  a.q_lens = q_lens;
  a.block_len = block_len;
  a.B = B;
  a.H = c.kv_heads;
  a.G = (int)(q_heads / c.kv_heads);
  a.L = (int)L;
  a.ncols = (int)(L * a.G);
  a.c = scale * 1.4426950408889634f;
  return a;
}

template <int D>
void launch_attention(const AttnPlan &p, const AttnArgs &a, dim3 grid, hipStream_t s) {
  const dim3 block(kAttnThreads);
  if constexpr (D <= 128) {
    if (p.qt == 2) {
      if (p.wide) hipLaunchKernelGGL((attention_kernel<D, 2, true>), grid, block, 0, s, a);
      else hipLaunchKernelGGL((attention_kernel<D, 2, false>), grid, block, 0, s, a);
      return;
    }
    hipLaunchKernelGGL((attention_kernel<D, 1, false>), grid, block, 0, s, a);
  } else {
    if (p.wide) hipLaunchKernelGGL((attention_kernel<D, 1, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((attention_kernel<D, 1, false>), grid, block, 0, s, a);
  }
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" size_t dllm_block_attention_workspace_size(int64_t B, int64_t L, int64_t q_heads,
                                                      int64_t kv_heads, int64_t head_dim,
                                                      int64_t max_pages) {
  if (B < 0 || L < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || max_pages < 0 ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return 0;
  const AttnPlan p = attn_plan(B, L * (q_heads / kv_heads), kv_heads, head_dim, max_pages);
  return attn_workspace(B * L * q_heads, p.splits, head_dim);
}

extern "C" int dllm_block_attention(const dllm_kv_cache *cache, const void *q,
                                    const int64_t *q_strides, int64_t B, int64_t L,
                                    int64_t q_heads, const int32_t *page_table,
                                    int64_t max_pages, int64_t table_stride,
                                    const int32_t *kv_lens, const int32_t *q_start,
                                    const int32_t *q_lens, int64_t block_len, float scale,
                                    void *out, const int64_t *out_strides, float *lse,
                                    void *workspace, size_t workspace_bytes, hipStream_t stream) {
  const char *who = "dllm_block_attention";
  const int rc = check_attention(who, cache, q, q_strides, B, L, q_heads, page_table, max_pages,
                                 table_stride, kv_lens, block_len, scale);
  if (rc != DLLM_OK) return rc;
  if (B == 0 || L == 0) return ok();
  if (!out || !out_strides || !lse)
    return fail(DLLM_ERR_ARG, "%s: out, out_strides and lse must be non-NULL", who);
  if ((uintptr_t)out % 2 != 0) return fail(DLLM_ERR_ARG, "%s: out must be aligned to its element", who);
  if (out == q) return fail(DLLM_ERR_ARG, "%s: out aliases q", who);
  AttnArgs a = attn_args(*cache, q, q_strides, B, L, q_heads, page_table, max_pages, table_stride,
                         kv_lens, q_start, q_lens, block_len, scale);
  const int D = cache->head_dim;
  const AttnPlan p = attn_plan(B, a.ncols, a.H, D, max_pages);
  const int64_t rows = B * L * q_heads;
  const size_t need = attn_workspace(rows, p.splits, D);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(DLLM_ERR_SHAPE, "%s: workspace has %zu bytes, needs %zu", who, workspace_bytes, need);
  if (need > 0 && (uintptr_t)workspace % 16 != 0)
    return fail(DLLM_ERR_ARG, "%s: workspace must be 16-byte aligned", who);
  const int64_t wgs = B * a.H * p.groups * p.splits;
  const int64_t limit = 0xffffffffLL / kAttnThreads;
  if (wgs > limit || (rows + kAttnWaves - 1) / kAttnWaves > limit)
    return fail(DLLM_ERR_UNSUPPORTED, "%s: too many queries in one call", who);
  a.out = (uint16_t *)out;
  a.out_vec = (uintptr_t)out % 8 == 0;
  for (int i = 0; i < 3; ++i) {
    a.os[i] = out_strides[i];
    if (a.os[i] % 4 != 0) a.out_vec = 0;
  }
  a.lse = lse;
  a.groups = p.groups;
  a.splits = p.splits;
  a.part_o = (float *)workspace;
  a.part_ml = (float *)workspace + (need > 0 ? rows * p.splits * D : 0);
  const dim3 grid((uint32_t)wgs);
  if (D == 64) launch_attention<64>(p, a, grid, stream);
  else if (D == 128) launch_attention<128>(p, a, grid, stream);
  else launch_attention<256>(p, a, grid, stream);
  const int st = check_launch(who);
  if (st != DLLM_OK || p.splits == 1) return st;
  const dim3 jgrid((uint32_t)((rows + kAttnWaves - 1) / kAttnWaves));
  if (D == 64)
    hipLaunchKernelGGL(attention_join_kernel<64>, jgrid, dim3(kAttnThreads), 0, stream, a);
  else if (D == 128)
    hipLaunchKernelGGL(attention_join_kernel<128>, jgrid, dim3(kAttnThreads), 0, stream, a);
  else
    hipLaunchKernelGGL(attention_join_kernel<256>, jgrid, dim3(kAttnThreads), 0, stream, a);
  return check_launch(who);
}

extern "C" int dllm_attention_weights(const dllm_kv_cache *cache, const void *q,
                                      const int64_t *q_strides, int64_t B, int64_t L,
                                      int64_t q_heads, const int32_t *page_table,
                                      int64_t max_pages, int64_t table_stride,
                                      const int32_t *kv_lens, const int32_t *q_start,
                                      const int32_t *q_lens, int64_t block_len, float scale,
                                      const float *lse, float *weights, hipStream_t stream) {
  const char *who = "dllm_attention_weights";
  const int rc = check_attention(who, cache, q, q_strides, B, L, q_heads, page_table, max_pages,
                                 table_stride, kv_lens, block_len, scale);
  if (rc != DLLM_OK) return rc;
  if (B == 0 || L == 0 || max_pages == 0) return ok();
  if (!lse || !weights) return fail(DLLM_ERR_ARG, "%s: lse and weights must be non-NULL", who);
  AttnArgs a = attn_args(*cache, q, q_strides, B, L, q_heads, page_table, max_pages, table_stride,
                         kv_lens, q_start, q_lens, block_len, scale);
  a.lse = const_cast<float *>(lse);
  a.weights = weights;
  const int64_t wgs = B * max_pages;
  if (B > (0xffffffffLL / kAttnThreads) / max_pages)
    return fail(DLLM_ERR_UNSUPPORTED, "%s: too many pages in one call", who);
  const dim3 grid((uint32_t)wgs);
  if (cache->head_dim == 64)
    hipLaunchKernelGGL(attention_weights_kernel<64>, grid, dim3(kAttnThreads), 0, stream, a);
  else if (cache->head_dim == 128)
    hipLaunchKernelGGL(attention_weights_kernel<128>, grid, dim3(kAttnThreads), 0, stream, a);
  else
    hipLaunchKernelGGL(attention_weights_kernel<256>, grid, dim3(kAttnThreads), 0, stream, a);
  return check_launch(who);
}
