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
// A page's value scale 2^e goes into the exponents: w = 2^(s + e - m) multiplies
// the codes, and the running reference m is that of s + e, what a token adds to
// the output, so float16 keeps 11 bits of every w down to 2^-28 of the largest
// and counts down to 2^-39 of it, however the scales differ.  m is an integer:
// then every subtraction in an exponent and every rescaling is exact.
//
// A workgroup is CW column waves times KW token waves: the column waves read
// the same pages (from the CU's cache), the token waves take turns at the pages
// and join through LDS.  When that leaves CUs idle the cache is also split
// along its tokens over workgroups, as evenly as the sequences' lengths allow
// (share_of), and a second kernel joins the parts.
#include <string.h>

#include <algorithm>

#include "kv_dev.h"

namespace dllm {

int check_cache(const char *who, const dllm_kv_cache *c);
int check_table(const char *who, const char *name, const int32_t *table, int64_t B,
                int64_t max_pages, int64_t stride);

namespace {

constexpr float kNegInf = -__builtin_inff();
constexpr int kJoinThreads = 256;
constexpr int kJoinWaves = kJoinThreads / 64;
constexpr float kBias = 14.0f;          // weights are held as 2^14 w
// The reference m follows the maximum when that has risen by more than this
// above it: weights stay below 2^15.5, within float16, and the accumulators are
// rescaled rarely.
constexpr float kRise = 1.0f;
// Smallest exponent that goes into m: the sum of weights, which takes it out
// again, stays within float32.  Pages of smaller values (below 2^-71) have
// their weights scaled by the rest, within float16's 2^-20.
constexpr int kMinExp = -80;

// n / d for n < 2^31 by multiplication: with 2^(s-1) < d <= 2^s and
// m = floor(2^32 (2^s - d) / d) + 1, n / d = (floor(n m / 2^32) + n) / 2^s
// (Granlund and Montgomery, "Division by invariant integers using
// multiplication", PLDI 1994).
struct Divisor { uint32_t mul, shift; };

inline Divisor divisor(uint32_t d) {
  uint32_t s = 0;
  while (s < 31 && (1u << s) < d) ++s;
  return {(uint32_t)((((uint64_t)1 << s) - d) * ((uint64_t)1 << 32) / d + 1), s};
}
__device__ __forceinline__ uint32_t divide(uint32_t n, Divisor d) {
  return (__umulhi(n, d.mul) + n) >> d.shift;
}

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
  uint32_t block_len;       // 0: no mask
  Divisor by_group, by_block;
  int64_t B;
  int H, G, L;
  int ncols;                // L * G
  int groups;               // column groups (workgroups per sequence, head and split)
  int slots;                // shares of the sequences, over all of them: B, no splits, or more
  int min_pages;            // of a share, unless its sequence has less
  int vec;                  // query rows are 16-byte aligned
  int out_vec;              // output rows are 8-byte aligned
  float c;                  // scale * log2 e
  float *lse;
  float *part_o;            // [slots][H * ncols][D]
  float *part_ml;           // [slots][H * ncols][2]
  int2 *part_of;            // [B]: a sequence's first slot and number of slots
  // dllm_attention_weights
  float *weights;
  float *part_w;            // [parts][B][T]
  int parts, shares;        // H * shares
  int token_groups;
};

// What a workgroup takes of the tokens: share `split` of the `splits` even ones
// of sequence b (b < 0: nothing), whose length is len.
struct Share { int b, split, splits, len; };

constexpr int kRowShr1 = 0x111, kRowShr2 = 0x112, kRowShr4 = 0x114, kRowShr8 = 0x118;

constexpr int kShareLanes = 4;           // sequences a lane looks after: splits need B <= 256

// The share in slot `slot`.  Lengths are on the device, so every workgroup works
// the division out for itself: with `per` pages a share, the smallest (within a
// sixteenth) for which the slots suffice, sequence b has ceil(pages_b / per)
// shares, one if it is empty, and their slots follow each other in the order of
// b.  The slots suffice for per >= total / (slots - B): at most B shares are not
// full.  Eight lengths of 32768 and seven times 500 take 27 us so, against 46 us
// with as many shares for each; equal ones take up to 1.6 us more (24 of 2000).
__device__ __forceinline__ Share share_of(const AttnArgs &a, int slot) {
  const int lane = threadIdx.x & 63;
  int len[kShareLanes] = {};
  float pages[kShareLanes];
#pragma unroll
  for (int j = 0; j < kShareLanes; ++j)
    if (j * 64 < a.B) len[j] = a.kv_lens[min((int64_t)(j * 64 + lane), a.B - 1)];
  int sum = 0;
#pragma unroll
  for (int j = 0; j < kShareLanes; ++j) {
    // 2^21 pages are as long as any for this purpose: sums stay within 2^30,
    // and page counts are exact in float32
    const int64_t n = (cut_len(len[j], a.max_pages) + kPage - 1) / kPage;
    const int m = j * 64 + lane < a.B ? (int)min(n, (int64_t)(1 << 21) - 1) : 0;
    pages[j] = (float)m;
    sum += m;
  }
  const float total = (float)wave_sum_i(sum);
  // ceil(n / per), or one, as 1 + floor(n r): r is below 1 / per, by more than
  // the roundings here and by too little to matter
  constexpr float kBelow = 1.0f - 0x1p-20f, kAbove = 1.0f + 0x1p-20f;
  auto shares = [&](int j, float r) { return j * 64 + lane < a.B ? 1 + (int)(pages[j] * r) : 0; };
  int lo = max(a.min_pages, (int)(total * __builtin_amdgcn_rcpf((float)a.slots)));
  int hi = max(lo, (int)(total * __builtin_amdgcn_rcpf((float)(a.slots - (int)a.B)) * kAbove) + 1);
  while (hi - lo > hi / 16) {
    const int mid = (lo + hi) / 2;
    const float r = __builtin_amdgcn_rcpf((float)mid) * kBelow;
    int count = 0;
#pragma unroll
    for (int j = 0; j < kShareLanes; ++j)
      if (j * 64 < a.B) count += shares(j, r);
    if (wave_sum_i(count) <= a.slots) hi = mid;
    else lo = mid + 1;
  }
  const float r = __builtin_amdgcn_rcpf((float)hi) * kBelow;
  int before = 0;                        // slots of the sequences before these 64
#pragma unroll
  for (int j = 0; j < kShareLanes; ++j)
    if (j * 64 < a.B) {
      const int mine = shares(j, r);
      int to = mine;                     // slots up to and with this lane's
      to += dpp_i<kRowShr1>(0, to);
      to += dpp_i<kRowShr2>(0, to);
      to += dpp_i<kRowShr4>(0, to);
      to += dpp_i<kRowShr8>(0, to);
      to += dpp_i<kRowBcast15, 0xA>(0, to);
      to += dpp_i<kRowBcast31, 0xC>(0, to);
      const int at = slot - before;
      const uint64_t in = __builtin_amdgcn_ballot_w64(at >= to - mine && at < to);
      if (in != 0) {
        const int i = __builtin_ctzll(in), n = __builtin_amdgcn_readlane(mine, i);
        return {__builtin_amdgcn_readfirstlane(j * 64 + i),
                at - (__builtin_amdgcn_readlane(to, i) - n), n, __builtin_amdgcn_readlane(len[j], i)};
      }
      before += __builtin_amdgcn_readlane(to, 63);
    }
  return {-1, 0, 1, 0};
}

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
  r.l = (int)divide((uint32_t)cc, a.by_group);
  r.g = cc - r.l * a.G;
  r.on = c < a.ncols && r.l < q_len;
  r.lim = r.on ? n : 0;
  if (a.block_len > 0) {
    // a position past 2^31 - 1 lies behind every token, as that does
    const uint32_t start = a.q_start ? (uint32_t)max(a.q_start[b], 0) : 0u;
    const uint32_t pos = min(start + (uint32_t)r.l, 0x7fffffffu);
    const uint64_t end = (uint64_t)(divide(pos, a.by_block) + 1u) * a.block_len;
    r.lim = (int)min((uint64_t)r.lim, end);
  }
  return r;
}

// The column's query row (channel 0).
__device__ __forceinline__ const uint16_t *query_row(const AttnArgs &a, int64_t b, int hkv,
                                                     const Column &col) {
  return a.q + b * a.qs[0] + (int64_t)hkv * a.G * a.qs[2] +
         ((int64_t)col.l * (int32_t)a.qs[1] + (int64_t)col.g * (int32_t)a.qs[2]);
}
// Its place in a (B, q_heads, L) array.
__device__ __forceinline__ int64_t lse_at(const AttnArgs &a, int64_t b, int hkv, const Column &col) {
  return (b * a.H + hkv) * a.G * a.L + (col.g * a.L + col.l);
}

// Pieces s0 .. s0 + N - 1 of the column's query: piece s of half h holds
// channels 32 (s / 2) + 16 h + 8 (s % 2) .. + 7, as the keys' pieces do.  A
// column that is no real query reads some query's row (in bounds) and is
// dropped later: columns do not mix.
template <int N>
__device__ __forceinline__ void load_query(const AttnArgs &a, const uint16_t *row, int s0,
                                           bf16x8 (&q)[N]) {
  const int h = (threadIdx.x & 63) >> 5;
  if (a.vec) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      q[i] = *reinterpret_cast<const bf16x8 *>(row + 32 * ((s0 + i) / 2) + 16 * h + 8 * ((s0 + i) % 2));
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint16_t *x = row + 32 * ((s0 + i) / 2) + 16 * h + 8 * ((s0 + i) % 2);
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = (uint32_t)x[2 * e] | (uint32_t)x[2 * e + 1] << 16;
    q[i] = __builtin_bit_cast(bf16x8, w);
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
  float m, l;           // reference (an integer, -inf: nothing met); biased sum over this half
};

// S^T of one page: tokens x columns, in the keys' own unit.
template <int D>
__device__ __forceinline__ f32x16 score_page(const u32x4 (&kw)[D / 32], float ks,
                                             const bf16x8 (&q)[D / 16]) {
  f32x16 s;
#pragma unroll
  for (int r = 0; r < 16; ++r) s[r] = 0.f;
#pragma unroll
  for (int st = 0; st < D / 16; ++st) {
    const bf16x8 k = decode_bf16(kw[st / 2][2 * (st % 2)], kw[st / 2][2 * (st % 2) + 1], ks);
    s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, q[st], s, 0, 0, 0);
  }
  return s;
}

// The reference after a page's scores s with value exponent e, the accumulators
// rescaled where it rose; returns what the scores' exponents subtract.
template <int D>
__device__ __forceinline__ float raise(float c, int e, const f32x16 &s, Tile<D> &tile) {
  float mx = s[0];
#pragma unroll
  for (int r = 1; r < 16; ++r) mx = fmaxf(mx, s[r]);
  mx = fmaf(halves_max(mx), c, (float)e);
  const bool rise = mx > tile.m + kRise;
  if (__builtin_amdgcn_ballot_w64(rise) != 0) {
    // (-inf) - (-inf) never arises: mx is above -inf where it rose
    const float m = __builtin_rintf(mx);
    const float f = rise ? __builtin_amdgcn_exp2f(tile.m - m) : 1.0f;
    tile.l *= f;
#pragma unroll
    for (int cc = 0; cc < D / 32; ++cc) tile.o[cc] *= f;
    tile.m = rise ? m : tile.m;
  }
  // a column that has met no token yet has m = -inf: weights 0
  return tile.m == kNegInf ? 0.f : tile.m - (kBias + (float)e);
}

// log of the sum of exponentials, from the reference and the biased sum: the
// sum's binary exponent joins the integers.  -inf for a column that met nothing.
__device__ __forceinline__ float log_sum(float m, float l) {
  if (!(l > 0.f)) return m + l;
  const int e = (int)(__float_as_uint(l) >> 23) - 127;
  return ((m - kBias + (float)e) + __builtin_amdgcn_logf(__builtin_amdgcn_ldexpf(l, -e))) * kLn2;
}

template <int D>
__device__ __forceinline__ void accumulate(const u32x4 (&vw)[D / 32], const f16x8 (&p)[2], Tile<D> &tile) {
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      tile.o[c] = __builtin_amdgcn_mfma_f32_32x32x16_f16(decode_f16(vw[c][2 * e], vw[c][2 * e + 1]), p[e],
                                                         tile.o[c], 0, 0, 0);
}

// Columns' results: the output itself (whole: the sequence has one share), or
// this share's part.
template <int D>
__device__ __forceinline__ void store_tile(const AttnArgs &a, int64_t b, int hkv, int64_t c, int slot,
                                           bool whole,
                                           const Column &col, const Tile<D> &t) {
  const int h = (threadIdx.x & 63) >> 5;
  const float l = halves_sum(t.l);
  if (!col.on) return;
  if (whole) {
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
          y[e] = __builtin_bit_cast(uint16_t, (__bf16)(t.o[cc][4 * g + e] * inv));
        const int d = 32 * cc + 8 * g + 4 * h;
        if (a.out_vec) {
          *reinterpret_cast<uint2 *>(o + d) = __builtin_bit_cast(uint2, y);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) o[d + e] = y[e];
        }
      }
    if (h == 0)
      a.lse[lse_at(a, b, hkv, col)] = log_sum(t.m, l);
    return;
  }
  const int64_t row = ((int64_t)slot * a.H + hkv) * a.ncols + c;
  float *po = a.part_o + row * D;
#pragma unroll
  for (int cc = 0; cc < D / 32; ++cc)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      f32x4 y;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = t.o[cc][4 * g + e];
      *reinterpret_cast<f32x4 *>(po + 32 * cc + 8 * g + 4 * h) = y;
    }
  if (h == 0) {
    a.part_ml[2 * row] = t.m;
    a.part_ml[2 * row + 1] = l;
  }
}

// One unit: key/value head, column group (32 CW columns), share of a sequence's
// tokens.
//
// Few columns (one query per sequence): bound by reading the cache, 420 MB of 8
// sequences in 80 us, 5.2 TB/s.  Many: bound by issue.  A wave spends 1490
// cycles of its SIMD on a page and 32 columns.  16 matrix instructions are 590
// of them, each of which keeps the vector unit from about 15 cycles of other
// work; 150 vector instructions, among them the decoding's 64 conversions of
// 4.5 cycles and 17 exponentials of 8.5, are the rest.  8192 queries of 32 heads
// under the mask of blocks of 32 take 700 us, 790 TFLOP/s.  Hence the order
// inside page_step, the decoding straight into operands and few rescalings.  Two
// column tiles a wave share the decoding but need 458 registers, one wave a
// SIMD, and lose the overlap of two (2061 us).  Scores on 8-bit matrix
// instructions, the query split into two codes, took a fifth off the time and
// were off by 2^-16 of sum|q k|: not taken.
template <int D, int CW, int KW>
__global__ __launch_bounds__(64 * CW * KW, D <= 128 ? 2 : 1) void attention_kernel(AttnArgs a) {
  constexpr int REGS = D / 2;                      // accumulator registers of a tile
  constexpr int SLOTS = KW / 2 * CW;               // tiles handed over in one step
  __shared__ float s_o[KW > 1 ? SLOTS * REGS * 64 : 1];
  __shared__ float s_ml[KW > 1 ? SLOTS * 2 * 64 : 1];
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cw = wave % CW, kw_id = wave / CW;
  uint32_t unit = blockIdx.x;
  if (a.groups > 1) {
    // Workgroups go round robin to the 8 XCDs: give each XCD a run of units, so
    // that the column groups of one head read its pages from one L2; longest
    // column groups first (under the block mask later queries see more).
    const uint32_t n8 = gridDim.x / 8, rest = gridDim.x % 8, x = unit % 8;
    unit = x * n8 + min(x, rest) + unit / 8;
  }
  const int group = a.groups - 1 - (int)(unit % (uint32_t)a.groups);
  unit /= (uint32_t)a.groups;
  const int hkv = (int)(unit % (uint32_t)a.H);
  const int slot = (int)(unit / (uint32_t)a.H);
  Share share = {slot, 0, 1, 0};
  if (a.slots == a.B) {
    share.len = a.kv_lens[slot];
  } else {
    share = share_of(a, slot);
    if (share.b < 0) return;
  }
  const int64_t b = share.b;
  if (a.slots != a.B && share.split == 0 && hkv == 0 && group == 0 && threadIdx.x == 0)
    a.part_of[b] = make_int2(slot, share.splits);
  const int64_t c0 = ((int64_t)group * CW + cw) * 32;
  const int n = (int)cut_len(share.len, a.max_pages);
  const int64_t q_len = a.q_lens ? min((int64_t)a.q_lens[b], (int64_t)a.L) : a.L;

  const Column col = column(a, b, c0 + (lane & 31), n, q_len);
  bf16x8 q[D / 16];
  load_query(a, query_row(a, b, hkv, col), 0, q);
  const int max_lim = -wave_min_i(-col.lim);
  const int min_lim = wave_min_i(col.lim);
  Tile<D> tile;
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
#pragma unroll
    for (int r = 0; r < 16; ++r) tile.o[c][r] = 0.f;
  tile.m = kNegInf;
  tile.l = 0.f;
  const int pages = (max_lim + kPage - 1) / kPage;
  const int per = (pages + share.splits - 1) / share.splits;
  const int lo = share.split * per, hi = min(lo + per, pages);
  const int32_t *row = a.table + b * a.table_stride;
  // This wave's pages are lo + kw_id + KW i.  Lane j of the directory knows page
  // i = 64 c + j of the current run of 64: no scalar load, with its wait for
  // everything before it, stands between two pages.
  int dir_at = -1, dir_ke = 0, dir_ve = 0;
  int64_t dir_ph = 0;
  const int count = (hi - lo - kw_id + KW - 1) / KW;
  auto directory = [&](int i) {
    const int t = lo + kw_id + (i + lane) * KW;
    const int64_t id = i + lane < count ? page_of(row, t, a.num_pages) : -1;
    dir_at = id < 0 ? -1 : t;
    dir_ph = max(id, (int64_t)0) * a.H + hkv;         // a missing page reads page 0, unused
    dir_ke = stored_exp(a.k_scale[dir_ph]);
    dir_ve = stored_exp(a.v_scale[dir_ph]);
    __builtin_amdgcn_s_waitcnt(0);
  };
  // Two page buffers in turn, fetched again when their page is done.  Loads are unconditional, past the end
  // they read page 0 or the last one again: a branch around them would make
  // every wait one for all loads.
  constexpr int NB = D == 256 ? 1 : 2;                // registers allow one at head_dim 256
  u32x4 kw[NB][D / 32], vw[NB][D / 32];
  int at[NB], ke[NB], ve[NB];                         // the buffers' pages (-1: none) and scales
  int64_t ph[NB];
  auto locate = [&](int x, int i) {
    if ((i & 63) == 0) directory(i);
    at[x] = __builtin_amdgcn_readlane(dir_at, i & 63);
    ke[x] = __builtin_amdgcn_readlane(dir_ke, i & 63);
    ve[x] = __builtin_amdgcn_readlane(dir_ve, i & 63);
    ph[x] = (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)dir_ph, i & 63) |
            (int64_t)__builtin_amdgcn_readlane((int)(dir_ph >> 32), i & 63) << 32;
  };
  // The page in buffer x, whose scores are in s; leaves the next page's there.
  // Each matrix instruction of the next page's scores has two of this page's
  // weights and its own operand's decoding beside it; the order is fixed, since
  // the scheduler's own (all the decoding first) needs more registers.
  auto page_step = [&](int x, int i, f32x16 &s) {
    const int here = at[x], e_page = ve[x], y = (x + 1) % NB;
    const int t0 = here * kPage;
    if (here >= 0) {
      if (t0 + kPage > n) {
        // the cache ends inside this page: what lies behind may be any bits,
        // and 0 * NaN is NaN, so the values there become 0
        const int live = n - t0 - 4 * h;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int m = min(max(live - 8 * g, 0), 4);
          const uint32_t keep = m == 4 ? ~0u : (1u << (8 * m)) - 1u;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) vw[x][c][g] &= keep;
        }
      }
      if (t0 + kPage > min_lim) {
        const int left = col.lim - t0 - 4 * h;
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (8 * (r / 4) + r % 4 >= left) s[r] = kNegInf;
      }
    } else {
      // no page: weights 0, and values 0 (page 0's may be any bits)
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = kNegInf;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) vw[x][c] = u32x4{0, 0, 0, 0};
    }
    const int e_in = max(e_page, kMinExp);
    const float sub = raise<D>(a.c, e_in, s, tile);
    f32x16 next;
    f16x8 p[2];
    float l = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) next[r] = 0.f;
    constexpr int RS = 256 / D;                       // weights beside one matrix instruction
#pragma unroll
    for (int st = 0; st < D / 16; ++st) {
      if constexpr (NB == 2) {
        const bf16x8 k = decode_bf16(kw[y][st / 2][2 * (st % 2)], kw[y][st / 2][2 * (st % 2) + 1], pow2(ke[y]));
        next = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, q[st], next, 0, 0, 0);
      }
#pragma unroll
      for (int r = st * RS; r < (st + 1) * RS; ++r) {
        float w = __builtin_amdgcn_exp2f(fmaf(s[r], a.c, -sub));
        l += w;
        p[r / 8][r % 8] = (_Float16)w;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    tile.l = fmaf(l, pow2(-e_in), tile.l);
    if (e_page < kMinExp) {
      const _Float16 f = (_Float16)__builtin_amdgcn_ldexpf(1.0f, e_page - kMinExp);
#pragma unroll
      for (int e = 0; e < 2; ++e) p[e] *= f;
    }
    accumulate<D>(vw[x], p, tile);
    __builtin_amdgcn_sched_barrier(0);
    // buffer x is free: its next page
    locate(x, i + NB);
    load_pieces<D>(a.k, ph[x], kw[x]);
    __builtin_amdgcn_sched_barrier(0);
    load_pieces<D>(a.v, ph[x], vw[x]);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (NB == 2) s = next;
    else s = score_page<D>(kw[x], pow2(ke[x]), q);
  };
  if (count > 0) {
#pragma unroll
    for (int x = 0; x < NB; ++x) {
      locate(x, x);
      load_pieces<D>(a.k, ph[x], kw[x]);
      __builtin_amdgcn_sched_barrier(0);
      load_pieces<D>(a.v, ph[x], vw[x]);
      __builtin_amdgcn_sched_barrier(0);
    }
    f32x16 s = score_page<D>(kw[0], pow2(ke[0]), q);
    for (int i = 0; i < count; i += NB) {
#pragma unroll
      for (int x = 0; x < NB; ++x) page_step(x, i + x, s);
    }
  }
  if constexpr (KW > 1) {
    // the upper half of the token waves into the lower, again and again: every
    // lane its own column's rows
#pragma unroll
    for (int step = KW / 2; step >= 1; step >>= 1) {
      __syncthreads();
      if (kw_id >= step && kw_id < 2 * step) {
        const int slot = (kw_id - step) * CW + cw;
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
#pragma unroll
          for (int r = 0; r < 16; ++r) s_o[(slot * REGS + c * 16 + r) * 64 + lane] = tile.o[c][r];
        s_ml[(slot * 2 + 0) * 64 + lane] = tile.m;
        s_ml[(slot * 2 + 1) * 64 + lane] = tile.l;
      }
      __syncthreads();
      if (kw_id < step) {
        const int slot = kw_id * CW + cw;
        const float om = s_ml[(slot * 2 + 0) * 64 + lane], ol = s_ml[(slot * 2 + 1) * 64 + lane];
        const float m1 = fmaxf(tile.m, om);
        const float fa = tile.m == kNegInf ? 0.f : __builtin_amdgcn_exp2f(tile.m - m1);
        const float fb = om == kNegInf ? 0.f : __builtin_amdgcn_exp2f(om - m1);
        tile.l = tile.l * fa + ol * fb;
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            tile.o[c][r] = tile.o[c][r] * fa + s_o[(slot * REGS + c * 16 + r) * 64 + lane] * fb;
        tile.m = m1;
      }
    }
    if (kw_id != 0) return;
  }
  store_tile<D>(a, b, hkv, c0 + (lane & 31), slot, share.splits == 1, col, tile);
}

// One wave per query and head: joins the shares' parts in their order.  Bound by
// reading them: 5.3 us for 3584 rows of 128 channels in about 8 parts each
// (15 MB), 4.7 us for 256 rows.
template <int D>
__global__ __launch_bounds__(kJoinThreads) void attention_join_kernel(AttnArgs a) {
  constexpr int PER = D / 64;
  const int lane = threadIdx.x & 63;
  // a call with shares has B <= 256 and few columns: rows fit 32 bits
  const uint32_t row = __builtin_amdgcn_readfirstlane(blockIdx.x * kJoinWaves + (threadIdx.x >> 6));
  if (row >= (uint32_t)a.B * a.H * a.ncols) return;
  const uint32_t bh = row / (uint32_t)a.ncols;
  const int c = (int)(row - bh * (uint32_t)a.ncols);
  const int64_t b = bh / (uint32_t)a.H;
  const int hkv = (int)(bh - (uint32_t)b * a.H);
  const int l = (int)divide((uint32_t)c, a.by_group), g = c - l * a.G;
  const int64_t q_len = a.q_lens ? min((int64_t)a.q_lens[b], (int64_t)a.L) : a.L;
  if (l >= q_len) return;
  const int2 of = a.part_of[b];
  if (of.y == 1) return;                                  // written already
  const int64_t step = (int64_t)a.H * a.ncols, first = of.x * step + hkv * (int64_t)a.ncols + c;
  const float *ml = a.part_ml + first * 2;
  float m = kNegInf;
  for (int s = lane; s < of.y; s += 64) m = fmaxf(m, ml[s * step * 2]);
  m = wave_max(m);
  const float *po = a.part_o + first * D + lane * PER;
  float acc[PER], sum = 0.f;
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int s = 0; s < of.y; ++s) {
    const float ms = ml[s * step * 2];
    const float f = ms == kNegInf ? 0.f : __builtin_amdgcn_exp2f(ms - m);
    sum = fmaf(ml[s * step * 2 + 1], f, sum);
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = fmaf(po[s * step * D + e], f, acc[e]);
  }
  const float inv = sum > 0.f ? 1.0f / sum : (sum == sum ? 0.f : sum);
  const int64_t head = (int64_t)hkv * a.G + g;
  uint16_t *o = a.out + b * a.os[0] + l * a.os[1] + head * a.os[2] + lane * PER;
#pragma unroll
  for (int e = 0; e < PER; ++e) o[e] = __builtin_bit_cast(uint16_t, (__bf16)(acc[e] * inv));
  if (lane == 0)
    a.lse[(b * a.H * a.G + head) * a.L + l] =
        log_sum(m, sum);
}

// Attention weights.  A wave holds the keys of two pages (64 tokens), decoded,
// and walks the columns of its head: per 32 columns it recomputes S^T and adds
// 2^(s - lse) into one register per token of its lane's columns.  The four
// waves of a workgroup take neighbouring tokens and the same columns.  A
// workgroup's columns are one part (a share of a head's columns); lanes are
// folded at its end, and a second kernel adds the parts of each token in order
// (no atomics: the result does not depend on which workgroup is first).
//
// Bound by issue as the attention is: 16 matrix instructions per 64 tokens and
// 32 columns, and three vector instructions for each of the 32 weights a lane
// has of them.  8192 queries of 32 heads: 355 us, 780 TFLOP/s; one page a wave
// with the queries read by every wave took 3660.
constexpr int kWeightPages = 2;
constexpr int kWeightTokens = kPage * kWeightPages * 4;     // of a workgroup

template <int D>
__global__ __launch_bounds__(256, D <= 128 ? 2 : 1) void attention_weights_kernel(AttnArgs a) {
  constexpr int P = kWeightPages;
  __shared__ float s_w[4][16][65];
  __shared__ bf16x8 s_q[2][D / 16][64];
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t unit = blockIdx.x;
  const int part = (int)(unit % (uint32_t)a.parts);
  unit /= (uint32_t)a.parts;
  const int tg = (int)(unit % (uint32_t)a.token_groups);
  const int64_t b = unit / (uint32_t)a.token_groups;
  const int hkv = part % a.H, share = part / a.H;
  const int n = (int)cut_len(a.kv_lens[b], a.max_pages);
  const int t0 = tg * kWeightTokens + wave * (kPage * P);
  if (tg * kWeightTokens >= n) return;                      // workgroup-uniform
  const int64_t q_len = a.q_lens ? min((int64_t)a.q_lens[b], (int64_t)a.L) : a.L;
  const int32_t *row = a.table + b * a.table_stride;
  // this part's column tiles, from the first query that sees the workgroup's
  // first token to the last real one
  const int tiles = (a.ncols + 31) / 32, per = (tiles + a.shares - 1) / a.shares;
  int u0 = share * per;
  const int64_t cols = max(q_len, (int64_t)0) * a.G;
  const int u1 = (int)min((int64_t)min(u0 + per, tiles), (cols + 31) / 32);
  if (a.block_len > 0) {
    const uint32_t s = a.q_start ? (uint32_t)max(a.q_start[b], 0) : 0u;
    const uint32_t from = (uint32_t)(tg * kWeightTokens) / a.block_len * a.block_len;
    if (from > s) u0 = (int)max((int64_t)u0, (int64_t)(from - s) * a.G / 32);
  }

  bf16x8 k[P][D / 16];
  int end[P];                                               // tokens of page p that count
  float w[P][16];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int t = t0 / kPage + p;
    const int64_t id = t0 + p * kPage < n ? page_of(row, t, a.num_pages) : -1;
    end[p] = id < 0 ? 0 : n;
    const int64_t ph = max(id, (int64_t)0) * a.H + hkv;
    u32x4 kw[D / 32];
    load_pieces<D>(a.k, ph, kw);
    const float ks = pow2(stored_exp(a.k_scale[ph]));
#pragma unroll
    for (int st = 0; st < D / 16; ++st)
      k[p][st] = decode_bf16(kw[st / 2][2 * (st % 2)], kw[st / 2][2 * (st % 2) + 1], ks);
#pragma unroll
    for (int r = 0; r < 16; ++r) w[p][r] = 0.f;
  }
  // The four waves share the tiles' queries through LDS, each fetching a
  // quarter of the next tile's while one is worked on, and the scores of one
  // tile become weights while the matrix instructions compute the next one's.
  struct Cols { float z; int lim; };                        // a tile's lse and limits, as loaded
  constexpr int QW = D / 64;                                // pieces a wave fetches
  bf16x8 part_q[QW];
  auto fetch = [&](int u, Cols &x) {
    const Column col = column(a, b, (int64_t)min(u, u1 - 1) * 32 + (lane & 31), n, q_len);
    x.z = a.lse[lse_at(a, b, hkv, col)];
    x.lim = col.lim;
    load_query(a, query_row(a, b, hkv, col), wave * QW, part_q);
  };
  auto publish = [&](int u) {
#pragma unroll
    for (int i = 0; i < QW; ++i) s_q[u & 1][wave * QW + i][lane] = part_q[i];
  };
  f32x16 s[P];                                              // the scores of the tile in work
  // Tile u, whose columns are x and scores s: its weights, and the next tile's
  // scores; part_q holds that one's queries, and takes those of tile u + 2.
  auto step = [&](int u, Cols &x) {
    publish(u + 1);
    __syncthreads();
    // met nothing, a query of NaN or infinities, or no query at all (whose lse may
    // be any bits): adds nothing
    const bool none = !bits_finite(__float_as_uint(x.z)) || x.lim == 0;
    const float sub = none ? 0.f : x.z * kLog2e;
    const int lim = none ? 0 : x.lim;
    fetch(u + 2, x);
    bf16x8 q[D / 16];
#pragma unroll
    for (int st = 0; st < D / 16; ++st) q[st] = s_q[(u + 1) & 1][st][lane];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int left = min(lim, end[p]) - t0 - p * kPage;
      if (__builtin_amdgcn_ballot_w64(left < kPage) != 0) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (8 * (r / 4) + r % 4 >= left - 4 * h) s[p][r] = kNegInf;
      }
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
      f32x16 next;
#pragma unroll
      for (int r = 0; r < 16; ++r) next[r] = 0.f;
#pragma unroll
      for (int st = 0; st < D / 16; ++st) {
        next = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[p][st], q[st], next, 0, 0, 0);
#pragma unroll
        for (int r = st * (256 / D); r < (st + 1) * (256 / D); ++r)
          w[p][r] += __builtin_amdgcn_exp2f(fmaf(s[p][r], a.c, -sub));
        __builtin_amdgcn_sched_barrier(0);
      }
      s[p] = next;
    }
  };
  if (u0 < u1) {
    Cols xa, xb;
    fetch(u0, xa);
    publish(u0);
    __syncthreads();
    fetch(u0 + 1, xb);
#pragma unroll
    for (int p = 0; p < P; ++p) {
#pragma unroll
      for (int r = 0; r < 16; ++r) s[p][r] = 0.f;
#pragma unroll
      for (int st = 0; st < D / 16; ++st)
        s[p] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[p][st], s_q[u0 & 1][st][lane], s[p], 0, 0, 0);
    }
    // the last step's next tile is the last tile again, dropped
    for (int u = u0; u < u1; u += 2) {
      step(u, xa);
      if (u + 1 < u1) step(u + 1, xb);
    }
  }
  // fold the 32 columns of each half: lane (token, column half) of a page sums 16
#pragma unroll
  for (int p = 0; p < P; ++p) {
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 16; ++r) s_w[wave][r][lane] = w[p][r];
    __syncthreads();
    const int tok = lane >> 1, r = tok / 8 * 4 + tok % 4, half = tok / 4 % 2;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum += s_w[wave][r][half * 32 + (lane & 1) * 16 + i];
    sum += __shfl_xor(sum, 1);
    const int t = t0 + p * kPage + tok;
    if ((lane & 1) == 0 && t < n)
      a.part_w[((int64_t)part * a.B + b) * (a.max_pages * kPage) + t] = end[p] ? sum : 0.f;
  }
}

// 4.9 us for 8192 tokens in 32 parts.
__global__ __launch_bounds__(kJoinThreads) void attention_weights_join_kernel(AttnArgs a) {
  const int64_t T = a.max_pages * kPage;
  const int64_t blocks = (T + kJoinThreads - 1) / kJoinThreads;
  const int64_t b = blockIdx.x / (uint32_t)blocks;
  const int64_t t = (int64_t)(blockIdx.x % (uint32_t)blocks) * kJoinThreads + threadIdx.x;
  if (t >= cut_len(a.kv_lens[b], a.max_pages)) return;
  const float *p = a.part_w + b * T + t;
  float sum = 0.f;
#pragma unroll 8
  for (int i = 0; i < a.parts; ++i) sum += p[(int64_t)i * a.B * T];
  a.weights[b * T + t] += sum;
}

// ---------------------------------------------------------------- host side

struct AttnPlan {
  int cw, kw;      // column waves, token waves
  int groups, slots, min_pages;
};

// 8 waves a workgroup (2 a SIMD at up to 256 registers; head_dim 256 needs 512,
// 4 waves): as many column waves as there are column tiles, up to 4, the others
// along the tokens.  Where the column groups alone give every CU two
// workgroups, 4 column waves and no token waves.
AttnPlan attn_plan(int64_t B, int64_t ncols, int64_t H, int64_t D, int64_t max_pages) {
  const int64_t cus = device_cu_count(), tiles = std::max<int64_t>(1, (ncols + 31) / 32);
  AttnPlan p;
  p.cw = tiles > 2 ? 4 : (int)tiles;
  if (D == 256) p.cw = tiles > 1 ? 4 : 1;
  p.groups = (int)((tiles + p.cw - 1) / p.cw);
  const int64_t units = std::max<int64_t>(1, B * H * p.groups);
  p.kw = (D == 256 ? 4 : 8) / p.cw;
  if (p.cw == 4 && units >= 2 * cus) p.kw = 1;
  // Split the tokens until every CU has its workgroup, with 2 pages or more per
  // token wave and 4 or more per share, where a sequence may have 3 shares:
  // 2 save less than the second kernel costs (one sequence of 8 heads and 1000
  // tokens: 13.0 us in 2 shares, 12.3 in one; 2000 tokens: 15.2 in 3, 17.0 in
  // one).  Where the sequences come near to that number or reach it without, as
  // many shares more, for the long ones among them, if one may have 4: 64
  // sequences of 8 heads, one of 32768 tokens and the others of 500, take 48 us
  // and not 147; batches of equal ones lose 5 us (64 of 2000: 57, 64 of 500: 29).
  p.min_pages = std::max(2 * p.kw, 4);
  const int64_t each = cus / (H * p.groups), most = max_pages / p.min_pages;
  int64_t s = B;
  if (each >= 2 * B && most >= 3) s = std::min(each, B * most);
  else if (each >= 1 && most >= 4) s = B + each;
  p.slots = (int)(B > 64 * kShareLanes ? B : std::min(s, B + 127));
  return p;
}

size_t attn_workspace(const AttnPlan &p, int64_t B, int64_t cols, int64_t D) {
  return p.slots == B ? 0 : (size_t)p.slots * cols * (D + 2) * 4 + (size_t)B * sizeof(int2);
}

// Sizes that the calls accept, and whose products fit 64 bits.
bool sane_sizes(int64_t B, int64_t L, int64_t q_heads, int64_t kv_heads, int64_t max_pages) {
  return B >= 0 && L >= 0 && q_heads >= 1 && q_heads <= 0x7fffffLL && kv_heads >= 1 &&
         kv_heads <= 4096 && q_heads % kv_heads == 0 && max_pages >= 0 &&
         max_pages <= 0x7fffffffLL / kPage && B <= 0x7fffffffLL && L <= 0x7fffff00LL / q_heads &&
         (B == 0 || L * q_heads <= (1LL << 40) / B);
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
  if (!(scale > 0.0f) || !(scale <= 0x1p127f))
    return fail(DLLM_ERR_ARG, "%s: scale must be > 0 and at most 2^127", who);
  if (B == 0 || L == 0) return DLLM_OK;
  if (!q || !q_strides || !kv_lens)
    return fail(DLLM_ERR_ARG, "%s: q, q_strides and kv_lens must be non-NULL", who);
  if ((uintptr_t)q % 2 != 0) return fail(DLLM_ERR_ARG, "%s: q must be aligned to its element", who);
  for (int i = 1; i < 3; ++i)
    if (q_strides[i] != (int32_t)q_strides[i])
      return fail(DLLM_ERR_UNSUPPORTED, "%s: q's strides along L and heads must fit 32 bits", who);
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
  a.block_len = (uint32_t)block_len;
  a.by_group = divisor((uint32_t)(q_heads / c.kv_heads));
  a.by_block = divisor(block_len > 0 ? (uint32_t)block_len : 1u);
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
  if constexpr (D == 256) {
    if (p.cw == 4) hipLaunchKernelGGL((attention_kernel<D, 4, 1>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((attention_kernel<D, 1, 4>), grid, dim3(256), 0, s, a);
  } else {
    if (p.cw == 4 && p.kw == 1)
      hipLaunchKernelGGL((attention_kernel<D, 4, 1>), grid, dim3(256), 0, s, a);
    else if (p.cw == 4) hipLaunchKernelGGL((attention_kernel<D, 4, 2>), grid, dim3(512), 0, s, a);
    else if (p.cw == 2) hipLaunchKernelGGL((attention_kernel<D, 2, 4>), grid, dim3(512), 0, s, a);
    else hipLaunchKernelGGL((attention_kernel<D, 1, 8>), grid, dim3(512), 0, s, a);
  }
}

// Parts of the attention weights: per key/value head, and shares of its columns
// while that gives every CU four workgroups, of 4 or more column tiles.
struct WeightPlan { int64_t token_groups; int shares; int64_t parts; };

WeightPlan weight_plan(int64_t B, int64_t ncols, int64_t H, int64_t max_pages) {
  WeightPlan p;
  p.token_groups = (max_pages * kPage + kWeightTokens - 1) / kWeightTokens;
  const int64_t tiles = std::max<int64_t>(1, (ncols + 31) / 32);
  const int64_t units = std::max<int64_t>(1, B * H * p.token_groups);
  int64_t s = (4LL * device_cu_count() + units - 1) / units;
  s = std::min<int64_t>(s, tiles / 4);
  p.shares = (int)std::max<int64_t>(1, s);
  p.parts = H * p.shares;
  return p;
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" size_t dllm_block_attention_workspace_size(int64_t B, int64_t L, int64_t q_heads,
                                                      int64_t kv_heads, int64_t head_dim,
                                                      int64_t max_pages) {
  if (!sane_sizes(B, L, q_heads, kv_heads, max_pages) ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return 0;
  const AttnPlan p = attn_plan(B, L * (q_heads / kv_heads), kv_heads, head_dim, max_pages);
  return attn_workspace(p, B, L * q_heads, head_dim);
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
  const size_t need = attn_workspace(p, B, L * q_heads, D);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(DLLM_ERR_SHAPE, "%s: workspace has %zu bytes, needs %zu", who, workspace_bytes, need);
  if (need > 0 && (uintptr_t)workspace % 16 != 0)
    return fail(DLLM_ERR_ARG, "%s: workspace must be 16-byte aligned", who);
  const int64_t wgs = (int64_t)p.slots * a.H * p.groups;
  if (wgs > 0xffffffffLL / 512 || (rows + kJoinWaves - 1) / kJoinWaves > 0xffffffffLL / kJoinThreads)
    return fail(DLLM_ERR_UNSUPPORTED, "%s: too many queries in one call", who);
  a.out = (uint16_t *)out;
  a.out_vec = (uintptr_t)out % 8 == 0;
  for (int i = 0; i < 3; ++i) {
    a.os[i] = out_strides[i];
    if (a.os[i] % 4 != 0) a.out_vec = 0;
  }
  a.lse = lse;
  a.groups = p.groups;
  a.slots = p.slots;
  a.min_pages = p.min_pages;
  if (need > 0) {
    const int64_t part_rows = (int64_t)p.slots * L * q_heads;
    a.part_o = (float *)workspace;
    a.part_ml = a.part_o + part_rows * D;
    a.part_of = (int2 *)(a.part_ml + part_rows * 2);
  }
  const dim3 grid((uint32_t)wgs);
  if (D == 64) launch_attention<64>(p, a, grid, stream);
  else if (D == 128) launch_attention<128>(p, a, grid, stream);
  else launch_attention<256>(p, a, grid, stream);
  const int st = check_launch(who);
  if (st != DLLM_OK || p.slots == B) return st;
  const dim3 jgrid((uint32_t)((rows + kJoinWaves - 1) / kJoinWaves));
  if (D == 64)
    hipLaunchKernelGGL(attention_join_kernel<64>, jgrid, dim3(kJoinThreads), 0, stream, a);
  else if (D == 128)
    hipLaunchKernelGGL(attention_join_kernel<128>, jgrid, dim3(kJoinThreads), 0, stream, a);
  else
    hipLaunchKernelGGL(attention_join_kernel<256>, jgrid, dim3(kJoinThreads), 0, stream, a);
  return check_launch(who);
}

extern "C" size_t dllm_attention_weights_workspace_size(int64_t B, int64_t L, int64_t q_heads,
                                                        int64_t kv_heads, int64_t max_pages) {
  if (!sane_sizes(B, L, q_heads, kv_heads, max_pages)) return 0;
  const WeightPlan p = weight_plan(B, L * (q_heads / kv_heads), kv_heads, max_pages);
  return (size_t)p.parts * B * max_pages * kPage * 4;
}

extern "C" int dllm_attention_weights(const dllm_kv_cache *cache, const void *q,
                                      const int64_t *q_strides, int64_t B, int64_t L,
                                      int64_t q_heads, const int32_t *page_table,
                                      int64_t max_pages, int64_t table_stride,
                                      const int32_t *kv_lens, const int32_t *q_start,
                                      const int32_t *q_lens, int64_t block_len, float scale,
                                      const float *lse, float *weights, void *workspace,
                                      size_t workspace_bytes, hipStream_t stream) {
  const char *who = "dllm_attention_weights";
  const int rc = check_attention(who, cache, q, q_strides, B, L, q_heads, page_table, max_pages,
                                 table_stride, kv_lens, block_len, scale);
  if (rc != DLLM_OK) return rc;
  if (B == 0 || L == 0 || max_pages == 0) return ok();
  if (!lse || !weights) return fail(DLLM_ERR_ARG, "%s: lse and weights must be non-NULL", who);
  AttnArgs a = attn_args(*cache, q, q_strides, B, L, q_heads, page_table, max_pages, table_stride,
                         kv_lens, q_start, q_lens, block_len, scale);
  const WeightPlan p = weight_plan(B, a.ncols, a.H, max_pages);
  const int64_t limit = 0xffffffffLL / 256;
  if (p.parts > limit / p.token_groups || B > limit / (p.parts * p.token_groups))
    return fail(DLLM_ERR_UNSUPPORTED, "%s: too many pages in one call", who);
  const size_t need = (size_t)p.parts * B * max_pages * kPage * 4;
  if (!workspace || workspace_bytes < need)
    return fail(DLLM_ERR_SHAPE, "%s: workspace has %zu bytes, needs %zu", who, workspace_bytes, need);
  if ((uintptr_t)workspace % 16 != 0)
    return fail(DLLM_ERR_ARG, "%s: workspace must be 16-byte aligned", who);
  a.lse = const_cast<float *>(lse);
  a.weights = weights;
  a.part_w = (float *)workspace;
  a.parts = (int)p.parts;
  a.shares = p.shares;
  a.token_groups = (int)p.token_groups;
  const dim3 grid((uint32_t)(B * p.token_groups * p.parts));
  if (cache->head_dim == 64)
    hipLaunchKernelGGL(attention_weights_kernel<64>, grid, dim3(256), 0, stream, a);
  else if (cache->head_dim == 128)
    hipLaunchKernelGGL(attention_weights_kernel<128>, grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL(attention_weights_kernel<256>, grid, dim3(256), 0, stream, a);
  const int st = check_launch(who);
  if (st != DLLM_OK) return st;
  const int64_t blocks = (max_pages * kPage + kJoinThreads - 1) / kJoinThreads;
  hipLaunchKernelGGL(attention_weights_join_kernel, dim3((uint32_t)(B * blocks)),
                     dim3(kJoinThreads), 0, stream, a);
  return check_launch(who);
}
