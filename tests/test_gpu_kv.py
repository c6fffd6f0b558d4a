"""GPU parity of the 8-bit cache (write, read, gather), eviction and block
attention against the float64 oracle.

The cache is exact: codes and power-of-two scales have one right value, so
everything read back must equal the oracle's.  Attention's tolerances, with
u = 2^-24: a score is a sum of D exact products, off by at most
ds = (D + 8) u scale sum|q k| + 4 u |s|, which moves a weight by ds relative;
a weight is rounded to 11 bits before it multiplies a value (2^-11 at most)
and may be dropped below 2^-39 of the largest (2^-38 sum|v| in all); the sums
over T tokens add T u; the output is rounded to bfloat16 (2^-8)."""
import numpy as np
import pytest
import torch

import commit_step_amd as dc
from oracle import kv as okv

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
PAGE = 32


def _bf16(a):
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch.bfloat16)


def _np(t):
    return t.detach().cpu().double().numpy()


def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _kv(rng, B, L, H, D):
    size = np.exp2(rng.uniform(-6, 6, (B, L, H, 1)))
    k = _bf16(rng.normal(0, 1, (B, L, H, D)) * size)
    v = _bf16(rng.normal(0, 1, (B, L, H, D)) * np.exp2(rng.uniform(-3, 3, (B, L // PAGE + 1, H, 1)).repeat(
        PAGE, axis=1)[:, :L]))
    return k, v


def _table(rng, B, pages, extra=0, spare=3):
    perm = rng.permutation(B * (pages + extra) + spare)
    t = perm[:B * (pages + extra)].reshape(B, pages + extra).astype(np.int32)
    return t[:, :pages].copy(), t[:, pages:].copy(), len(perm)


def _same_cache(cache, ref, table, lens):
    k, v = dc.kv_read(cache, _i32(table), _i32(lens))
    rk, rv = ref.read(table, lens)
    assert np.array_equal(_np(k), rk) and np.array_equal(_np(v), rv)


@pytest.mark.parametrize("D,H", [(64, 1), (128, 3), (256, 2)])
@pytest.mark.parametrize("start,L", [(0, 1), (0, 32), (0, 100), (5, 3), (31, 2), (30, 70), (64, 33)])
def test_write_read(D, H, start, L):
    rng = np.random.default_rng(D + start + L)
    B, pages = 2, 5
    table, _, n = _table(rng, B, pages)
    cache, ref = dc.KVCache(n, H, D), okv.Cache(n, H, D)
    if start:
        k, v = _kv(rng, B, start, H, D)
        dc.kv_write(cache, k.cuda(), v.cuda(), _i32(table), _i32([0, 0]))
        ref.write(_np(k), _np(v), table, [0, 0])
    k, v = _kv(rng, B, L, H, D)
    for _ in range(2):                                # again: the block is replaced by itself
        dc.kv_write(cache, k.cuda(), v.cuda(), _i32(table), _i32([start, start]))
        ref.write(_np(k), _np(v), table, [start, start])
        _same_cache(cache, ref, table, [start + L, start + L - 1])


@pytest.mark.parametrize("D", [64, 128])
def test_write_ragged_strided_and_missing_pages(D):
    rng = np.random.default_rng(D)
    B, L, H, pages = 5, 50, 2, 4
    table, _, n = _table(rng, B, pages)
    table[3, 1] = -1                                  # no page
    table[4, 0] = n + 7                               # out of the pool
    cache, ref = dc.KVCache(n, H, D), okv.Cache(n, H, D)
    start, lens = [3, 100, -1, 20, 10], [50, 40, 50, 49, 99]      # past the table, nothing, ...
    big = _bf16(rng.normal(0, 1, (B, H, L, 2 * D + 3))).cuda()
    k = big[..., 1:1 + D].transpose(1, 2)             # off 16-byte alignment, heads before tokens
    v = big[..., D + 2:2 * D + 2].transpose(1, 2)
    wide = _i32(np.concatenate([table, table * 0 - 5], axis=1))[:, :pages]
    dc.kv_write(cache, k, v, wide, _i32(start), _i32(lens))
    ref.write(_np(k), _np(v), table, start, lens)
    for ln in ([128] * B, [40, 111, 0, 69, -4]):
        _same_cache(cache, ref, table, ln)


def test_write_special_values():
    rng = np.random.default_rng(4)
    cache, ref = dc.KVCache(3, 1, 64), okv.Cache(3, 1, 64)
    table = np.array([[1, 0, 2]], dtype=np.int32)
    x = rng.normal(0, 1, (1, 96, 1, 64)).astype(np.float32)
    x[0, 3, 0, 5], x[0, 4, 0, 6], x[0, 5, 0, 7] = np.nan, np.inf, -np.inf
    x[0, 32:64] = 0
    x[0, 64:] *= 2.0 ** -90
    x[0, 70, 0, 0] = 3e38
    k, v = _bf16(x), _bf16(-x[:, ::-1].copy())
    dc.kv_write(cache, k.cuda(), v.cuda(), _i32(table), _i32([0]))
    ref.write(_np(k), _np(v), table, [0])
    _same_cache(cache, ref, table, [96])
    assert np.isfinite(ref.read(table, [96])[0]).all()


def test_slots_behind_the_sequence_stay():
    rng = np.random.default_rng(6)
    cache = dc.KVCache(2, 1, 64)
    cache.k.copy_(torch.from_numpy(rng.integers(0, 120, cache.k.shape).astype(np.uint8)))
    cache.v.copy_(torch.from_numpy(rng.integers(0, 120, cache.v.shape).astype(np.uint8)))
    before = [t.clone() for t in (cache.k, cache.v)]
    k, v = _kv(rng, 1, 7, 1, 64)
    dc.kv_write(cache, k.cuda(), v.cuda(), _i32([[1, 0]]), _i32([0]))
    kb = lambda x: x.view(2, 1, 4, 32, 16).permute(0, 1, 3, 2, 4).reshape(2, 1, 32, 64)
    # values: (channel block, half, channel, 4 g + i) of token 8 g + 4 h + i
    vb = lambda x: x.view(2, 1, 2, 2, 32, 4, 4).permute(0, 1, 5, 3, 6, 2, 4).reshape(2, 1, 32, 64)
    for f, a, b in ((kb, cache.k, before[0]), (vb, cache.v, before[1])):
        a, b = f(a), f(b)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1, :, 7:], b[1, :, 7:])
        assert not torch.equal(a[1, :, :7], b[1, :, :7])


@pytest.mark.parametrize("D,H,T,budget,sink,recent", [
    (64, 1, 40, 17, 0, 0), (128, 2, 200, 64, 4, 32), (256, 1, 130, 100, 2, 5), (64, 2, 90, 200, 4, 4),
    (128, 1, 1500, 700, 4, 64), (64, 1, 33, 1, 1, 0)])
def test_evict(D, H, T, budget, sink, recent):
    rng = np.random.default_rng(T + budget)
    B, pages = 3, -(-T // PAGE)
    npages = -(-budget // PAGE)
    table, new, n = _table(rng, B, pages, npages)
    cache, ref = dc.KVCache(n, H, D), okv.Cache(n, H, D)
    k, v = _kv(rng, B, T, H, D)
    dc.kv_write(cache, k.cuda(), v.cuda(), _i32(table), _i32([0] * B))
    ref.write(_np(k), _np(v), table, [0] * B)
    lens = [T, T // 2, 0]
    w = np.exp(rng.normal(0, 3, (B, pages * PAGE))).astype(np.float32)
    w[0, :T // 3] = 0.5                              # ties
    kept, nl = okv.evict_select(w, lens, budget, sink, recent)
    r = dc.kv_evict(cache, _i32(table), _i32(lens), torch.from_numpy(w).cuda(), budget, _i32(new),
                    sink, recent)
    assert np.array_equal(r.kept.cpu().numpy(), kept) and np.array_equal(r.lens.cpu().numpy(), nl)
    nw = np.zeros((B, npages * PAGE), dtype=np.float32)
    for b in range(B):
        nw[b, :nl[b]] = w[b, kept[b, :nl[b]]]
    assert np.array_equal(r.weights.cpu().numpy(), nw)
    ref.gather(table, kept, nl, new)
    _same_cache(cache, ref, new, nl)
    # the rest of the last new page is zero
    k2, v2 = dc.kv_read(cache, _i32(new), _i32([npages * PAGE] * B))
    for b in range(B):
        end = -(-nl[b] // PAGE) * PAGE
        assert not k2[b, nl[b]:end].any() and not v2[b, nl[b]:end].any()


def test_gather_far_scales_and_bad_entries():
    """Pages of very different scales meet in one; entries outside the table and
    missing pages give zero tokens."""
    rng = np.random.default_rng(8)
    B, H, D = 1, 1, 64
    table, new, n = _table(rng, B, 4, 2)
    cache, ref = dc.KVCache(n, H, D), okv.Cache(n, H, D)
    x = rng.normal(0, 1, (1, 128, 1, 64)) * np.exp2(np.array([-110.0, 60, 0, -100]).repeat(32))[None, :, None, None]
    x[0, 40:64] = 0
    k, v = _bf16(x), _bf16(x[:, :, :, ::-1].copy())
    dc.kv_write(cache, k.cuda(), v.cuda(), _i32(table), _i32([0]))
    ref.write(_np(k), _np(v), table, [0])
    kept = np.array([[1, 5, 45, 46, 64, 65, 99, 127, 128, 4000] + [-1] * 30 + [3, 41, 50, 100]], dtype=np.int32)
    holes = table.copy()
    holes[0, 3] = -1
    for tb in (table, holes):
        for counts in ([44], [8], [2], [0]):
            dc.kv_gather(cache, _i32(tb), _i32(kept), _i32(counts), _i32(new))
            ref.gather(tb, kept, counts, new)
            _same_cache(cache, ref, new, [64] if counts[0] > 32 else [min(counts[0], 32)])


@pytest.mark.parametrize("T", [1, 5, 64, 1000, 5000])
def test_evict_select_values(T):
    rng = np.random.default_rng(T)
    B = 6
    w = rng.normal(0, 1, (B, T)).astype(np.float32)
    w[1] = 0.0
    w[1, ::2] = -0.0
    w[2, rng.random(T) < 0.3] = np.nan
    w[3, rng.random(T) < 0.3] = np.inf
    w[4] = np.round(w[4])
    w[5] = np.exp2(rng.integers(-140, 120, T)).astype(np.float32)
    wide = torch.from_numpy(np.concatenate([w, w[:, :1]], axis=1)).cuda()[:, :T]
    for budget in sorted({1, max(1, T // 3), max(1, T - 1), T, T + 5}):
        for sink, recent in ((0, 0), (min(2, budget), 0), (budget // 2, budget - budget // 2)):
            lens = [T, T, T, T - 1, T + 9, T]
            r = dc.evict_select(wide, _i32(lens), budget, sink, recent)
            kept, nl = okv.evict_select(w, lens, budget, sink, recent)
            assert np.array_equal(r.kept.cpu().numpy(), kept), (budget, sink, recent)
            assert np.array_equal(r.lens.cpu().numpy(), nl)


def test_evict_select_long():
    """More tokens than one workgroup holds in registers, and all weights equal."""
    rng = np.random.default_rng(1)
    T = 70001
    w = np.stack([np.exp(rng.normal(0, 3, T)), np.zeros(T)]).astype(np.float32)
    for budget in (100, 50000):
        r = dc.evict_select(torch.from_numpy(w).cuda(), _i32([T, T]), budget, 4, 64)
        kept, nl = okv.evict_select(w, [T, T], budget, 4, 64)
        assert np.array_equal(r.kept.cpu().numpy(), kept) and np.array_equal(r.lens.cpu().numpy(), nl)


@pytest.mark.parametrize("T", [300, 9000, 33000])
def test_evict_select_ranges(T):
    """Weights whose keys take wide, narrow and single ranges, at either end."""
    rng = np.random.default_rng(T + 1)
    w = np.stack([1.0 + rng.integers(0, 9, T) * 2.0 ** -23, 3e38 * rng.random(T), rng.random(T) * 1e-44,
                  np.where(rng.random(T) < 0.01, np.inf, 2.5), np.where(rng.random(T) < 0.5, -np.inf, np.nan),
                  np.where(np.arange(T) < 3, np.inf, rng.random(T) ** 8), np.full(T, np.inf),
                  -rng.random(T)]).astype(np.float32)
    for budget in (7, T // 4, T - 2):
        for sink, recent in ((0, 0), (4, 3), (budget // 2, budget - budget // 2)):
            r = dc.evict_select(torch.from_numpy(w).cuda(), _i32([T] * len(w)), budget, sink, recent)
            kept, nl = okv.evict_select(w, [T] * len(w), budget, sink, recent)
            assert np.array_equal(r.kept.cpu().numpy(), kept), (budget, sink, recent)
            want = np.take_along_axis(w, np.maximum(kept, 0).astype(np.int64), 1)
            assert np.array_equal(r.weights.cpu().numpy(), want, equal_nan=True)


# ---------------------------------------------------------------- attention

def _attention_case(seed, B, L, Hq, H, D, T, lens, table=None, scale_q=1.0):
    rng = np.random.default_rng(seed)
    pages = -(-T // PAGE)
    if table is None:
        table, _, n = _table(rng, B, pages)
    else:
        n = B * pages
    cache, ref = dc.KVCache(n, H, D), okv.Cache(n, H, D)
    # whatever lies behind a sequence's end may be any bits, NaN codes among them
    cache.k.fill_(0x7f)
    cache.v.fill_(0xff)
    k, v = _kv(rng, B, T, H, D)
    k = k / k.float().abs().amax(dim=(1, 3), keepdim=True).to(torch.bfloat16) * 2
    dc.kv_write(cache, k.cuda(), v.cuda(), _i32(table), _i32([0] * B), _i32(lens))
    ref.write(_np(k), _np(v), table, [0] * B, lens)
    q = _bf16(rng.normal(0, scale_q, (B, L, Hq, D)))
    return cache, ref, table, q, n


def _check_attention(cache, ref, table, q, lens, n, out=None, r=None, **kw):
    B, L, Hq, D = q.shape
    T = table.shape[1] * PAGE
    w = torch.full((B, T), 0.25, device="cuda")
    if r is None:
        opt = {a: _i32(b) if a in ("q_start", "q_lens") and b is not None else b for a, b in kw.items()}
        r = dc.block_attention(q.cuda(), cache, _i32(table), _i32(lens), weights=w, **opt)
    rk, rv = ref.read(table, lens)
    o, lse, rw, mass, mag = okv.block_attention(_np(q), rk, rv, table, lens, n, **kw)
    got, gl, gw = _np(r.out), _np(r.lse), _np(w) - 0.25
    live = np.isfinite(lse)
    assert np.array_equal(np.isfinite(gl), live) and (gl[~live] == -np.inf).all()
    s = np.where(live, np.abs(lse), 0)
    ds = (D + 8) * U * mag + 4 * U * (s + mag)
    assert (np.abs(gl[live] - lse[live]) <= (ds + T * U + 8 * U * (s + 1))[live]).all()
    dso = ds.transpose(0, 2, 1)[..., None]
    vmax = np.abs(rv).max() if rv.size else 0.0
    tol = 2.0 ** -8 * np.abs(o) + mass * (2.0 ** -11 + 2 * dso + (T + 40) * U) * 1.01 + 2.0 ** -38 * T * vmax
    err = np.abs(got - o)
    assert (err <= tol).all(), (err - tol).max()
    # a sum of L Hq weights, each off by 2 ds and the exponential's rounding
    rel = 2 * (ds.max() if ds.size else 0) + (s.max() if s.size else 0) * 4 * U + (L * Hq + 40) * U
    assert (np.abs(gw - rw) <= rw * rel + 2 * U).all(), np.abs(gw - rw).max()
    return r


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("L,Hq,H", [(1, 1, 1), (1, 4, 4), (1, 14, 2), (3, 5, 1), (32, 4, 2), (16, 7, 1), (33, 6, 2)])
@pytest.mark.parametrize("T", [1, 31, 32, 33, 500])
def test_attention_shapes(D, L, Hq, H, T):
    lens = [T, max(0, T - 7)]
    cache, ref, table, q, n = _attention_case(L + T, 2, L, Hq, H, D, T, lens)
    _check_attention(cache, ref, table, q, lens, n)


@pytest.mark.parametrize("bl", [1, 7, 32, 48])
@pytest.mark.parametrize("L,T,Hq,H", [(40, 40, 2, 1), (150, 170, 4, 4), (5, 300, 3, 3)])
def test_attention_block_causal(bl, L, T, Hq, H):
    starts = [0, T - L, 3]
    lens = [min(T, s + L) for s in starts]
    cache, ref, table, q, n = _attention_case(bl + L, 3, L, Hq, H, 64, T, lens)
    _check_attention(cache, ref, table, q, lens, n, block_len=bl, q_start=starts)
    _check_attention(cache, ref, table, q, lens, n, block_len=bl)


def test_attention_long_split_and_ragged():
    T = 6000
    for L, Hq, H, D in ((1, 8, 2, 128), (8, 4, 4, 64), (32, 8, 1, 128), (2, 2, 1, 256)):
        lens = [T, 1, 0, T // 3]
        cache, ref, table, q, n = _attention_case(T + L, 4, L, Hq, H, D, T, lens)
        qn = [L, max(1, L - 1), L, 0]
        r = _check_attention(cache, ref, table, q, lens, n, q_lens=qn)
        assert not r.out[3].any() and not r.out[1, qn[1]:].any()


@pytest.mark.parametrize("B,H,G,D,T", [(1, 1, 1, 64, 5000), (3, 2, 9, 128, 3000), (70, 1, 2, 64, 2100),
                                       (130, 1, 1, 128, 2100), (200, 1, 1, 256, 1100), (300, 1, 1, 256, 520), (600, 1, 1, 256, 300)])
@pytest.mark.parametrize("kind", ["one long", "halves", "any"])
def test_attention_lengths_of_one_batch(B, H, G, D, T, kind):
    """Sequences of one cache prefix, of lengths far apart: however the tokens
    are shared out, every sequence's result is its own."""
    rng = np.random.default_rng(B + T)
    lens = {"one long": np.full(B, 5), "halves": np.where(np.arange(B) % 2, T, T // 2),
            "any": rng.integers(0, T + 1, B)}[kind]
    if kind == "one long":
        lens[B // 2] = T
    pages = -(-T // PAGE)
    cache, ref = dc.KVCache(pages, H, D), okv.Cache(pages, H, D)
    k, v = _kv(rng, 1, T, H, D)
    one = np.arange(pages, dtype=np.int32)[::-1].copy()[None]
    dc.kv_write(cache, k.cuda(), v.cuda(), _i32(one), _i32([0]))
    ref.write(_np(k), _np(v), one, [0])
    rk, rv = (x[0, :T] for x in ref.read(one, [T]))              # (T, H, D)
    q = _bf16(rng.normal(0, 1, (B, 1, H * G, D)) * 4 / np.abs(rk).max())
    r = dc.block_attention(q.cuda(), cache, _i32(one.repeat(B, 0)), _i32(lens))
    out, lse = _np(r.out)[:, 0].reshape(B, H, G, D), _np(r.lse).reshape(B, H, G)
    qd, scale = _np(q)[:, 0].reshape(B, H, G, D), D ** -0.5
    live = np.arange(T)[None] < lens[:, None]                    # (B, T)
    for h in range(H):
        s = scale * (qd[:, h] @ rk[:, h].T)                      # (B, G, T)
        ds = (D + 8) * U * scale * (np.abs(qd[:, h]) @ np.abs(rk[:, h]).T).max() + 4 * U * np.abs(s).max()
        s = np.where(live[:, None], s, -np.inf)
        m = np.maximum(s.max(-1, keepdims=True), -1e300)
        e = np.exp(s - m)
        z = e.sum(-1, keepdims=True)
        p = e / np.maximum(z, 1e-300)
        o, mass = p @ rv[:, h], p @ np.abs(rv[:, h])
        tol = 2.0 ** -8 * np.abs(o) + mass * (2.0 ** -11 + 2 * ds + (T + 40) * U) * 1.01 \
            + 2.0 ** -38 * T * np.abs(rv).max()
        assert (np.abs(out[:, h] - o) <= tol).all(), (np.abs(out[:, h] - o) - tol).max()
        some = lens > 0
        want = (m + np.log(np.maximum(z, 1e-300)))[..., 0]
        assert (np.abs(lse[some, h] - want[some]) <= ds + (T + 40) * U + 4 * U * np.abs(want[some])).all()
        assert (lse[~some] == -np.inf).all() and not out[~some].any()


def test_attention_rows_past_q_lens_are_left():
    cache, ref, table, q, n = _attention_case(1, 2, 4, 2, 2, 64, 70, [70, 9])
    for lens in ([70, 9],):
        out = torch.full((2, 4, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((2, 2, 4), 7.0, device="cuda")
        dc.block_attention(q.cuda(), cache, _i32(table), _i32(lens), q_lens=_i32([2, 0]), out=out, lse=lse)
        assert (out[0, 2:] == 7).all() and (out[1] == 7).all() and (lse[0, :, 2:] == 7).all()
        assert (lse[1] == 7).all() and not (out[0, :2] == 7).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_padded_queries_of_any_bits_add_no_weight(D):
    """Queries past q_lens and what stands in the caller's lse there do not
    reach the weights."""
    cache, ref, table, q, n = _attention_case(3, 3, 40, 4, 2, D, 300, [300, 77, 9])
    lens, qn = _i32([300, 77, 9]), [33, 1, 0]
    want = torch.zeros((3, table.shape[1] * PAGE), device="cuda")
    dc.block_attention(q.cuda(), cache, _i32(table), lens, q_lens=_i32(qn), weights=want)
    assert torch.isfinite(want).all() and abs(float(want[0].sum()) - 33 * 4) < 1e-2 and not want[2].any()
    bad = q.cuda().clone()
    for b in range(3):
        bad[b, qn[b]:] = float("nan")
    for bits in (float("nan"), float("inf"), -3e38, 3e38):
        got = torch.zeros_like(want)
        lse = torch.full((3, 4, 40), bits, device="cuda")
        out = torch.full((3, 40, 4, D), 2.0, dtype=torch.bfloat16, device="cuda")
        dc.block_attention(bad, cache, _i32(table), lens, q_lens=_i32(qn), weights=got, lse=lse, out=out)
        assert torch.equal(got, want)


def test_attention_missing_pages_strides_and_shared_pages():
    T, L, Hq, H, D = 200, 5, 4, 2, 128
    lens = [T, T]
    cache, ref, table, q, n = _attention_case(2, 2, L, Hq, H, D, T, lens)
    holes = table.copy()
    holes[0, 2], holes[0, 6], holes[1, 0] = -1, n, 2 ** 30
    _check_attention(cache, ref, holes, q, lens, n)
    gone = holes * 0 - 1
    _check_attention(cache, ref, gone, q, lens, n)               # nothing to attend to
    both = np.stack([table[0], table[0]])                        # a prefix shared by two sequences
    _check_attention(cache, ref, both, q, lens, n)
    # queries and outputs as views: heads first, off 16-byte alignment
    big = torch.zeros((2, Hq, L, D + 3), dtype=torch.bfloat16, device="cuda")
    view = big[..., 1:1 + D].transpose(1, 2)
    view.copy_(q)
    obig = torch.full((2, L, Hq, D + 5), 3.0, dtype=torch.bfloat16, device="cuda")
    o = obig[..., 2:2 + D]
    r = dc.block_attention(view, cache, _i32(table), _i32(lens), out=o)
    want = dc.block_attention(q.cuda(), cache, _i32(table), _i32(lens))
    assert torch.equal(r.out, want.out) and torch.equal(r.lse, want.lse)
    assert (obig[..., :2] == 3).all() and (obig[..., 2 + D:] == 3).all()


def test_attention_large_scores_and_far_scales():
    """Scores in the hundreds (one weight carries all), value scales 2^40 apart."""
    T, L, Hq, H, D = 160, 4, 2, 1, 64
    cache, ref, table, q, n = _attention_case(7, 1, L, Hq, H, D, T, [T], scale_q=60.0)
    _check_attention(cache, ref, table, q, [T], n)
    rng = np.random.default_rng(3)
    k = _bf16(rng.normal(0, 0.1, (1, T, H, D)))
    v = _bf16(rng.normal(0, 1, (1, T, H, D)) * np.exp2(np.array([-40.0, 0, 30, -90, 20]).repeat(32))[None, :, None, None])
    dc.kv_write(cache, k.cuda(), v.cuda(), _i32(table), _i32([0]))
    ref.write(_np(k), _np(v), table, [0])
    q = _bf16(rng.normal(0, 0.1, (1, L, Hq, D)))
    _check_attention(cache, ref, table, q, [T], n)
    _check_attention(cache, ref, table, q, [32], n)               # the small page alone


def test_a_large_page_that_nothing_attends_to_costs_no_bits():
    """A page of values 2^50 times the others' whose weight is below 2^-90: the
    others' values come out as exactly as without it."""
    rng = np.random.default_rng(12)
    T, D = 96, 64
    table = np.array([[0, 1, 2]], dtype=np.int32)
    k, v = rng.normal(0, 0.05, (1, T, 1, D)), rng.normal(0, 1, (1, T, 1, D))
    k[0, 32:64] = -3.0
    v[0, 32:64] *= 2.0 ** 50
    v[0, 64:] *= 2.0 ** -30
    q = _bf16(np.full((1, 3, 1, D), 4.0))
    cache, ref = dc.KVCache(3, 1, D), okv.Cache(3, 1, D)
    kt, vt = _bf16(k), _bf16(v)
    dc.kv_write(cache, kt.cuda(), vt.cuda(), _i32(table), _i32([0]))
    ref.write(_np(kt), _np(vt), table, [0])
    r = dc.block_attention(q.cuda(), cache, _i32(table), _i32([T]))
    rk, rv = ref.read(table, [T])
    o, _, _, mass, _ = okv.block_attention(_np(q), rk, rv, table, [T], 3)
    # the outputs are of order 1 though values of 2^50 are there; the tolerance
    # has no term of their size
    tol = 2.0 ** -8 * np.abs(o) + mass * (2.0 ** -11 + 2.0 ** -12)
    assert (np.abs(_np(r.out) - o) <= tol).all() and np.abs(o).max() < 2


def test_nan_query_stays_in_its_row():
    cache, ref, table, q, n = _attention_case(9, 1, 6, 2, 1, 64, 100, [100])
    want = dc.block_attention(q.cuda(), cache, _i32(table), _i32([100]))
    bad = q.clone()
    bad[0, 2, 1, 5] = float("nan")
    r = dc.block_attention(bad.cuda(), cache, _i32(table), _i32([100]))
    assert r.out[0, 2, 1].isnan().all() and r.lse[0, 1, 2].isnan()
    keep = torch.ones((6, 2), dtype=torch.bool)
    keep[2, 1] = False
    assert torch.equal(r.out[0][keep.cuda()], want.out[0][keep.cuda()])
    # the other queries' weights go on adding up
    bad[0, 4, 0, 7] = float("inf")
    w = torch.zeros((1, table.shape[1] * PAGE), device="cuda")
    r = dc.block_attention(bad.cuda(), cache, _i32(table), _i32([100]), weights=w)
    assert not torch.isfinite(r.lse[0, 0, 4]) and torch.isfinite(w).all()
    assert abs(float(w.sum()) - 10) < 1e-3


def test_offsets_past_32_bits():
    """A pool whose last pages lie more than 2^31 bytes from its start."""
    H, D = 8, 256
    pages = (2 ** 31 // (H * D * PAGE)) + 40
    cache = dc.KVCache(pages, H, D)
    rng = np.random.default_rng(2)
    table = np.array([[pages - 1, 0, pages - 30]], dtype=np.int32)
    small = np.array([[1, 0, 2]], dtype=np.int32)
    k, v = _kv(rng, 1, 90, H, D)
    ref = okv.Cache(3, H, D)
    ref.write(_np(k), _np(v), small, [0])
    dc.kv_write(cache, k.cuda(), v.cuda(), _i32(table), _i32([0]))
    gk, gv = dc.kv_read(cache, _i32(table), _i32([90]))
    rk, rv = ref.read(small, [90])
    assert np.array_equal(_np(gk), rk) and np.array_equal(_np(gv), rv)
    near = dc.KVCache(3, H, D)
    dc.kv_write(near, k.cuda(), v.cuda(), _i32(small), _i32([0]))
    q = _bf16(rng.normal(0, 0.05, (1, 3, H, D))).cuda()
    a = dc.block_attention(q, cache, _i32(table), _i32([90]))
    b = dc.block_attention(q, near, _i32(small), _i32([90]))
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)


def test_streams_graphs_and_repeats():
    """A block step captured (write, attention with weights) and replayed against
    eager calls; two graphs side by side; another stream; equal bits each time."""
    B, L, Hq, H, D, T = 2, 32, 8, 2, 128, 2000
    lens = [T, 1500]
    cache, ref, table, q, n = _attention_case(5, B, L, Hq, H, D, T, lens)
    rng = np.random.default_rng(0)
    qs, tb = q.cuda(), _i32(table)
    start = _i32([T - 32, 1500 - 32])
    ln = _i32(lens)
    kn, vn = (t.cuda() for t in _kv(rng, B, L, H, D))
    w1, w2 = (torch.zeros((B, table.shape[1] * PAGE), device="cuda") for _ in range(2))

    def step(w):
        dc.kv_write(cache, kn, vn, tb, start)
        return dc.block_attention(qs, cache, tb, ln, weights=w)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        eager = step(w1.clone())
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        r1 = step(w1)
    with torch.cuda.graph(g2):
        r2 = dc.block_attention(qs, cache, tb, ln, weights=w2)
    for i in range(4):
        kn.copy_(torch.roll(kn, 1, dims=1))
        w1.zero_()
        w2.zero_()
        ew = torch.zeros_like(w1)
        e = step(ew)
        g1.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            g2.replay()
        with torch.cuda.stream(torch.cuda.Stream()):
            e2 = dc.block_attention(qs, cache, tb, ln)
        torch.cuda.synchronize()
        for a in (r1, r2, e2):
            assert torch.equal(a.out, e.out) and torch.equal(a.lse, e.lse)
        assert torch.equal(w1, ew) and torch.equal(w2, ew)


def test_eviction_captured():
    """Selection and gather in a graph, replayed over new weights and lengths."""
    rng = np.random.default_rng(21)
    B, H, D, T, budget = 2, 2, 64, 300, 100
    table, new, n = _table(rng, B, 10, 4)
    cache, ref = dc.KVCache(n, H, D), okv.Cache(n, H, D)
    k, v = _kv(rng, B, T, H, D)
    dc.kv_write(cache, k.cuda(), v.cuda(), _i32(table), _i32([0, 0]))
    ref.write(_np(k), _np(v), table, [0, 0])
    tb, nt, lens = _i32(table), _i32(new), _i32([T, T])
    w = torch.rand((B, 320), device="cuda")
    dc.kv_evict(cache, tb, lens, w, budget, nt, 2, 8)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = dc.kv_evict(cache, tb, lens, w, budget, nt, 2, 8)
    for i in range(4):
        w.copy_(torch.from_numpy(rng.random((B, 320)).astype(np.float32)))
        lens.copy_(_i32([T - 70 * i, 50 + i]))
        graph.replay()
        torch.cuda.synchronize()
        kept, nl = okv.evict_select(w.cpu().numpy(), lens.cpu().numpy(), budget, 2, 8)
        assert np.array_equal(r.kept.cpu().numpy(), kept) and np.array_equal(r.lens.cpu().numpy(), nl)
        ref.gather(table, kept, nl, new)
        _same_cache(cache, ref, new, nl)


def test_refusals_on_the_device():
    cache = dc.KVCache(4, 2, 64)
    tb, ln = _i32([[0, 1]]), _i32([10])
    x = torch.zeros((1, 4, 2, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((1, 4, 4, 64), dtype=torch.bfloat16, device="cuda")
    for k, v, t, s in ((x.float(), x, tb, ln), (x, x[:, :, :1], tb, ln), (x[..., :32], x, tb, ln),
                       (x, x, tb.long(), ln), (x, x, tb[0], ln), (x, x, tb, ln.float()), (x, x, tb, None),
                       (x, x.cpu(), tb, ln), (x, x, tb.cpu(), ln), (x, x, _i32([[0, 1], [2, 3]]), ln),
                       (x[0], x[0], tb, ln), (x.transpose(2, 3).contiguous().transpose(2, 3), x, tb, ln)):
        with pytest.raises(ValueError):
            dc.kv_write(cache, k, v, t, s)
    good = dict(q=q, cache=cache, page_table=tb, kv_lens=ln)
    for bad in (dict(q=q.float()), dict(q=q[:, :, :3]), dict(q=q[..., :32]), dict(kv_lens=None),
                dict(kv_lens=ln.long()), dict(block_len=-1), dict(scale=0.0), dict(scale=float("nan")),
                dict(weights=torch.zeros((1, 63), device="cuda")), dict(out=q), dict(out=q.float()),
                dict(lse=torch.zeros((1, 4, 3), device="cuda")), dict(q_lens=ln.cpu()),
                dict(page_table=_i32([[0, 1, 2, 3]])[:, ::2]),
                dict(out=torch.zeros_like(q[:, :1]).expand(1, 4, 4, 64)),
                dict(q=q.clone().requires_grad_())):
        with pytest.raises(ValueError):
            dc.block_attention(**{**good, **bad})
    w = torch.zeros((1, 64), device="cuda")
    for bad in (dict(budget=0), dict(sink=9, recent=9), dict(new_pages=_i32([[2]]), budget=40),
                dict(weights=w[:, :60]), dict(new_pages=tb)):
        with pytest.raises(ValueError):
            dc.kv_evict(**{**dict(cache=cache, page_table=tb, kv_lens=ln, weights=w, budget=16,
                                  new_pages=_i32([[2]])), **bad})
    with torch.no_grad():
        dc.block_attention(**{**good, "q": q.clone().requires_grad_()})
    # empty calls
    r = dc.block_attention(q[:, :0], cache, tb, ln)
    assert r.out.shape == (1, 0, 4, 64) and r.lse.shape == (1, 4, 0)
    dc.kv_write(cache, x[:, :0], x[:, :0], tb, ln)
    assert dc.block_attention(q, cache, tb[:, :0], ln).lse.isneginf().all()
    e = dc.kv_evict(cache, tb[:, :0], ln, w[:, :0], 16, _i32([[2]]))
    assert int(e.lens) == 0 and (e.kept == -1).all() and not e.weights.any()
    dc.kv_gather(cache, tb, e.kept[:, :0], e.lens, _i32([[3]]))
