"""Pins of the oracle of the scores, the 8-bit cache, block attention and
eviction: closed forms, differences, torch's own e4m3 rounding, brute force."""
import itertools
import math

import numpy as np
import pytest
import torch

from oracle import block_causal_mask, kv, scores


def test_scores_closed_forms():
    x = np.array([[[0.0, math.log(3.0), -np.inf, 0.0]]])
    r = scores.token_logprobs(x, np.array([[1]]), top=4)
    assert r.logprob[0, 0] == pytest.approx(math.log(0.6))
    assert r.entropy[0, 0] == pytest.approx(-(0.6 * math.log(0.6) + 0.4 * math.log(0.2)))
    assert r.top_ids[0, 0].tolist() == [1, 0, 3, -1]          # the tie by lower id, p = 0 not listed
    r = scores.token_logprobs(2 * x, np.array([[1]]), T=2.0, suppress=(1,), top=2)
    assert r.logprob[0, 0] == -np.inf and r.entropy[0, 0] == pytest.approx(math.log(2.0))
    assert r.top_ids[0, 0].tolist() == [0, 3]
    uniform = scores.token_logprobs(np.full((1, 1, 5), -np.inf), np.array([[4]]), top=2)
    assert uniform.logprob[0, 0] == pytest.approx(-math.log(5.0))
    assert uniform.top_ids[0, 0].tolist() == [0, 1]
    off = scores.token_logprobs(x, np.array([[-1]]), top=1)
    assert off.logprob[0, 0] == 0 and off.entropy[0, 0] == 0 and off.top_ids[0, 0, 0] == -1


@pytest.mark.parametrize("T,suppress", [(1.0, ()), (0.7, (2,)), (1.9, (0, 5))])
def test_scores_gradient_against_differences(T, suppress):
    rng = np.random.default_rng(5)
    x = rng.normal(0, 2, (1, 2, 7))
    t, g, h = np.array([[1, 3]]), rng.normal(size=(1, 2)), rng.normal(size=(1, 2))

    def f(y):
        r = scores.token_logprobs(y, t, T, suppress)
        return (g * r.logprob + h * r.entropy).sum()

    got = scores.token_logprobs_grad(scores.token_logprobs(x, t, T, suppress), t, g, h, T, suppress)
    for i in itertools.product(range(1), range(2), range(7)):
        e = np.zeros_like(x)
        e[i] = 1e-5
        # central difference: O(1e-10) truncation, 1e-16 / 1e-5 rounding
        assert got[i] == pytest.approx((f(x + e) - f(x - e)) / 2e-5, abs=1e-8)


def test_e4m3_coding_is_torchs_rounding():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.normal(0, 40, 2000), rng.normal(0, 0.01, 2000), kv.e4m3_values(),
                        (kv.e4m3_values()[:-1] + kv.e4m3_values()[1:]) / 2])
    x = np.clip(x.astype(np.float32), -448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(kv.code(x.astype(np.float64), 1.0), want)
    assert kv.e4m3_values()[-1] == 448.0 and len(kv.e4m3_values()) == 127


def test_scales():
    for a, e in [(0.0, -100), (448.0, 0), (448.01, 1), (1.75, -8), (1.76, -7), (1e-40, -100),
                 (3.3e38, 119)]:
        assert kv.scale_of(np.array([[a, np.inf, np.nan]])) == 2.0 ** e


def test_write_read_and_growth():
    c = kv.Cache(4, 1, 64)
    table = np.array([[2, 0]])
    x = np.full((1, 3, 1, 64), 1.0)
    c.write(x, 2 * x, table, [30])
    k, v = c.read(table, [33])
    assert (k[0, 30:33] == 1.0).all() and (v[0, 30:33] == 2.0).all() and not k[0, :30].any()
    c.write(1e4 * x, x, table, [33])                 # grows the second page's key scale
    k, _ = c.read(table, [36])
    assert k[0, 32, 0, 0] == 1.0 and abs(k[0, 33, 0, 0] - 1e4) <= 1e4 / 16


def test_attention_is_the_dense_formula_under_the_block_mask():
    rng = np.random.default_rng(3)
    L, bl, D = 40, 7, 64
    q, k, v = rng.normal(size=(1, L, 2, D)), rng.normal(size=(1, 64, 1, D)), rng.normal(size=(1, 64, 1, D))
    out, lse, w, _, _ = kv.block_attention(q, k, v, np.array([[0, 1]]), [L], 2, block_len=bl)
    mask = block_causal_mask(L, bl)
    for h in range(2):
        s = q[0, :, h] @ k[0, :L, 0].T / 8.0 + mask
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        assert np.allclose(out[0, :, h], p @ v[0, :L, 0], rtol=0, atol=1e-12)
    assert w.sum() == pytest.approx(2 * L) and not w[0, L:].any()
    out, lse, w, _, _ = kv.block_attention(q, k, v, np.array([[0, 1]]), [0], 2)
    assert not out.any() and (lse == -np.inf).all() and not w.any()


def test_evict_select_against_brute_force():
    rng = np.random.default_rng(9)
    for _ in range(200):
        n = int(rng.integers(1, 9))
        w = rng.integers(0, 4, (1, n)).astype(np.float64)
        budget = int(rng.integers(1, 9))
        sink = int(rng.integers(0, budget + 1))
        recent = int(rng.integers(0, budget - sink + 1))
        kept, lens = kv.evict_select(w, [n], budget, sink, recent)
        got = [t for t in kept[0] if t >= 0]
        assert len(got) == lens[0] == min(n, budget) and got == sorted(got)
        if n > budget:
            safe = {t for t in range(n) if t < sink or t >= n - recent}
            assert safe <= set(got)
            free = [c for c in itertools.combinations(range(n), budget) if safe <= set(c)]
            best = max(sum(w[0, t] for t in c) for c in free)
            assert sum(w[0, t] for t in got) == best
            # ties: the lexicographically lowest set of the best ones
            assert tuple(got) == min(c for c in free if sum(w[0, t] for t in c) == best)
