"""The operators together, as a decoding loop uses them, over a stub model: the
prompt's keys go into the cache, blocks are denoised against it step by step
(write the block's keys, attend, commit), finished blocks are scored, and the
cache is cut by the attention weights it has gathered.  The same loop in
float64 on the CPU, teacher-forced with the GPU's decisions, checks every step;
a training step over the result checks the gradient."""
import numpy as np
import pytest
import torch

import commit_step_amd as dc
import oracle
from oracle import kv as okv
from oracle import scores

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
PAGE = 32


class Stub:
    """Fixed random projections: embeddings to q, k, v, attention outputs to
    logits.  The device and the CPU see the same bfloat16 numbers."""

    def __init__(self, V, E, Hq, H, D, seed):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)
        self.emb = r(V, E)
        self.wq, self.wk, self.wv = r(E, Hq * D) / E ** 0.5, r(E, H * D) / E ** 0.5, r(E, H * D) / E ** 0.5
        self.head = r(Hq * D, V) * 3 / (Hq * D) ** 0.5
        self.Hq, self.H, self.D = Hq, H, D

    def qkv(self, tokens, pos):
        x = self.emb[tokens] + torch.sin(pos[..., None] / 7.0)
        f = lambda w, n: (x @ w).reshape(*tokens.shape, n, self.D).to(torch.bfloat16)
        return f(self.wq, self.Hq), f(self.wk, self.H), f(self.wv, self.H)

    def logits(self, att):                       # (B, L, Hq, D) bfloat16 -> (B, L, V) bfloat16
        return (att.float().reshape(*att.shape[:2], -1) @ self.head).to(torch.bfloat16)


def test_block_decoding_with_cache_scores_and_eviction():
    B, V, P, bl, blocks, budget = 2, 211, 70, 32, 3, 96
    mask = V - 1
    m = Stub(V, 24, 4, 2, 64, 3)
    rng = np.random.default_rng(0)
    pages, spare = 8, -(-budget // PAGE) + 2
    pool = rng.permutation(B * (pages + blocks * spare)).astype(np.int32)
    tables = pool[:B * pages].reshape(B, pages)
    fresh = list(pool[B * pages:].reshape(blocks, B, spare))
    n = len(pool)
    cache, ref = dc.KVCache(n, m.H, m.D), okv.Cache(n, m.H, m.D)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
    np64 = lambda t: t.detach().cpu().double().numpy()

    prompt = torch.from_numpy(rng.integers(0, mask, (B, P)))
    plens = np.array([P, P - 25])
    _, k, v = m.qkv(prompt, torch.arange(P).expand(B, P))
    dc.kv_write(cache, k.cuda(), v.cuda(), i32(tables), i32([0] * B), i32(plens))
    ref.write(np64(k), np64(v), tables, [0] * B, plens)
    lens = plens.copy()                          # finished tokens in the cache
    pos0 = plens.copy()                          # their positions go on after an eviction
    weights = torch.zeros((B, pages * PAGE), device="cuda")
    want_w = np.zeros((B, pages * PAGE))
    evictions = 0
    for blk in range(blocks):
        tokens = torch.full((B, bl), mask, dtype=torch.int32, device="cuda")
        total = lens + bl
        for step in range(bl):
            host = tokens.cpu().long()
            pos = torch.from_numpy(pos0)[:, None] + torch.arange(bl)
            q, k, v = m.qkv(host, pos)
            dc.kv_write(cache, k.cuda(), v.cuda(), i32(tables), i32(lens))
            ref.write(np64(k), np64(v), tables, lens)
            last = int((tokens == mask).sum(dim=1).max()) <= 8
            att = dc.block_attention(q.cuda(), cache, i32(tables), i32(total),
                                     weights=weights if last else None)
            rk, rv = ref.read(tables, total)
            o, lse, w, mass, mag = okv.block_attention(np64(q), rk, rv, tables, total, n)
            ds = (m.D + 8) * U * mag.max() + 8 * U * (np.abs(lse).max() + mag.max())
            tol = 2.0 ** -8 * np.abs(o) + mass * (2.0 ** -11 + 2 * ds + 300 * U) * 1.01 + 2.0 ** -30
            assert (np.abs(np64(att.out) - o) <= tol).all()
            if last:
                want_w += w
            logits = m.logits(att.out.cpu())
            dev = logits.cuda()
            cand = tokens == mask
            rule = dc.Rule.topk(cand, 8)
            r = dc.commit_step(dev, tokens, [rule], suppress_ids=[mask])
            st = oracle.token_stats(logits.view(torch.int16).numpy().view(np.uint16), "bf16",
                                    suppress_ids=[mask])
            got = tokens.cpu().numpy()
            done = rule.out.cpu().numpy()
            assert np.array_equal(got[done], st.x0[done]) and (done <= cand.cpu().numpy()).all()
            if int(r.counts[:, 0].sum()) == 0:
                break
        # the finished block: its keys, its scores under the model that wrote it
        q, k, v = m.qkv(tokens.cpu().long(), pos)
        dc.kv_write(cache, k.cuda(), v.cuda(), i32(tables), i32(lens))
        ref.write(np64(k), np64(v), tables, lens)
        s = dc.token_logprobs(dev, tokens, suppress_ids=[mask], top=3)
        exact = scores.token_logprobs(logits.double().numpy(), tokens.cpu().numpy(), suppress=(mask,), top=3)
        assert np.array_equal(s.top_ids.cpu().numpy(), exact.top_ids)
        # one lane adds one element of 211, 64 lanes and 4 waves are folded
        rel = (1 + 64 + 300) * U
        assert (np.abs(np64(s.logprob) - exact.logprob) <= rel * (exact.entropy + 1) + 4 * U * np.abs(exact.logprob)).all()
        lens, pos0 = total, pos0 + bl
        assert (np.abs(np64(weights) - want_w) <= want_w * 1e-4 + 1e-6).all()
        if (lens > budget).any():
            new = fresh.pop()
            e = dc.kv_evict(cache, i32(tables), i32(lens), weights, budget, i32(new), sink=2, recent=bl)
            kept, nl = okv.evict_select(weights.cpu().numpy(), lens, budget, 2, bl)
            assert np.array_equal(e.kept.cpu().numpy(), kept) and np.array_equal(e.lens.cpu().numpy(), nl)
            ref.gather(tables, kept, nl, new)
            gk, gv = dc.kv_read(cache, i32(new), i32(nl))
            rk, rv = ref.read(new, nl)
            assert np.array_equal(np64(gk), rk) and np.array_equal(np64(gv), rv)
            tables, lens, weights = new, nl.astype(np.int64), e.weights
            want_w = np64(weights)
            evictions += 1
    assert evictions >= 1

    # a masked-diffusion training step on the last block's logits
    x = dev.detach().requires_grad_(True)
    t = tokens.clone()
    t[:, ::2] = -1
    lp = dc.token_logprobs(x, t, suppress_ids=[mask]).logprob
    loss = -(lp * 0.25).sum()
    loss.backward()
    s64 = scores.token_logprobs(logits.double().numpy(), t.cpu().numpy(), suppress=(mask,))
    g = np.full((B, bl), -0.25)
    want = scores.token_logprobs_grad(s64, t.cpu().numpy(), g, 0 * g, 1.0, (mask,))
    # rounded once to bfloat16; p carries (365 + 100) u
    assert (np.abs(np64(x.grad) - want) <= 2.0 ** -8 * np.abs(want) + 0.25 * np.exp(s64.logp) * 465 * U + 1e-30).all()
