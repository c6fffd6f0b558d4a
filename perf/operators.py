"""Timed cases of the library's operators around the commit step: scores of
given tokens and their gradient, the 8-bit key/value cache, block attention
over it, and eviction from it.

Every case runs in two forms.  The plain form (own = False) is elementary torch
in float32; the other form (own = True) is the calls a program makes of
commit_step_amd.  exact() gives the same outputs in float64 from the operators'
definitions.

Sizes: the vocabularies, block length and batch shapes of the bench workloads
(LLaDA-like V = 126464, Dream-like V = 151936, blocks of 32), an odd vocabulary
of 50257, and head layouts from one key/value head per query head to seven
query heads per key/value head.
"""
import math

import numpy as np
import torch

own = False

PAGE = 32            # tokens per cache page: one scale per page and head
FP8_MAX = 448.0      # largest e4m3 value
SCALE_FLOOR = -100   # smallest scale exponent


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one served token with its alternatives: latency
        {"name": "score_token", "op": "score", "B": 1, "L": 1, "V": 126464, "dtype": "bf16",
         "top": 20, "T": 1.0, "scored": 1.0},
        # scoring a batch of finished canvases
        {"name": "score_batch", "op": "score", "B": 4, "L": 256, "V": 151936, "dtype": "bf16",
         "top": 5, "T": 0.7, "scored": 1.0},
        # a small training step on float32 logits of an odd vocabulary
        {"name": "train_odd", "op": "train", "B": 2, "L": 100, "V": 50257, "dtype": "f32",
         "top": 0, "T": 1.0, "scored": 0.5},
        # a masked-diffusion training step: loss on the masked half of the positions
        {"name": "train_masked", "op": "train", "B": 8, "L": 512, "V": 126464, "dtype": "bf16",
         "top": 0, "T": 1.0, "scored": 0.5},
        # one new token per sequence, in the middle of a page
        {"name": "append_token", "op": "write", "B": 8, "L": 1, "Hkv": 4, "D": 128, "start": 500},
        # prompts written into the cache, ending inside a page
        {"name": "write_prompt", "op": "write", "B": 4, "L": 8000, "Hkv": 8, "D": 128, "start": 0},
        # one query over a short context, one key/value head per query head: latency
        {"name": "attend_token", "op": "attend", "B": 1, "L": 1, "Hq": 32, "Hkv": 32, "D": 128,
         "kv": 500, "block": 0, "weights": False},
        # one query per sequence over long contexts of different lengths
        {"name": "attend_long", "op": "attend", "B": 8, "L": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "kv": 32768, "block": 0, "weights": False},
        # a block of 32 denoised over the finished prefixes, seven query heads per
        # key/value head, with the weights the eviction goes by
        {"name": "attend_block", "op": "attend", "B": 4, "L": 32, "Hq": 28, "Hkv": 4, "D": 128,
         "kv": 8191, "block": 0, "weights": True},
        # a whole prompt under the block-causal mask, with weights
        {"name": "attend_prompt", "op": "attend", "B": 1, "L": 8192, "Hq": 32, "Hkv": 32, "D": 128,
         "kv": 8192, "block": 32, "weights": True},
        # halving a short cache
        {"name": "evict_short", "op": "evict", "B": 1, "kv": 1000, "budget": 512, "Hkv": 32,
         "D": 128, "sink": 4, "recent": 64},
        # long caches down to a quarter
        {"name": "evict_long", "op": "evict", "B": 4, "kv": 32768, "budget": 8192, "Hkv": 8,
         "D": 128, "sink": 4, "recent": 128},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["score", "train", "write", "attend", "attend", "evict"])
    if op in ("score", "train"):
        V = rng.choice([126464, 151936, 50257, _log_int(rng, 1000, 160000)])
        cap = 4 * 10 ** 8 if op == "train" else 10 ** 8
        rows = _log_int(rng, 1, max(1, cap // V))
        B = rng.choice([b for b in (1, 2, 3, 4, 8) if b <= rows])
        return {"op": op, "B": B, "L": max(1, rows // B), "V": V,
                "dtype": rng.choice(["bf16", "f32"]) if rows * V < 10 ** 8 else "bf16",
                "top": 0 if op == "train" else rng.choice([0, 1, 5, 20]),
                "T": rng.choice([1.0, 0.7, 1.3]), "scored": rng.choice([1.0, 0.5, 0.15])}
    Hkv, G = rng.choice([(32, 1), (4, 7), (8, 4), (2, 8), (3, 5)])
    D = rng.choice([64, 128, 128, 256])
    if op == "write":
        return {"op": op, "B": rng.choice([1, 2, 5, 8]), "L": _log_int(rng, 1, 4000),
                "Hkv": min(Hkv, 8), "D": min(D, 128), "start": rng.choice([0, 32, 77, 500])}
    if op == "evict":
        kv = _log_int(rng, 100, 30000)
        budget = max(40, int(kv * rng.uniform(0.1, 0.9)))
        return {"op": op, "B": rng.choice([1, 2, 4]), "kv": kv, "budget": budget,
                "Hkv": min(Hkv, 8), "D": min(D, 128), "sink": rng.choice([0, 4]),
                "recent": rng.choice([0, 16, 32])}
    kind = rng.choice(["token", "block", "prompt"])
    if kind == "token":
        L, kv, block, B = 1, _log_int(rng, 1, 30000), 0, rng.choice([1, 2, 8])
    elif kind == "block":
        L, kv, block, B = rng.choice([16, 32, 32, 64]), _log_int(rng, 64, 8000), 0, \
            rng.choice([1, 2, 4])
    else:
        L = _log_int(rng, 64, 3000)
        kv, block, B = L, rng.choice([1, 32, 64]), rng.choice([1, 2])
    return {"op": "attend", "B": B, "L": L, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "kv": kv,
            "block": block, "weights": rng.random() < 0.4}


def _lens(case):
    """Tokens in each sequence's cache: from kv down to about half of it, except
    for prompts, which are whole."""
    B, kv = case["B"], case["kv"]
    if case.get("block", 0) > 0:
        return [kv] * B
    return [max(1, kv - (kv * b) // (2 * B)) for b in range(B)]


def _pages(tokens):
    return (tokens + PAGE - 1) // PAGE


def work(case):
    op = case["op"]
    if op in ("score", "train"):
        s = 2 if case["dtype"] == "bf16" else 4
        rows = case["B"] * case["L"]
        scored = int(round(rows * case["scored"]))
        V = case["V"]
        if op == "score":
            return {"bytes": scored * V * s + rows * (12 + 8 * case["top"]),
                    "flops": 6 * scored * V}
        return {"bytes": scored * V * s + rows * V * s + 20 * rows, "flops": 14 * scored * V}
    Hkv, D = case["Hkv"], case["D"]
    if op == "write":
        n = case["B"] * case["L"] * Hkv * D * 2
        # read bf16, write codes, and the read-back: codes in, bf16 out
        return {"bytes": n * 2 + n + n + n * 2, "flops": 4 * n}
    lens = _lens(case)
    if op == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        codes = kept * Hkv * D * 2
        # weights in, survivors' codes in and out, and the read-back
        return {"bytes": 4 * sum(lens) + 8 * kept + 2 * codes + codes + 2 * codes,
                "flops": 4 * codes}
    L, Hq = case["L"], case["Hq"]
    if case["block"] > 0:
        bl = case["block"]
        pairs = sum(min(n, (i // bl + 1) * bl) for n in lens for i in range(L))
    else:
        pairs = sum(L * n for n in lens)
    flops = (6 if case["weights"] else 4) * pairs * Hq * D
    kv = sum(lens) * Hkv * D * 2
    return {"bytes": kv + 2 * case["B"] * L * Hq * D * 2 + 4 * case["B"] * L * Hq
            + (4 * sum(lens) if case["weights"] else 0), "flops": flops}


# ---------------------------------------------------------------- inputs

def _gen(seed, salt=0):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17 + salt)


def _logit_inputs(case, seed):
    """Normal logits, the given token raised at most positions (a trained
    model's canvases), some positions not scored."""
    B, L, V = case["B"], case["L"], case["V"]
    g = _gen(seed)
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    logits = torch.empty((B, L, V), dtype=dtype, device="cuda")
    for b in range(B):
        logits[b] = torch.randn((L, V), generator=g, device="cuda").mul_(2.5)
    targets = torch.randint(0, V, (B, L), generator=g, device="cuda", dtype=torch.int32)
    lift = 14.0 * torch.rand((B, L), generator=g, device="cuda")
    at = targets.long().unsqueeze(-1)
    raised = torch.gather(logits, 2, at).float() + lift.unsqueeze(-1)
    logits.scatter_(2, at, raised.to(dtype))
    n = int(round(B * L * case["scored"]))
    order = torch.randperm(B * L, generator=g, device="cuda")
    targets.view(-1)[order[n:]] = -1
    g_lp = torch.randn((B, L), generator=g, device="cuda")
    g_ent = 0.1 * torch.randn((B, L), generator=g, device="cuda")
    return logits, targets, g_lp, g_ent


def _kv_inputs(case, seed, tokens, salt):
    """Keys with a few strong channels, values without, as models have them;
    heads of different size."""
    g = _gen(seed, salt)
    B, H, D = case["B"], case["Hkv"], case["D"]
    size = torch.exp2(2.0 * torch.rand((1, 1, H, 1), generator=g, device="cuda") - 1.0)
    strong = 1.0 + 6.0 * (torch.rand((1, 1, H, D), generator=g, device="cuda") < 0.04)
    k = torch.randn((B, tokens, H, D), generator=g, device="cuda").mul_(size * strong)
    v = torch.randn((B, tokens, H, D), generator=g, device="cuda").mul_(size)
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _tables(case, seed, pages, extra=0):
    """Page tables into a shuffled pool, and as many more pages per row."""
    g = _gen(seed, 7)
    B = case["B"]
    perm = torch.randperm(B * (pages + extra), generator=g, device="cuda").to(torch.int32)
    perm = perm.view(B, pages + extra)
    return perm[:, :pages].contiguous(), perm[:, pages:].contiguous()


def _queries(case, seed):
    g = _gen(seed, 11)
    q = torch.randn((case["B"], case["L"], case["Hq"], case["D"]), generator=g, device="cuda")
    return q.to(torch.bfloat16)


def _token_weights(case, seed):
    """Accumulated attention weights: spread over many powers of two."""
    g = _gen(seed, 13)
    T = _pages(case["kv"]) * PAGE
    w = torch.exp(2.5 * torch.randn((case["B"], T), generator=g, device="cuda"))
    return w


class _PlainPool:
    """The plain form's cache: e4m3 values in token order and their scales."""

    def __init__(self, pages, heads, dim):
        self.k = torch.zeros((pages, heads, PAGE, dim), dtype=torch.float8_e4m3fn, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.k_scale = torch.ones((pages, heads), device="cuda")
        self.v_scale = torch.ones((pages, heads), device="cuda")


def _scale_of(amax):
    """The smallest power of two s, at least 2^-100, with amax / s <= 448."""
    m, e = torch.frexp(amax / FP8_MAX)
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(amax > 0, e, torch.full_like(e, SCALE_FLOOR)).clamp(min=SCALE_FLOOR)
    return torch.ldexp(torch.ones_like(amax), e)


def _plain_store(codes, scales, x, table, start):
    """Write x (B, n, H, D) at positions start.. of every sequence."""
    B, n, H, D = x.shape
    p0, p1 = start // PAGE, (start + n - 1) // PAGE + 1
    ids = table[:, p0:p1].long()
    np_ = p1 - p0
    new = torch.zeros((B, np_ * PAGE, H, D), device=x.device)
    lo = start - p0 * PAGE
    new[:, lo:lo + n] = x.float()
    new = new.view(B, np_, PAGE, H, D).permute(0, 1, 3, 2, 4)
    scale = _scale_of(new.abs().amax(dim=(3, 4)))
    out = (new / scale[..., None, None]).to(torch.float8_e4m3fn).float()
    if lo > 0:
        # tokens of the first page before start stay: the page's scale grows
        # if it has to, and they are coded again in the new one
        old_scale = scales[ids[:, 0]]
        scale[:, 0] = torch.maximum(scale[:, 0], old_scale)
        kept = codes[ids[:, 0]].float() * old_scale[..., None, None]
        first = torch.where((torch.arange(PAGE, device=x.device) < lo)[:, None],
                            kept, new[:, 0])
        out[:, 0] = (first / scale[:, 0, :, None, None]).to(torch.float8_e4m3fn).float()
    out = out.to(torch.float8_e4m3fn)
    scales[ids] = scale
    codes[ids] = out


def _plain_values(codes, scales, table, lens):
    """(B, T, H, D) values of the cached tokens, 0 behind each sequence's end."""
    ids = table.long()
    x = codes[ids].float() * scales[ids][..., None, None]
    B, P, H, _, D = x.shape
    x = x.permute(0, 1, 3, 2, 4).reshape(B, P * PAGE, H, D)
    pos = torch.arange(P * PAGE, device=x.device)
    return torch.where((pos < lens[:, None])[..., None, None], x, torch.zeros_like(x))


def _make_cache(case, pages, table, k, v):
    if own:
        import commit_step_amd as dc
        cache = dc.KVCache(pages, case["Hkv"], case["D"], device="cuda")
        dc.kv_write(cache, k, v, table, torch.zeros(case["B"], dtype=torch.int32, device="cuda"))
        return cache
    pool = _PlainPool(pages, case["Hkv"], case["D"])
    _plain_store(pool.k, pool.k_scale, k, table, 0)
    _plain_store(pool.v, pool.v_scale, v, table, 0)
    return pool


def prepare(case, seed):
    op = case["op"]
    st = {"case": case, "op": op}
    if op in ("score", "train"):
        st["logits"], st["targets"], st["g_lp"], st["g_ent"] = _logit_inputs(case, seed)
        return st
    B = case["B"]
    if op == "write":
        start, L = case["start"], case["L"]
        pages = _pages(start + L)
        st["table"], _ = _tables(case, seed, pages)
        k0, v0 = _kv_inputs(case, seed, max(start, 1), 3)
        st["cache"] = _make_cache(case, B * pages, st["table"], k0, v0)
        st["k"], st["v"] = _kv_inputs(case, seed, L, 5)
        st["start"] = torch.full((B,), start, dtype=torch.int32, device="cuda")
        # the pages this write touches, read back as the values they stand for
        first = start // PAGE
        st["touched"] = st["table"][:, first:].contiguous()
        st["touched_lens"] = torch.full((B,), start + L - first * PAGE, dtype=torch.int32,
                                        device="cuda")
        return st
    kv = case["kv"]
    pages = _pages(kv)
    extra = _pages(case["budget"]) if op == "evict" else 0
    st["table"], st["new_pages"] = _tables(case, seed, pages, extra)
    k, v = _kv_inputs(case, seed, kv, 3)
    st["cache"] = _make_cache(case, B * (pages + extra), st["table"], k, v)
    st["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
    if op == "attend":
        st["q"] = _queries(case, seed)
    else:
        st["weights"] = _token_weights(case, seed)
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import commit_step_amd as dc
    case, op = st["case"], st["op"]
    if op == "score":
        r = dc.token_logprobs(st["logits"], st["targets"], temperature=case["T"], top=case["top"])
        return [r.logprob, r.entropy] + ([r.top_ids, r.top_logprobs] if case["top"] else [])
    if op == "train":
        x = st["logits"].detach().requires_grad_(True)
        r = dc.token_logprobs(x, st["targets"], temperature=case["T"])
        (gx,) = torch.autograd.grad((r.logprob, r.entropy), (x,), (st["g_lp"], st["g_ent"]))
        return [r.logprob.detach(), r.entropy.detach(), gx]
    if op == "write":
        dc.kv_write(st["cache"], st["k"], st["v"], st["table"], st["start"])
        return list(dc.kv_read(st["cache"], st["touched"], st["touched_lens"]))
    if op == "evict":
        r = dc.kv_evict(st["cache"], st["table"], st["lens"], st["weights"], case["budget"],
                        st["new_pages"], sink=case["sink"], recent=case["recent"])
        k, v = dc.kv_read(st["cache"], st["new_pages"], r.lens)
        return [r.kept, r.lens, r.weights, k, v]
    w = None
    if case["weights"]:
        w = torch.zeros((case["B"], st["table"].shape[1] * PAGE), device="cuda")
    r = dc.block_attention(st["q"], st["cache"], st["table"], st["lens"],
                           block_len=case["block"], weights=w)
    return [r.out, r.lse] + ([w] if w is not None else [])


def _run_plain(st):
    case, op = st["case"], st["op"]
    if op in ("score", "train"):
        return _plain_logprobs(st, case, op)
    if op == "write":
        pool = st["cache"]
        _plain_store(pool.k, pool.k_scale, st["k"], st["table"], case["start"])
        _plain_store(pool.v, pool.v_scale, st["v"], st["table"], case["start"])
        k = _plain_values(pool.k, pool.k_scale, st["touched"], st["touched_lens"])
        v = _plain_values(pool.v, pool.v_scale, st["touched"], st["touched_lens"])
        return [k.to(torch.bfloat16), v.to(torch.bfloat16)]
    if op == "evict":
        return _plain_evict(st, case)
    return _plain_attend(st, case)


def _plain_logprobs(st, case, op):
    logits, targets = st["logits"], st["targets"]
    scored = targets >= 0
    at = targets.clamp(min=0).long()
    x = logits.float() / case["T"]
    m = x.amax(dim=-1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    z = e.sum(dim=-1, keepdim=True)
    logz = torch.log(z)
    lp = torch.gather(d, 2, at.unsqueeze(-1)) - logz
    p = e / z
    ent = logz - (p * d).sum(dim=-1, keepdim=True)
    zero = torch.zeros((), device=x.device)
    logprob = torch.where(scored, lp.squeeze(-1), zero)
    entropy = torch.where(scored, ent.squeeze(-1), zero)
    if op == "train":
        # d logprob / dx = (onehot - p) / T, d entropy / dx = -p (log p + H) / T
        g = st["g_lp"].unsqueeze(-1)
        h = st["g_ent"].unsqueeze(-1)
        grad = -p * (g + h * (d - logz + ent))
        grad.scatter_add_(2, at.unsqueeze(-1), g)
        grad = torch.where(scored.unsqueeze(-1), grad / case["T"], zero)
        return [logprob, entropy, grad.to(logits.dtype)]
    if not case["top"]:
        return [logprob, entropy]
    # ties go to the lowest id: a stable sort
    K = case["top"]
    top_x, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    ids = ids[..., :K].to(torch.int32)
    top = top_x[..., :K].float() / case["T"] - m - logz
    s = scored.unsqueeze(-1)
    return [logprob, entropy, torch.where(s, ids, torch.full_like(ids, -1)),
            torch.where(s, top, torch.full_like(top, -math.inf))]


def _allowed(case, n, T, device):
    """(L, T) bool: the keys each query attends to, of a sequence of n tokens."""
    pos = torch.arange(T, device=device)
    ok = (pos < n)[None, :].expand(case["L"], T)
    if case["block"] > 0:
        i = torch.arange(case["L"], device=device)
        ok = ok & (pos[None, :] // case["block"] <= i[:, None] // case["block"])
    return ok


def _plain_attend(st, case):
    q, pool, table, lens = st["q"], st["cache"], st["table"], st["lens"]
    B, L, Hq, D = q.shape
    Hkv = case["Hkv"]
    G = Hq // Hkv
    T = table.shape[1] * PAGE
    scale = 1.0 / math.sqrt(D)
    out = torch.empty_like(q)
    lse = torch.empty((B, Hq, L), device=q.device)
    w = torch.zeros((B, T), device=q.device) if case["weights"] else None
    # heads at a time, so that the scores of a long prompt fit
    step = max(1, min(Hkv, 2 ** 30 // max(1, G * L * T)))
    for b in range(B):
        ok = _allowed(case, lens[b], T, q.device)
        ids = table[b].long()
        for h0 in range(0, Hkv, step):
            h1 = min(Hkv, h0 + step)
            n = h1 - h0
            k = pool.k[ids, h0:h1].float() * pool.k_scale[ids, h0:h1, None, None]
            v = pool.v[ids, h0:h1].float() * pool.v_scale[ids, h0:h1, None, None]
            k = k.permute(1, 0, 2, 3).reshape(n, T, D)
            v = v.permute(1, 0, 2, 3).reshape(n, T, D)
            v = torch.where((torch.arange(T, device=q.device) < lens[b])[None, :, None], v,
                            torch.zeros_like(v))
            qh = q[b, :, h0 * G:h1 * G].float().reshape(L, n, G, D).permute(1, 2, 0, 3)
            s = torch.matmul(qh.reshape(n, G * L, D), k.transpose(1, 2).contiguous()) * scale
            s = s.reshape(n, G, L, T)
            s = torch.where(ok, s, torch.full_like(s, -math.inf))
            m = s.amax(dim=-1, keepdim=True)
            m = torch.where(m == -math.inf, torch.zeros_like(m), m)
            e = torch.exp(s - m)
            z = e.sum(dim=-1, keepdim=True)
            p = e / torch.where(z > 0, z, torch.ones_like(z))
            o = torch.matmul(p.reshape(n, G * L, T), v).reshape(n, G, L, D)
            out[b, :, h0 * G:h1 * G] = o.permute(2, 0, 1, 3).reshape(L, n * G, D).to(q.dtype)
            lse[b, h0 * G:h1 * G] = (m + torch.log(z)).reshape(n * G, L)
            if w is not None:
                w[b] += p.sum(dim=(0, 1, 2))
    return [out, lse] + ([w] if w is not None else [])


def _plain_evict(st, case):
    pool, table, lens, weights = st["cache"], st["table"], st["lens"], st["weights"]
    new_pages = st["new_pages"]
    B, T = weights.shape
    budget = case["budget"]
    pos = torch.arange(T, device=weights.device)
    inside = pos[None, :] < lens[:, None]
    safe = inside & ((pos[None, :] < case["sink"]) | (pos[None, :] >= lens[:, None] - case["recent"]))
    # rank: protected tokens, then by weight, the lowest position first on ties
    key = torch.where(safe, torch.full_like(weights, math.inf), weights)
    key = torch.where(inside, key, torch.full_like(weights, -math.inf))
    order = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :budget]
    n = lens.clamp(max=budget)
    slot = torch.arange(budget, device=weights.device)
    order = torch.where(slot[None, :] < n[:, None], order, torch.full_like(order, T))
    kept = torch.sort(order, dim=1)[0]
    live = slot[None, :] < n[:, None]
    src = torch.where(live, kept, torch.zeros_like(kept))
    T2 = new_pages.shape[1] * PAGE
    new_w = torch.zeros((B, T2), device=weights.device)
    new_w[:, :budget] = torch.where(live, torch.gather(weights, 1, src), torch.zeros_like(new_w[:, :budget]))
    n32 = n.to(torch.int32)
    vals = []
    for codes, scales in ((pool.k, pool.k_scale), (pool.v, pool.v_scale)):
        x = _plain_values(codes, scales, table, lens)
        H, D = x.shape[2:]
        x = torch.gather(x, 1, src[:, :, None, None].expand(B, budget, H, D))
        x = torch.where(live[..., None, None], x, torch.zeros_like(x))
        _plain_store(codes, scales, x, new_pages, 0)
        vals.append(_plain_values(codes, scales, new_pages, n32).to(torch.bfloat16))
    kept = torch.where(live, kept, torch.full_like(kept, -1)).to(torch.int32)
    return [kept, n32, new_w] + vals


# ---------------------------------------------------------------- float64

def _e4m3_exact(x, s):
    """x / s rounded to the nearest e4m3 value (ties to even), times s, in float64."""
    v = x / s
    a = v.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -60)))
    # log2 next to a power of two: put a into [2^e, 2^(e+1))
    e = torch.where(torch.exp2(e) > a, e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= a, e + 1, e)
    step = torch.exp2(e.clamp(min=-6.0) - 3.0)
    return torch.round(v / step) * step * s


def _scale_exact(amax):
    """Scales from the absolute maxima, on the host in exact binary arithmetic."""
    a = amax.cpu().numpy().astype(np.float64)
    out = np.empty_like(a)
    flat, o = a.reshape(-1), out.reshape(-1)
    for i, x in enumerate(flat):
        e = SCALE_FLOOR
        if x > 0:
            m, ex = math.frexp(x)               # x = m 2^ex, m in [0.5, 1); 448 = 0.875 * 2^9
            e = max(SCALE_FLOOR, ex - 9 + (1 if m > 0.875 else 0))
        o[i] = math.ldexp(1.0, e)
    return torch.from_numpy(out).to(amax.device)


def _page_code_exact(x):
    """x (B, T, H, D), T whole pages: its values after one coding."""
    B, T, H, D = x.shape
    x = x.view(B, T // PAGE, PAGE, H, D)
    s = _scale_exact(x.abs().amax(dim=(2, 4)))[:, :, None, :, None]
    return _e4m3_exact(x, s).view(B, T, H, D), s


def _pad_pages(x):
    n = _pages(x.shape[1]) * PAGE
    y = torch.zeros((x.shape[0], n) + x.shape[2:], dtype=torch.float64, device=x.device)
    y[:, :x.shape[1]] = x.double()
    return y


def exact(case, seed):
    op = case["op"]
    if op in ("score", "train"):
        return _exact_logprobs(case, seed)
    if op == "write":
        return _exact_write(case, seed)
    if op == "evict":
        return _exact_evict(case, seed)
    return _exact_attend(case, seed)


def _exact_logprobs(case, seed):
    logits, targets, g_lp, g_ent = _logit_inputs(case, seed)
    B, L, V = logits.shape
    K = case["top"]
    logprob = torch.zeros((B, L), dtype=torch.float64, device="cuda")
    entropy = torch.zeros_like(logprob)
    grad = torch.zeros((B, L, V), dtype=torch.float64, device="cuda") if case["op"] == "train" else None
    ids = torch.full((B, L, K), -1, dtype=torch.int32, device="cuda")
    tops = torch.full((B, L, K), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        rows = torch.nonzero(targets[b] >= 0).view(-1)
        if rows.numel() == 0:
            continue
        t = targets[b, rows].long()
        logp = torch.log_softmax(logits[b, rows].double() / case["T"], dim=-1)
        p = logp.exp()
        at = torch.arange(rows.numel(), device="cuda")
        logprob[b, rows] = logp[at, t]
        ent = -(p * logp).sum(dim=-1)
        entropy[b, rows] = ent
        if grad is not None:
            d = -p * (g_lp[b, rows].double()[:, None]
                      + g_ent[b, rows].double()[:, None] * (logp + ent[:, None]))
            d[at, t] += g_lp[b, rows].double()
            grad[b, rows] = d / case["T"]
        if K:
            # the K largest, one after another, the lowest id first
            left = logits[b, rows].double()
            for j in range(K):
                best = left.amax(dim=-1, keepdim=True)
                first = (left == best).to(torch.int8).argmax(dim=-1)
                ids[b, rows, j] = first.to(torch.int32)
                tops[b, rows, j] = logp[at, first]
                left[at, first] = -math.inf
    if grad is not None:
        return [logprob, entropy, grad]
    return [logprob, entropy] + ([ids, tops] if K else [])


def _exact_write(case, seed):
    B, L, start = case["B"], case["L"], case["start"]
    k0, v0 = _kv_inputs(case, seed, max(start, 1), 3)
    k1, v1 = _kv_inputs(case, seed, L, 5)
    first = start // PAGE
    lo = start - first * PAGE
    out = []
    for x0, x1 in ((k0, k1), (v0, v1)):
        new = torch.zeros((B, lo + L) + x1.shape[2:], dtype=torch.float64, device="cuda")
        new[:, lo:] = x1.double()
        new = _pad_pages(new)
        s = _scale_exact(new.view(B, -1, PAGE, *new.shape[2:]).abs().amax(dim=(2, 4)))
        if lo:
            old, old_s = _page_code_exact(_pad_pages(x0))
            new[:, :lo] = old[:, first * PAGE:first * PAGE + lo]
            s[:, 0] = torch.maximum(s[:, 0], old_s[:, first, 0, :, 0])
        T, H, D = new.shape[1:]
        y = _e4m3_exact(new.view(B, T // PAGE, PAGE, H, D), s[:, :, None, :, None])
        y = y.reshape(B, T, H, D)
        y[:, lo + L:] = 0
        out.append(y)
    return out


def _exact_attend(case, seed):
    B, L, Hq, Hkv, D = (case[n] for n in ("B", "L", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    k, v = _kv_inputs(case, seed, case["kv"], 3)
    k, v = _page_code_exact(_pad_pages(k))[0], _page_code_exact(_pad_pages(v))[0]
    q = _queries(case, seed).double()
    T = k.shape[1]
    lens = _lens(case)
    out = torch.zeros((B, L, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, Hq, L), dtype=torch.float64, device="cuda")
    w = torch.zeros((B, T), dtype=torch.float64, device="cuda")
    for b in range(B):
        n = lens[b]
        for h in range(Hq):
            for i0 in range(0, L, 4096):
                i1 = min(L, i0 + 4096)
                s = (q[b, i0:i1, h] @ k[b, :n, h // G].T.contiguous()) / math.sqrt(D)
                if case["block"] > 0:
                    i = torch.arange(i0, i1, device="cuda")
                    end = (i // case["block"] + 1) * case["block"]
                    s.masked_fill_(torch.arange(n, device="cuda")[None, :] >= end[:, None], -math.inf)
                lz = torch.logsumexp(s, dim=-1)
                p = torch.exp(s - lz[:, None])
                out[b, i0:i1, h] = p @ v[b, :n, h // G]
                lse[b, h, i0:i1] = lz
                w[b, :n] += p.sum(dim=0)
    return [out, lse] + ([w] if case["weights"] else [])


def _exact_evict(case, seed):
    B, budget = case["B"], case["budget"]
    k, v = _kv_inputs(case, seed, case["kv"], 3)
    k, v = _page_code_exact(_pad_pages(k))[0], _page_code_exact(_pad_pages(v))[0]
    w = _token_weights(case, seed)
    lens = _lens(case)
    T2 = _pages(budget) * PAGE
    kept = torch.full((B, budget), -1, dtype=torch.int32)
    new_w = torch.zeros((B, T2), dtype=torch.float64)
    nk = torch.zeros((B, T2) + k.shape[2:], dtype=torch.float64, device="cuda")
    nv = torch.zeros_like(nk)
    for b in range(B):
        n = lens[b]
        wb = w[b, :n].cpu().numpy()
        safe = np.zeros(n, dtype=bool)
        safe[:case["sink"]] = True
        safe[max(0, n - case["recent"]):] = True
        order = np.lexsort((np.arange(n), -wb.astype(np.float64), ~safe))
        keep = np.sort(order[:budget])
        m = len(keep)
        kept[b, :m] = torch.from_numpy(keep.astype(np.int32))
        new_w[b, :m] = torch.from_numpy(wb[keep].astype(np.float64))
        at = torch.from_numpy(keep).cuda()
        nk[b, :m], nv[b, :m] = k[b, at], v[b, at]
    live = torch.tensor([min(n, budget) for n in lens], dtype=torch.int32)
    return [kept.cuda(), live.cuda(), new_w.cuda(), _page_code_exact(nk)[0], _page_code_exact(nv)[0]]
