"""Refusals of the scores, cache, attention and eviction entry points, checked
on the CPU: every call here fails validation (or has nothing to do) before
anything is launched.  And, by reading the build: no scratch memory in their
kernels, and LDS within a workgroup's limit."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

import commit_step_amd as dc
from test_kernel_resources import CSRC, HIPCC, LDS_LIMIT, ROOT, _parse

P = ctypes.c_void_p
fake = P(256)
S3 = (ctypes.c_int64 * 3)(4096, 128, 64)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(dc.library_path()):
        from commit_step_amd.build import build
        build(verbose=False)
    return dc.load_library()


def _err(lib):
    return lib.dllm_last_error().decode()


def test_logprobs_refusals(lib):
    def call(logits=fake, dtype=1, B=1, L=1, V=8, stride=8, T=1.0, sup=None, nsup=0, targets=fake,
             top=0, lp=fake, ids=fake, lps=fake, ws=fake, wsb=1 << 20):
        return lib.dllm_token_logprobs(logits, dtype, B, L, V, stride, T, sup, nsup, targets, top,
                                       lp, fake, fake, ids, lps, ws, wsb, None)

    assert call(dtype=2) == -2 and "dtype" in _err(lib)
    for bad in (dict(B=-1), dict(L=-1), dict(V=0), dict(V=1 << 31, stride=1 << 31), dict(stride=7),
                dict(T=0.0), dict(T=-1.0), dict(T=math.nan), dict(T=math.inf), dict(T=1e-38), dict(nsup=1),
                dict(nsup=65), dict(top=33), dict(top=-1), dict(logits=None), dict(targets=None),
                dict(lp=None), dict(top=1, ids=None), dict(top=1, lps=None), dict(logits=P(257))):
        assert call(**bad) == -1, bad
    assert call(sup=(ctypes.c_int32 * 2)(3, 3), nsup=2) == -1 and "twice" in _err(lib)
    assert call(sup=(ctypes.c_int32 * 1)(8), nsup=1) == -1 and "outside" in _err(lib)
    assert call(V=1, stride=1, sup=(ctypes.c_int32 * 1)(0), nsup=1) == -1
    assert call(B=1 << 20, L=1 << 20) == -5
    need = lib.dllm_token_logprobs_workspace_size(1, 1, 1, 126464, 20)
    assert need > 0 and lib.dllm_token_logprobs_workspace_size(1, 1, 1, 126464, 33) == 0
    assert call(V=126464, stride=126464, top=20, wsb=need - 1) == -3 and "workspace" in _err(lib)
    assert call(V=126464, stride=126464, top=20, ws=P(260), wsb=need) == -1
    assert call(B=0) == 0 and call(L=0) == 0


def test_logprobs_grad_refusals(lib):
    def call(logits=fake, dtype=1, B=1, L=1, V=8, stride=8, T=1.0, norm=fake, grad=P(512), gs=8):
        return lib.dllm_token_logprobs_grad(logits, dtype, B, L, V, stride, T, None, 0, fake, norm,
                                            fake, None, None, grad, gs, None)

    assert call(dtype=9) == -2
    for bad in (dict(gs=7), dict(norm=None), dict(grad=None), dict(grad=P(513)), dict(T=0.0),
                dict(V=0), dict(grad=fake, gs=16)):
        assert call(**bad) == -1, bad
    assert call(B=0) == 0


def _c(k=256, v=512, ks=1024, vs=2048, pages=4, heads=2, dim=64):
    return ctypes.byref(dc._CCache(k, v, ks, vs, pages, heads, dim))


BAD_CACHES = [(dict(k=None), -1), (dict(v=None), -1), (dict(ks=None), -1), (dict(vs=None), -1),
              (dict(k=8), -1), (dict(v=8), -1), (dict(ks=2), -1), (dict(pages=0), -1),
              (dict(pages=1 << 31), -1), (dict(heads=0), -1), (dict(dim=96), -5), (dict(dim=0), -5)]


def test_kv_refusals(lib):
    def write(c=None, k=fake, v=fake, B=1, L=1, table=fake, pages=2, stride=2, start=fake):
        return lib.dllm_kv_write(c if c is not None else _c(), k, S3, v, S3, B, L, table, pages,
                                 stride, start, None, None)

    def read(c=None, B=1, pages=2, stride=2, lens=fake, k=fake, v=fake, table=fake):
        return lib.dllm_kv_read(c if c is not None else _c(), B, table, pages, stride, lens, k, v,
                                None)

    def gather(c=None, B=1, pages=2, stride=2, kept=fake, ks=4, counts=fake, new=P(512), np_=2,
               ns=2):
        return lib.dllm_kv_gather(c if c is not None else _c(), B, fake, pages, stride, kept, ks,
                                  counts, new, np_, ns, None)

    for f in (write, read, gather):
        for bad, status in BAD_CACHES:
            assert f(c=_c(**bad)) == status, (f, bad)
        assert f(B=-1) == -1 and f(pages=-1) == -1 and f(pages=1 << 26, stride=1 << 26) == -1
        assert f(stride=1) == -1 and "stride" in _err(lib)
        assert f(B=0) == 0
        assert f(B=1 << 30) == -5
    assert lib.dllm_kv_write(None, fake, S3, fake, S3, 1, 1, fake, 2, 2, fake, None, None) == -1
    for bad in (dict(L=-1), dict(k=None), dict(v=None), dict(k=P(257)), dict(start=None),
                dict(table=None), dict(table=P(258))):
        assert write(**bad) == -1, bad
    assert write(L=0) == 0 and write(pages=0, stride=0, table=None) == 0
    for bad in (dict(lens=None), dict(k=None), dict(v=None), dict(k=P(264)), dict(table=None)):
        assert read(**bad) == -1, bad
    for bad in (dict(kept=None), dict(counts=None), dict(ks=-1), dict(new=fake), dict(new=None),
                dict(np_=-1), dict(ns=1)):
        assert gather(**bad) == -1, bad
    assert gather(np_=0, ns=0) == 0


def test_attention_refusals(lib):
    def attend(c=None, q=fake, B=1, L=1, Hq=4, table=fake, pages=2, stride=2, lens=fake, bl=0,
               scale=0.1, out=P(512), lse=fake, ws=None, wsb=0):
        return lib.dllm_block_attention(c if c is not None else _c(), q, S3, B, L, Hq, table, pages,
                                        stride, lens, None, None, bl, scale, out, S3, lse, ws, wsb,
                                        None)

    def weigh(c=None, q=fake, B=1, L=1, Hq=4, table=fake, pages=2, stride=2, lens=fake, bl=0,
              scale=0.1, lse=fake, weights=fake, ws=fake, wsb=1 << 40):
        return lib.dllm_attention_weights(c if c is not None else _c(), q, S3, B, L, Hq, table,
                                          pages, stride, lens, None, None, bl, scale, lse, weights,
                                          ws, wsb, None)

    for f in (attend, weigh):
        for bad, status in BAD_CACHES:
            assert f(c=_c(**bad)) == status, (f, bad)
        for bad in (dict(B=-1), dict(L=-1), dict(Hq=3), dict(Hq=0), dict(bl=-1), dict(bl=1 << 31),
                    dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf),
                    dict(scale=2e38),
                    dict(q=None), dict(q=P(257)), dict(lens=None), dict(table=None),
                    dict(stride=1), dict(pages=1 << 26, stride=1 << 26), dict(lse=None)):
            assert f(**bad) == -1, (f, bad)
        assert f(B=0) == 0 and f(L=0) == 0
        assert f(L=1 << 30) == -5
    assert attend(out=None) == -1 and attend(out=fake) == -1 and attend(out=P(513)) == -1
    assert weigh(weights=None) == -1
    need = lib.dllm_attention_weights_workspace_size(1, 1, 4, 2, 2)
    assert weigh(ws=None) == -3 and weigh(wsb=need - 1) == -3 and weigh(ws=P(260)) == -1
    assert lib.dllm_attention_weights_workspace_size(1, 1, 4, 3, 2) == 0
    need = lib.dllm_block_attention_workspace_size(1, 1, 4, 2, 64, 1000)
    assert need > 0 and attend(pages=1000, stride=1000, ws=fake, wsb=need - 1) == -3
    assert attend(pages=1000, stride=1000, ws=P(260), wsb=need) == -1
    assert lib.dllm_block_attention_workspace_size(1, 1, 4, 3, 64, 10) == 0
    big = 1 << 62                                     # products that would not fit
    assert lib.dllm_block_attention_workspace_size(big, big, 4, 2, 64, 10) == 0
    assert lib.dllm_attention_weights_workspace_size(1, 1, 4, 2, big) == 0
    assert lib.dllm_token_logprobs_workspace_size(1, big, big, 8, 1) == 0
    wide = (ctypes.c_int64 * 3)(1 << 40, 1 << 33, 64)
    assert lib.dllm_block_attention(_c(), fake, wide, 1, 1, 4, fake, 2, 2, fake, None, None, 0, 0.1,
                                    P(512), S3, fake, None, 0, None) == -5
    assert lib.dllm_block_attention_workspace_size(1, 1, 4, 2, 80, 10) == 0


def test_evict_select_refusals(lib):
    def call(w=fake, B=1, T=100, stride=100, lens=fake, budget=10, sink=2, recent=3, kept=fake,
             nl=fake, nw=P(512), nT=10):
        return lib.dllm_evict_select(w, B, T, stride, lens, budget, sink, recent, kept, nl, nw, nT,
                                     None)

    for bad in (dict(B=-1), dict(T=-1), dict(T=(1 << 31) - 1, stride=1 << 31), dict(stride=99),
                dict(budget=0), dict(budget=1 << 31), dict(sink=-1), dict(recent=-1),
                dict(sink=8, recent=3), dict(sink=11), dict(nT=9), dict(w=None), dict(lens=None),
                dict(kept=None), dict(nl=None), dict(nw=fake)):
        assert call(**bad) == -1, bad
    assert call(B=1 << 30) == -5 and call(B=0) == 0


def test_binding_refuses_cpu_tensors():
    x = torch.zeros((1, 1, 8))
    t = torch.zeros((1, 1), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        dc.token_logprobs(x, t)
    with pytest.raises(ValueError, match="CUDA"):
        dc.token_logprobs(x.requires_grad_(), t)
    cache = dc.KVCache(2, 1, 64, device="cpu")
    z = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        dc.kv_write(cache, z, z, torch.zeros((1, 2), dtype=torch.int32), t[0])
    with pytest.raises(ValueError, match="CUDA"):
        dc.block_attention(z, cache, torch.zeros((1, 2), dtype=torch.int32), t[0])
    with pytest.raises(ValueError, match="CUDA"):
        dc.evict_select(torch.zeros((1, 8)), t[0], 4)
    with pytest.raises(ValueError, match="KVCache"):
        dc.kv_read(None, torch.zeros((1, 2), dtype=torch.int32), t[0])
    for bad in (dict(num_pages=0), dict(kv_heads=0), dict(head_dim=96)):
        with pytest.raises(ValueError):
            dc.KVCache(**{**dict(num_pages=1, kv_heads=1, head_dim=64, device="cpu"), **bad})


def test_outputs_that_share_memory_are_refused():
    x = torch.zeros(2, 3, 4, 8)
    for good in (x, x.transpose(1, 2), x[..., 1:5], x[:, ::2], x[:1].expand(1, 3, 4, 8),
                 x.permute(3, 2, 1, 0), x[:, :0]):
        dc._apart(good, "out")
    for bad in (x[:1].expand(2, 3, 4, 8), x[:, :, :1].expand(2, 3, 4, 8),
                torch.as_strided(x, (2, 3, 4, 8), (96, 8, 8, 1)), x[..., :1].expand(2, 3, 4, 8)):
        with pytest.raises(ValueError, match="share memory"):
            dc._apart(bad, "out")


def test_pool_memory_cannot_be_exchanged():
    """The calls hold the pool's addresses: a new tensor in its place would leave
    them pointing at freed memory."""
    cache = dc.KVCache(2, 1, 64, device="cpu")
    for name in ("k", "v", "k_scale", "v_scale"):
        with pytest.raises(AttributeError):
            setattr(cache, name, getattr(cache, name).clone())


@pytest.mark.parametrize("d", [1, 2, 3, 5, 7, 28, 31, 32, 33, 641, 2 ** 16, 2 ** 30 + 1, 2 ** 31 - 1])
def test_division_by_multiplication(d):
    """The kernels' n / d for n < 2^31 (columns by heads of a group, positions by
    block length): the formula in attention.hip, in Python's integers."""
    s = 0
    while s < 31 and (1 << s) < d:
        s += 1
    m = ((((1 << s) - d) << 32) // d + 1) & 0xffffffff
    ns = {0, 1, d - 1, d, d + 1, 2 ** 31 - 1, 2 ** 31 - 2}
    ns |= {k * d + e for k in (2, 3, 1000, (2 ** 31 - 1) // d) for e in (-1, 0, 1)}
    for n in ns:
        if 0 <= n < 2 ** 31:
            total = ((n * m) >> 32) + n
            assert total < 2 ** 32 and total >> s == n // d


SOURCES = ["logprobs.hip", "kv_cache.hip", "attention.hip", "evict.hip"]


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
@pytest.mark.parametrize("src", SOURCES)
def test_no_scratch_and_lds_within_the_limit(src, tmp_path):
    from commit_step_amd.build import FLAGS
    flags = [f for f in FLAGS if f not in ("-shared", "-fPIC")]
    out = tmp_path / (src + ".s")
    subprocess.run([HIPCC, *flags, "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    "--cuda-device-only", "-S", "-o", str(out), os.path.join(CSRC, src)],
                   check=True, capture_output=True)
    kernels = _parse(str(out))
    assert kernels
    for name, r in kernels.items():
        assert r["private_segment_fixed_size"] == 0, f"{name} uses scratch: {r}"
        assert r["group_segment_fixed_size"] <= LDS_LIMIT, f"{name}: {r}"
