"""GPU parity of token_logprobs and its gradient against the float64 oracle.

Tolerances.  u = 2^-24.  Every sum over the vocabulary has at most
n = ceil(V / 256) + 64 roundings in a row (a lane's share, then the lanes), and
each term 2^d carries |d| u + 2 ulp from its exponent, |d| <= 200: a relative
error of at most (n + 300) u on sums of terms of one sign.  log p_t adds three
roundings of (x - M) / T.  A probability recomputed by the gradient carries the
same, and the result is rounded once to the logits' type (half a step)."""
import numpy as np
import pytest
import torch

import commit_step_amd as dc
from gpu_util import to_dev
from oracle import scores

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _make(seed, B, L, V, dtype, off=0.4, sigma=2.5, stride=None):
    """Logits on the device (rows `stride` apart), their exact float64 values,
    targets with a share not scored."""
    rng = np.random.default_rng(seed)
    stride = V if stride is None else stride
    x = torch.from_numpy(rng.normal(0, sigma, (B, L, stride)).astype(np.float32)).to(DT[dtype])
    t = rng.integers(0, V, (B, L)).astype(np.int32)
    lift = torch.from_numpy((rng.random((B, L)) * 14).astype(np.float32)).to(DT[dtype])
    for b in range(B):
        for l in range(L):
            x[b, l, t[b, l]] += lift[b, l]
    t[rng.random((B, L)) < off] = -1
    dev = x.cuda()[:, :, :V]
    return dev, x[:, :, :V].double().numpy(), t, rng


def _n(V):
    return (-(-V // 256) + 64 + 300) * U


def _check(r, ref, targets, V, T=1.0, top=0, logits=None):
    torch.cuda.synchronize()
    lp, ent = r.logprob.cpu().double().numpy(), r.entropy.cpu().double().numpy()
    fin = np.isfinite(ref.logprob)
    assert np.array_equal(np.isfinite(lp), fin) and (lp[~fin] == ref.logprob[~fin]).all()
    tol = _n(V) * (ref.entropy + 1) + 4 * U * np.where(fin, np.abs(ref.logprob), 0)
    miss = np.abs(lp[fin] - ref.logprob[fin])
    assert (miss <= tol[fin]).all(), miss.max()
    err = np.abs(ent - ref.entropy)
    assert (err <= _n(V) * ref.entropy + 1e-30).all(), (err / (ref.entropy + 1e-30)).max()
    if top:
        assert np.array_equal(r.top_ids.cpu().numpy(), ref.top_ids)
        got = r.top_logprobs.cpu().double().numpy()
        live = np.isfinite(ref.top_logprobs)
        assert (got[~live] == -np.inf).all()
        e = np.abs(got[live] - ref.top_logprobs[live])
        wide = np.broadcast_to(tol[..., None], got.shape)
        assert (e <= wide[live] + 4 * U * np.abs(ref.top_logprobs[live])).all()
    off = (targets < 0) | (targets >= V)
    assert not lp[off].any() and not ent[off].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,L,V,top", [
    (1, 1, 1, 1), (1, 1, 2, 5), (2, 3, 7, 3), (1, 5, 257, 0), (3, 7, 1000, 20), (1, 2, 4099, 32),
    (2, 150, 2056, 1), (1, 1, 50257, 20), (1, 3, 126464, 20), (2, 2, 151937, 5), (2, 140, 8200, 32)])
def test_scores(dtype, B, L, V, top):
    x, exact, t, _ = _make(V + L, B, L, V, dtype)
    r = dc.token_logprobs(x, torch.from_numpy(t).cuda(), top=top)
    _check(r, scores.token_logprobs(exact, t, top=top), t, V, top=top)


@pytest.mark.parametrize("dtype,stride", [("bf16", 1009), ("bf16", 1016), ("f32", 1003), ("f32", 1004)])
@pytest.mark.parametrize("T", [0.5, 1.7])
def test_strides_temperature_suppress(dtype, stride, T):
    V, sup = 1001, (0, 5, 6, 1000, 512)
    x, exact, t, _ = _make(stride, 2, 9, V, dtype, stride=stride)
    t[0, 0], t[0, 1], t[1, 2] = 5, 1000, V          # suppressed targets; one past the end
    r = dc.token_logprobs(x, torch.from_numpy(t).cuda(), temperature=T, suppress_ids=sup, top=6)
    _check(r, scores.token_logprobs(exact, t, T, sup, 6), t, V, T, 6)
    # a base off 16-byte alignment (and, for slices, off it by an odd count)
    y = x[:, :, 1:]
    sup1 = (0, 3)
    t1 = np.where(t > 0, t - 1, t).astype(np.int32)
    r = dc.token_logprobs(y, torch.from_numpy(t1).cuda(), temperature=T, suppress_ids=sup1, top=6)
    _check(r, scores.token_logprobs(exact[:, :, 1:], t1, T, sup1, 6), t1, V - 1, T, 6)


@pytest.mark.parametrize("V", [300, 20000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_degenerate_rows_and_ties(V, dtype):
    rng = np.random.default_rng(V)
    x = torch.from_numpy(rng.normal(0, 2, (1, 9, V)).astype(np.float32)).to(DT[dtype])
    inf = float("inf")
    x[0, 0] = -inf
    x[0, 1] = float("nan")
    x[0, 2, ::3] = float("nan")
    x[0, 3, 7], x[0, 3, V - 1] = inf, inf
    x[0, 4] = torch.finfo(DT[dtype]).min
    x[0, 5] = 1.5                                    # all equal
    x[0, 6] = x[0, 6].round()                        # many ties
    x[0, 7, 2:] = -inf                               # two ids left
    x[0, 8] = torch.arange(V).to(DT[dtype]) / V      # ascending: every chunk raises the list
    t = np.array([[3, 4, 5, 7, 8, 9, 10, 0, V - 1]], dtype=np.int32)
    for sup in ((), (0, 1, V - 1)):
        r = dc.token_logprobs(x.cuda(), torch.from_numpy(t).cuda(), suppress_ids=sup, top=8)
        _check(r, scores.token_logprobs(x.double().numpy(), t, 1.0, sup, 8), t, V, top=8)


def _grad_tol(ref, s, g, h, V, T, dtype):
    p = np.exp(s.logp)
    lp = np.where(p > 0, np.abs(s.logp), 0.0)
    own = torch.finfo(DT[dtype]).eps / 2
    w = p * (np.abs(g)[..., None] + np.abs(h)[..., None] * (lp + s.entropy[..., None] + 1))
    # p and log p: the norm's error and |d| u of the exponent; then the formula's roundings
    rel = _n(V) * (s.entropy + 2)[..., None] + (lp + 8) * 2 * U
    return own * np.abs(ref) + (rel * w + 4 * U * np.abs(ref)) / T * (1 + own) + 1e-38


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,L,V,T,sup,ent", [
    (1, 1, 1, 1.0, (), True), (2, 3, 7, 1.0, (2,), True), (2, 5, 1001, 0.7, (), True),
    (1, 4, 4096, 1.0, (0, 4095), False), (1, 3, 50257, 1.3, (), True), (1, 2, 126464, 1.0, (), True)])
def test_gradient(dtype, B, L, V, T, sup, ent):
    x, exact, t, rng = _make(V, B, L, V, dtype)
    t[0, 0] = V - 1 if t[0, 0] < 0 else t[0, 0]
    g, h = rng.normal(size=(B, L)), rng.normal(size=(B, L)) * ent
    tg, th = (torch.from_numpy(a.astype(np.float32)).cuda() for a in (g, h))
    g, h = g.astype(np.float32).astype(np.float64), h.astype(np.float32).astype(np.float64)
    xr = x.detach().requires_grad_(True)
    r = dc.token_logprobs(xr, torch.from_numpy(t).cuda(), temperature=T, suppress_ids=sup, top=2)
    assert r.logprob.requires_grad and r.entropy.requires_grad
    assert not r.top_logprobs.requires_grad and not r.norm.requires_grad
    outs, gs = ((r.logprob, r.entropy), (tg, th)) if ent else ((r.logprob,), (tg,))
    (gx,) = torch.autograd.grad(outs, (xr,), gs)
    assert gx.dtype == x.dtype
    s = scores.token_logprobs(exact, t, T, sup)
    ref = scores.token_logprobs_grad(s, t, g, h, T, sup)
    got = gx.cpu().double().numpy()
    err, tol = np.abs(got - ref), _grad_tol(ref, s, g, h, V, T, dtype)
    assert (err <= tol).all(), (err / tol).max()
    assert not got[(t < 0) | (t >= V)].any() and not got[..., list(sup)].any()
    # the same through the raw call, in place over a copy of the logits
    y = x.detach().clone()
    raw = dc.token_logprobs_grad(y, torch.from_numpy(t).cuda(), r.norm, r.entropy.detach(), tg,
                                 th if ent else None, temperature=T, suppress_ids=sup, out=y)
    assert raw is y and torch.equal(y, gx)


def test_gradient_strides_and_degenerate_rows():
    V = 515
    x, exact, t, rng = _make(3, 2, 4, V, "bf16", off=0.0, stride=521)
    buf = torch.zeros((2, 4, 530), dtype=torch.bfloat16, device="cuda")
    out = buf[:, :, 3:3 + V]                          # aligned unlike the logits
    tt = torch.from_numpy(t).cuda()
    g = torch.ones((2, 4), device="cuda")
    r = dc.token_logprobs(x, tt)
    dc.token_logprobs_grad(x, tt, r.norm, r.entropy, g, None, out=out)
    s = scores.token_logprobs(exact, t)
    one = np.ones((2, 4))
    ref = scores.token_logprobs_grad(s, t, one, 0 * one)
    err = np.abs(out.cpu().double().numpy() - ref)
    assert (err <= _grad_tol(ref, s, one, 0 * one, V, 1.0, "bf16")).all()
    assert not buf[:, :, :3].any() and not buf[:, :, 3 + V:].any()
    y = torch.zeros((1, 3, 64), device="cuda")
    y[0, 0] = -float("inf")
    y[0, 1, 5] = y[0, 1, 9] = float("inf")
    y[0, 2, 3] = float("nan")
    yr = y.requires_grad_(True)
    t3 = torch.tensor([[1, 5, 2]], dtype=torch.int32, device="cuda")
    r = dc.token_logprobs(yr, t3)
    (gy,) = torch.autograd.grad((r.logprob, r.entropy), (yr,), (torch.ones_like(r.logprob),) * 2)
    s = scores.token_logprobs(y.detach().cpu().double().numpy(), t3.cpu().numpy())
    ref = scores.token_logprobs_grad(s, t3.cpu().numpy(), np.ones((1, 3)), np.ones((1, 3)))
    assert np.abs(gy.cpu().double().numpy() - ref).max() <= 1e-5


def test_saved_inputs_are_guarded_and_second_order_is_refused():
    x = torch.randn((1, 2, 50), device="cuda", requires_grad=True)
    t = torch.tensor([[1, 2]], dtype=torch.int32, device="cuda")
    r = dc.token_logprobs(x, t)
    (g,) = torch.autograd.grad(r.logprob.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
    z = x.detach().clone().requires_grad_(True)
    y = z * 1.0
    r = dc.token_logprobs(y, t)
    y.mul_(2.0)
    with pytest.raises(RuntimeError, match="modified"):
        r.logprob.sum().backward()
    y = z * 1.0
    r = dc.token_logprobs(y, t)
    with torch.no_grad():                              # the gradient written over the logits
        dc.token_logprobs_grad(y, t, r.norm, r.entropy.detach(), torch.ones((1, 2), device="cuda"), out=y)
    with pytest.raises(RuntimeError, match="modified"):
        r.logprob.sum().backward()


def test_strided_upstream_gradients_and_unused_outputs():
    x = torch.randn((2, 3, 40), device="cuda", requires_grad=True)
    t = torch.ones((2, 3), dtype=torch.int32, device="cuda")
    dc.token_logprobs(x, t).logprob.sum().backward()          # an expanded gradient
    want = x.grad.clone()
    x.grad = None
    torch.log_softmax(x, -1)[:, :, 1].sum().backward()
    # p carries (n + 300) u; both sides round once more
    assert (want - x.grad).abs().max() <= 2 * _n(40) * 4
    x.grad = None
    dc.token_logprobs(x, t).entropy.sum().backward()
    p = torch.softmax(x.detach().double(), -1)
    H = -(p * p.log()).sum(-1, keepdim=True)
    assert (x.grad + p * (p.log() + H)).abs().max() <= 2 * _n(40) * 8


def test_other_stream_and_graph():
    x, exact, t, _ = _make(11, 1, 3, 126464, "bf16", off=0.0)     # split rows: a workspace
    tt = torch.from_numpy(t).cuda()
    want = dc.token_logprobs(x, tt, top=4)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other = dc.token_logprobs(x, tt, top=4)
    torch.cuda.current_stream().wait_stream(st)
    for a, b in zip(want, other):
        assert torch.equal(a, b)
    # forward and backward captured: leaves, then replays against eager
    xs = x.clone().requires_grad_(True)
    gl = torch.ones((1, 3), device="cuda")

    def step():
        # no autograd graph outlives the call: one kept alive would be met again
        # by the capture of the same leaf
        r = dc.token_logprobs(xs, tt, top=4)
        g = torch.autograd.grad((r.logprob, r.entropy), (xs,), (gl, gl))[0]
        return [t.detach() for t in r], g

    with torch.cuda.stream(st):
        step()
    torch.cuda.synchronize()
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, gx = step()
    with torch.cuda.graph(second):
        r2, gx2 = step()
    for i in range(4):
        with torch.no_grad():
            xs.copy_(torch.roll(x, 17 * i, dims=2))
        er, eg = step()
        dc.token_logprobs(x, tt, top=2)                # eager work on the stream's workspace
        graph.replay()
        with torch.cuda.stream(st):                    # two graphs side by side
            st.wait_stream(torch.cuda.current_stream())
            second.replay()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(er, r, r2):
            assert torch.equal(a, b) and torch.equal(a, c)
        assert torch.equal(eg, gx) and torch.equal(eg, gx2)


def test_captured_backward_beside_a_living_graph_of_the_leaf():
    x = torch.randn((1, 2, 300), device="cuda", requires_grad=True)
    t = torch.tensor([[5, -1]], dtype=torch.int32, device="cuda")
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()

    def step():
        return torch.autograd.grad(dc.token_logprobs(x, t).logprob.sum(), x)[0]

    alive = dc.token_logprobs(x, t)                    # on the current stream
    want = torch.autograd.grad(alive.logprob.sum(), x, retain_graph=True)[0]
    with torch.cuda.stream(st):
        assert torch.equal(step(), want)               # eager: streams may differ
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        with pytest.raises(RuntimeError, match="lives on another stream"):
            dc.token_logprobs(x, t)
        dc.token_logprobs(x.detach(), t)               # no backward pass: no tie
    del alive
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        got = step()
    for _ in range(3):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_refusals_on_the_device():
    x = torch.zeros((1, 2, 40), device="cuda")
    t = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    for bad in (dict(targets=t.long()), dict(targets=t[:, :1]), dict(targets=t.cpu()),
                dict(logits=x.half()), dict(logits=x[0]), dict(logits=x[:, :, ::2]), dict(top=33),
                dict(temperature=0.0), dict(suppress_ids=(40,))):
        with pytest.raises(ValueError):
            dc.token_logprobs(**{**dict(logits=x, targets=t), **bad})
    big = torch.zeros((1, 1, 126464), device="cuda")
    with pytest.raises(ValueError, match="workspace"):
        dc.token_logprobs(big, t[:, :1].contiguous(), top=4,
                          workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    # empty batches
    r = dc.token_logprobs(x[:, :0], t[:, :0].contiguous(), top=3)
    assert r.logprob.shape == (1, 0) and r.top_ids.shape == (1, 0, 3)
