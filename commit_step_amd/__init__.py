"""Python binding of libdllm_commit (the dLLM commit step on MI355X).

Argument marshalling only: every step of the computation runs in the HIP
library ``libdllm_commit.so`` next to this file.  PyTorch provides device
memory and the current stream.  There is no CPU fallback: if the library is
not built, every call raises.

Names and keyword arguments follow mlx-arsenal's ``mlx_arsenal.diffusion``
functions ("dLLM block decoding", "What mlx-arsenal ships"): token_stats,
threshold_transfer, topk_transfer, factor_transfer, entropy_bound_transfer,
edit_transfer, transfer_schedule, block_ranges, block_causal_mask.  Around the
step: token_logprobs (scores of given tokens, differentiable), and the 8-bit
key/value cache of block decoding (KVCache, kv_write, kv_read, block_attention,
kv_evict).
"""
import contextlib
import ctypes
import math
import os
from collections import namedtuple

import torch

__all__ = ["Stats", "Rule", "token_stats", "threshold_transfer", "topk_transfer",
           "factor_transfer", "entropy_bound_transfer", "edit_transfer",
           "transfer_schedule", "block_ranges", "block_causal_mask",
           "workspace_size", "library_path", "load_library", "commit_step", "CommitStep",
           "linear_temperature", "uniform_canvas", "renoise", "StableConfidentStopping",
           "decaying_threshold", "Logprobs", "token_logprobs", "token_logprobs_grad", "KVCache",
           "kv_write", "kv_read", "Attention", "block_attention", "Evicted",
           "evict_select", "kv_gather", "kv_evict", "KV_PAGE"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libdllm_commit.so")

DLLM_F32, DLLM_BF16 = 0, 1
RULE_THRESHOLD, RULE_TOPK, RULE_FACTOR, RULE_ENTROPY_BOUND, RULE_EDIT = 1, 2, 3, 4, 5
SCORE_PROB, SCORE_MARGIN, SCORE_NEG_ENTROPY = 0, 1, 2
_SCORES = {"prob": SCORE_PROB, "margin": SCORE_MARGIN, "neg_entropy": SCORE_NEG_ENTROPY}
MAX_L = 4096
MAX_SUPPRESS = 64
MAX_TOP = 32
KV_PAGE = 32

Stats = namedtuple("Stats", ["x0", "prob", "entropy", "margin", "argmax"])
CommitStep = namedtuple("CommitStep", ["stats", "counts"])
Logprobs = namedtuple("Logprobs", ["logprob", "entropy", "top_ids", "top_logprobs", "norm"])
Attention = namedtuple("Attention", ["out", "lse"])
Evicted = namedtuple("Evicted", ["kept", "lens", "weights"])


class _CRule(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("mask", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("param", ctypes.c_double), ("strict", ctypes.c_int),
                ("k", ctypes.c_void_p), ("tokens", ctypes.c_void_p), ("score", ctypes.c_int),
                ("taus", ctypes.c_void_p)]


class _CStatsExtra(ctypes.Structure):
    _fields_ = [("margin", ctypes.c_void_p), ("argmax", ctypes.c_void_p),
                ("stats_temperature", ctypes.c_float)]


class _CCanvas(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("skip_rows", ctypes.c_int)]


class _CCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


_lib = None

# The exported C entry points and their signatures (include/dllm_commit.h).
_I64, _I32, _P = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
_SIGNATURES = {
    "dllm_token_stats": (_I32, [_P, _I32, _I64, _I64, _I64, _I64, ctypes.c_float, ctypes.c_uint64,
                                ctypes.c_uint64, _P, _I32, _P, _P, _P, _P, _P, _I32, _P,
                                ctypes.c_size_t, _P]),
    "dllm_token_stats_workspace_size": (ctypes.c_size_t, [_I32, _I64, _I64, _I64]),
    "dllm_commit_step": (_I32, [_P, _I32, _I64, _I64, _I64, _I64, ctypes.c_float, ctypes.c_uint64,
                                ctypes.c_uint64, _P, _I32, _P, _P, _P, _P, _P, _I32, _P, _P,
                                ctypes.c_size_t, _P]),
    "dllm_commit_step_static": (_I32, [_P, _I32, _I64, _I64, _I64, _I64, ctypes.c_float,
                                       ctypes.c_uint64, ctypes.c_uint64, _P, _I32, _P, _P, _P, _P,
                                       _P, _I32, _P, _P]),
    "dllm_transfer_threshold": (_I32, [_P, _P, _I64, _I64, ctypes.c_double, _I32, _P, _P]),
    "dllm_transfer_threshold_rows": (_I32, [_P, _P, _P, _I64, _I64, _I32, _P, _P]),
    "dllm_decaying_threshold": (_I32, [ctypes.c_double, ctypes.c_double, ctypes.c_double, _I64,
                                       ctypes.POINTER(ctypes.c_double)]),
    "dllm_transfer_topk": (_I32, [_P, _P, _P, _I64, _I64, _P, _P]),
    "dllm_transfer_factor": (_I32, [_P, _P, _I64, _I64, ctypes.c_double, _P, _P]),
    "dllm_transfer_entropy_bound": (_I32, [_P, _P, _I64, _I64, ctypes.c_double, _P, _P]),
    "dllm_transfer_edit": (_I32, [_P, _P, _P, _P, _I64, _I64, ctypes.c_double, _P, _P]),
    "dllm_transfer_schedule": (_I32, [_P, _I64, ctypes.c_int32, _P, _P]),
    "dllm_block_ranges": (_I64, [_I64, _I64, _I64, _I32, _P, _I64]),
    "dllm_block_causal_mask": (_I32, [_I64, _I64, _P, _P]),
    "dllm_linear_temperature": (_I32, [_I32, _I32, ctypes.c_double, ctypes.c_double,
                                       ctypes.POINTER(ctypes.c_double)]),
    "dllm_uniform_canvas": (_I32, [_P, _I64, _I64, _I64, ctypes.c_uint64, ctypes.c_uint64, _P]),
    "dllm_renoise": (_I32, [_P, _P, _P, _I64, _I64, _P, _P]),
    "dllm_stable_confident_stop": (_I32, [_P, _P, _I64, _I64, _I32, ctypes.c_double, _I32, _P, _P,
                                          _P, _P]),
    "dllm_token_logprobs": (_I32, [_P, _I32, _I64, _I64, _I64, _I64, ctypes.c_float, _P, _I32, _P,
                                   _I32, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "dllm_token_logprobs_workspace_size": (ctypes.c_size_t, [_I32, _I64, _I64, _I64, _I32]),
    "dllm_token_logprobs_grad": (_I32, [_P, _I32, _I64, _I64, _I64, _I64, ctypes.c_float, _P, _I32,
                                        _P, _P, _P, _P, _P, _P, _I64, _P]),
    "dllm_kv_write": (_I32, [_P, _P, _P, _P, _P, _I64, _I64, _P, _I64, _I64, _P, _P, _P]),
    "dllm_kv_read": (_I32, [_P, _I64, _P, _I64, _I64, _P, _P, _P, _P]),
    "dllm_block_attention": (_I32, [_P, _P, _P, _I64, _I64, _I64, _P, _I64, _I64, _P, _P, _P, _I64,
                                    ctypes.c_float, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "dllm_block_attention_workspace_size": (ctypes.c_size_t, [_I64, _I64, _I64, _I64, _I64, _I64]),
    "dllm_attention_weights": (_I32, [_P, _P, _P, _I64, _I64, _I64, _P, _I64, _I64, _P, _P, _P,
                                      _I64, ctypes.c_float, _P, _P, _P, ctypes.c_size_t, _P]),
    "dllm_attention_weights_workspace_size": (ctypes.c_size_t, [_I64, _I64, _I64, _I64, _I64]),
    "dllm_evict_select": (_I32, [_P, _I64, _I64, _I64, _P, _I64, _I64, _I64, _P, _P, _P, _I64, _P]),
    "dllm_kv_gather": (_I32, [_P, _I64, _P, _I64, _I64, _P, _I64, _P, _P, _I64, _I64, _P]),
    "dllm_read_probe": (_I32, [_P, _I64, _I64, _I32, _P, _P]),
    "dllm_stage_timestamps": (_I32, [_P, ctypes.c_size_t, _I32]),
    "dllm_last_error": (ctypes.c_char_p, []),
}


def library_path():
    return _LIB_PATH


_STAGES_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdllm_commit_stages.so")
_lib_stages = None


def _open(path):
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


def load_library(stages=False):
    """Load libdllm_commit.so (raises if it has not been built).  stages=True
    loads libdllm_commit_stages.so instead, the same library with stage
    timestamps on (for commit_step_amd.stage_timing only)."""
    global _lib, _lib_stages
    if stages:
        if _lib_stages is None:
            if not os.path.exists(_STAGES_PATH):
                raise RuntimeError(f"{_STAGES_PATH} is not built; run "
                                   "`python -m commit_step_amd.build --stages`")
            _lib_stages = _open(_STAGES_PATH)
        return _lib_stages
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is not built; run `python -m commit_step_amd.build`")
        _lib = _open(_LIB_PATH)
    return _lib


def _check(status, what):
    if status < 0:
        msg = load_library().dllm_last_error().decode(errors="replace")
        raise ValueError(f"{what} failed with status {status}: {msg}")
    return status


def _stream(t):
    return torch.cuda.current_stream(t.device).cuda_stream


def _dev(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    return t


def _bl(t, name, dtypes, shape=None):
    _dev(t, name)
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must have dtype in {dtypes}, not {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    return t


def _on(device):
    """The device's context, skipped when it is already the current device
    (entering it costs more host time than the launch itself)."""
    if device.index is None or device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


_ws_sizes = {}


def _ws_size(dt, B, L, V, device):
    key = (dt, B, L, V, device.index)
    n = _ws_sizes.get(key)
    if n is None:
        n = int(load_library().dllm_token_stats_workspace_size(dt, B, L, V))
        _ws_sizes[key] = n
    return n


# commit_step(..., workspace=STATIC_WORKSPACE) runs dllm_commit_step_static: no
# workspace tensor, no allocation (the library's own per-GPU array; calls that
# overlap on one GPU race).
STATIC_WORKSPACE = "static"
_MASK_DTYPES = (torch.bool, torch.uint8)
_workspaces = {}


def workspace_size(logits):
    B, L, V = logits.shape
    dt = DLLM_BF16 if logits.dtype == torch.bfloat16 else DLLM_F32
    with _on(logits.device):
        return int(load_library().dllm_token_stats_workspace_size(dt, B, L, V))


def _capturing(device):
    return device.type == "cuda" and torch.cuda.is_current_stream_capturing()


def _workspace(device, stream, nbytes):
    """The default workspace: a zero-filled byte buffer per (device, stream),
    grown on demand.  The library leaves it zero-filled after every
    successful call.  Calls in flight at the same time must not share a
    workspace (their row and batch-row counters would mix), and calls on one
    stream never overlap, so one buffer per stream is safe.  A buffer cannot
    be created or grown while the stream is being captured into a graph (the
    zero fill would become a node of the graph): make one eager call of the
    same or a larger shape first, or pass ``workspace=``."""
    key = (device.type, device.index, stream)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        if _capturing(device):
            raise RuntimeError(
                "the default workspace of this stream has to be created or grown during graph "
                "capture; make one eager call of this shape on the stream first, or pass "
                "workspace= (zero-filled, workspace_size() bytes)")
        ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


class Rule:
    """A commit rule fused into token_stats (same launch).

    Build with Rule.threshold / topk / factor / entropy_bound / edit; the
    result lands in ``rule.out`` (a bool (B, L) tensor).
    """

    def __init__(self, kind, mask, param=0.0, strict=False, k=None, tokens=None, out=None,
                 score="prob"):
        if score not in _SCORES:
            raise ValueError(f"score must be one of {sorted(_SCORES)}")
        self.taus = param if isinstance(param, torch.Tensor) else None
        if self.taus is not None and kind != RULE_THRESHOLD:
            raise ValueError("only the threshold rule takes one threshold per row")
        self.param = 0.0 if self.taus is not None else float(param)
        self.kind, self.mask, self.strict = kind, mask, bool(strict)
        self.k, self.tokens, self.out, self.score = k, tokens, out, _SCORES[score]

    @classmethod
    def threshold(cls, candidates, tau, strict=False, score="prob"):
        """score: "prob" (LLaDA, maskgit_plus), "margin" (topk_margin) or
        "neg_entropy" (Dream's entropy confidence).  tau: a number, or a (B,)
        float64 device tensor with one threshold per batch row."""
        return cls(RULE_THRESHOLD, candidates, tau, strict=strict, score=score)

    @classmethod
    def topk(cls, candidates, k, score="prob"):
        return cls(RULE_TOPK, candidates, k=k, score=score)

    @classmethod
    def factor(cls, candidates, f, score="prob"):
        return cls(RULE_FACTOR, candidates, f, score=score)

    @classmethod
    def entropy_bound(cls, candidates, gamma):
        return cls(RULE_ENTROPY_BOUND, candidates, gamma)

    @classmethod
    def edit(cls, editable, tokens, tau_edit):
        """tokens: the current canvas (may be None inside commit_step, which
        passes its own canvas)."""
        return cls(RULE_EDIT, editable, tau_edit, tokens=tokens)


def _k_tensor(k, B, device):
    if isinstance(k, torch.Tensor):
        return _bl(k, "k", (torch.int32,), (B,))
    return torch.full((B,), int(k), dtype=torch.int32, device=device)


def _row_stride(logits):
    """Elements between consecutive positions of (B, L, V) logits.  Sizes 0 and
    1 carry no stride information; otherwise the rows must be unit-stride and
    evenly spaced (position (b, l) at (b * L + l) * row_stride)."""
    B, L, V = logits.shape
    if B * L * V == 0:
        return max(V, 1)
    if V > 1 and logits.stride(2) != 1:
        raise ValueError("logits rows must be contiguous (unit stride along V)")
    if L > 1:
        rs = logits.stride(1)
    elif B > 1:
        rs = logits.stride(0)
    else:
        rs = V
    if B > 1 and logits.stride(0) != L * rs:
        raise ValueError("logits positions must be evenly strided: stride(0) == L * stride(1)")
    if rs < V:
        raise ValueError("logits rows overlap (row stride < V)")
    return rs


def token_stats(logits, temperature=0.0, seed=None, step=0, suppress_ids=(), rules=(),
                out=None, workspace=None, margin=False, argmax=False, stats_temperature=None):
    """Per-position (x0, prob, entropy, margin) of (B, L, V) float32 / bfloat16 logits.

    temperature > 0 draws x0 by Gumbel-max and then needs an explicit ``seed``
    (an integer key; ``step`` selects the per-step noise).  ``rules`` is a list
    of up to two Rule objects run in the same launch; their ``out`` tensors
    are filled.  ``margin`` (or a rule ranking by margin) adds the topk_margin
    confidence p1 - p2; otherwise Stats.margin is None.  ``argmax`` adds the
    greedy argmax (useful when x0 is sampled).  ``stats_temperature`` Ts makes
    prob / entropy / margin those of softmax(logits / Ts).  ``out`` may give
    preallocated (x0, prob, entropy[, margin]) tensors.
    """
    return _stats_call(logits, temperature, seed, step, suppress_ids, rules, out, workspace,
                       None, margin, argmax, stats_temperature)


def commit_step(logits, tokens, rules, temperature=0.0, seed=None, step=0, suppress_ids=(),
                skip_rows=True, counts=True, out=None, workspace=None, margin=False, argmax=False,
                stats_temperature=None):
    """One step of the decoding loop in one launch: token_stats with up to one
    ranking rule and one edit rule, then ``tokens`` (B, L) int32 is updated in
    place to x0 wherever a position was committed or edited.

    With ``skip_rows`` the logits of positions that no rule looks at are not
    read (their x0 / prob / entropy are left as they were).  ``counts`` (True,
    or a preallocated (B, 2) int32 tensor, device or pinned host) receives per
    batch row the candidates left uncommitted and the positions edited.
    ``workspace``: None (the stream's default buffer), a zero-filled uint8
    tensor of workspace_size() bytes, or STATIC_WORKSPACE (the library's own
    per-GPU array, no allocation; shapes up to DLLM_STATIC_SCRATCH_BYTES of
    workspace; calls that overlap on one GPU race).
    Returns CommitStep(stats, counts).
    """
    B, L = logits.shape[0], logits.shape[1]
    if tokens is not None:
        _bl(tokens, "tokens", (torch.int32,), (B, L))
    if counts is True:
        counts = torch.empty((B, 2), dtype=torch.int32, device=logits.device)
    elif counts is False:
        counts = None
    if counts is not None:
        if counts.dtype != torch.int32 or tuple(counts.shape) != (B, 2) or not counts.is_contiguous():
            raise ValueError("counts must be a contiguous (B, 2) int32 tensor")
        if not (counts.is_cuda or counts.is_pinned()):
            raise ValueError("counts must be device memory or pinned host memory")
    canvas = _CCanvas()
    canvas.tokens = tokens.data_ptr() if tokens is not None else None
    canvas.counts = counts.data_ptr() if counts is not None else None
    canvas.skip_rows = int(bool(skip_rows))
    stats = _stats_call(logits, temperature, seed, step, suppress_ids, rules, out, workspace,
                        (canvas, tokens, counts), margin, argmax, stats_temperature)
    return CommitStep(stats, counts)


def _stats_call(logits, temperature, seed, step, suppress_ids, rules, out, workspace, canvas,
                margin, argmax=False, stats_temperature=None):
    _dev(logits, "logits")
    if logits.dim() != 3:
        raise ValueError("logits must be (B, L, V)")
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("logits must be float32 or bfloat16")
    B, L, V = logits.shape
    row_stride = _row_stride(logits)
    if temperature > 0 and seed is None:
        raise ValueError("sampling (temperature > 0) needs an explicit seed")
    dev = logits.device
    want_margin = bool(margin) or any(getattr(r, "score", 0) == SCORE_MARGIN for r in rules)
    mar = None
    if out is None:
        x0 = torch.empty((B, L), dtype=torch.int32, device=dev)
        prob = torch.empty((B, L), dtype=torch.float32, device=dev)
        ent = torch.empty((B, L), dtype=torch.float32, device=dev)
    else:
        x0, prob, ent = out[0], out[1], out[2]
        mar = out[3] if len(out) > 3 else None
        _bl(x0, "x0", (torch.int32,), (B, L))
        _bl(prob, "prob", (torch.float32,), (B, L))
        _bl(ent, "entropy", (torch.float32,), (B, L))
    if want_margin and mar is None:
        mar = torch.empty((B, L), dtype=torch.float32, device=dev)
    if mar is not None:
        _bl(mar, "margin", (torch.float32,), (B, L))
    am = torch.empty((B, L), dtype=torch.int32, device=dev) if argmax else None
    extra = _CStatsExtra()
    extra.margin = mar.data_ptr() if mar is not None else None
    extra.argmax = am.data_ptr() if am is not None else None
    extra.stats_temperature = float(stats_temperature) if stats_temperature else 0.0
    sup = (ctypes.c_int32 * max(len(suppress_ids), 1))(*[int(s) for s in suppress_ids])
    crules = (_CRule * 2)()
    keep = []
    for i, r in enumerate(rules):
        _bl(r.mask, "rule mask", _MASK_DTYPES, (B, L))
        if r.out is None:
            r.out = torch.empty((B, L), dtype=torch.bool, device=dev)
        _bl(r.out, "rule out", _MASK_DTYPES, (B, L))
        c = crules[i]
        c.kind, c.mask, c.out = r.kind, r.mask.data_ptr(), r.out.data_ptr()
        c.param, c.strict, c.score = r.param, int(r.strict), r.score
        if r.taus is not None:
            c.taus = _bl(r.taus, "taus", (torch.float64,), (B,)).data_ptr()
        if r.kind == RULE_TOPK:
            kt = _k_tensor(r.k, B, dev)
            keep.append(kt)
            c.k = kt.data_ptr()
        if r.kind == RULE_EDIT:
            if r.tokens is None and canvas is None:
                raise ValueError("the edit rule needs the current tokens")
            if r.tokens is not None:
                _bl(r.tokens, "tokens", (torch.int32,), (B, L))
                c.tokens = r.tokens.data_ptr()
    dt = DLLM_BF16 if logits.dtype == torch.bfloat16 else DLLM_F32
    lib = load_library()
    with _on(dev):
        stream = _stream(logits)
        args = [logits.data_ptr(), dt, B, L, V, row_stride, float(temperature),
                int(seed or 0) & 0xFFFFFFFFFFFFFFFF, int(step), sup, len(suppress_ids),
                x0.data_ptr(), prob.data_ptr(), ent.data_ptr(), ctypes.byref(extra),
                crules if len(rules) else None, len(rules)]
        if isinstance(workspace, str):
            if workspace != STATIC_WORKSPACE or canvas is None:
                raise ValueError("workspace='static' is taken by commit_step only")
            _check(lib.dllm_commit_step_static(*args, ctypes.byref(canvas[0]), stream),
                   "dllm_commit_step_static")
            return Stats(x0, prob, ent, mar, am)
        need = _ws_size(dt, B, L, V, dev)
        ws = workspace if workspace is not None else _workspace(dev, stream, need)
        if canvas is None:
            _check(lib.dllm_token_stats(*args, ws.data_ptr(), ws.numel(), stream),
                   "dllm_token_stats")
        else:
            _check(lib.dllm_commit_step(*args, ctypes.byref(canvas[0]), ws.data_ptr(),
                                        ws.numel(), stream), "dllm_commit_step")
    return Stats(x0, prob, ent, mar, am)


def _rule_out(conf, candidates, out):
    B, L = conf.shape
    _bl(candidates, "candidates", _MASK_DTYPES, (B, L))
    if out is None:
        out = torch.empty((B, L), dtype=torch.bool, device=conf.device)
    return _bl(out, "out", _MASK_DTYPES, (B, L))


def threshold_transfer(prob, candidates, threshold, strict=False, out=None):
    """Commit candidates with prob >= threshold (> when strict); force one if none pass.
    threshold: a number, or a (B,) float64 device tensor, one per batch row."""
    _bl(prob, "prob", (torch.float32,))
    out = _rule_out(prob, candidates, out)
    B, L = prob.shape
    if isinstance(threshold, torch.Tensor):
        taus = _bl(threshold, "threshold", (torch.float64,), (B,))
        with _on(prob.device):
            _check(load_library().dllm_transfer_threshold_rows(
                prob.data_ptr(), candidates.data_ptr(), taus.data_ptr(), B, L,
                int(bool(strict)), out.data_ptr(), _stream(prob)), "dllm_transfer_threshold_rows")
        return out
    with _on(prob.device):
        _check(load_library().dllm_transfer_threshold(
            prob.data_ptr(), candidates.data_ptr(), B, L, float(threshold), int(bool(strict)),
            out.data_ptr(), _stream(prob)), "dllm_transfer_threshold")
    return out


def decaying_threshold(tau_initial, tau_floor, decay, step):
    """max(tau_floor, tau_initial - decay * step): the linearly decaying
    confidence threshold with a floor."""
    out = ctypes.c_double()
    _check(load_library().dllm_decaying_threshold(float(tau_initial), float(tau_floor),
                                                   float(decay), int(step), ctypes.byref(out)),
           "dllm_decaying_threshold")
    return out.value


def topk_transfer(prob, candidates, k, out=None):
    """Commit the k[b] most confident candidates of every batch row."""
    _bl(prob, "prob", (torch.float32,))
    out = _rule_out(prob, candidates, out)
    B, L = prob.shape
    kt = _k_tensor(k, B, prob.device)
    with _on(prob.device):
        _check(load_library().dllm_transfer_topk(
            prob.data_ptr(), candidates.data_ptr(), kt.data_ptr(), B, L, out.data_ptr(),
            _stream(prob)), "dllm_transfer_topk")
    return out


def factor_transfer(prob, candidates, factor, out=None):
    """Commit the longest confidence-sorted prefix with (i+1)(1 - c_(i)) <= factor."""
    _bl(prob, "prob", (torch.float32,))
    out = _rule_out(prob, candidates, out)
    B, L = prob.shape
    with _on(prob.device):
        _check(load_library().dllm_transfer_factor(
            prob.data_ptr(), candidates.data_ptr(), B, L, float(factor), out.data_ptr(),
            _stream(prob)), "dllm_transfer_factor")
    return out


def entropy_bound_transfer(entropy, candidates, gamma, out=None):
    """Commit the longest entropy-sorted prefix with sum_{j<i} H_(j) <= gamma."""
    _bl(entropy, "entropy", (torch.float32,))
    out = _rule_out(entropy, candidates, out)
    B, L = entropy.shape
    with _on(entropy.device):
        _check(load_library().dllm_transfer_entropy_bound(
            entropy.data_ptr(), candidates.data_ptr(), B, L, float(gamma), out.data_ptr(),
            _stream(entropy)), "dllm_transfer_entropy_bound")
    return out


def edit_transfer(x0, prob, tokens, editable, editing_threshold, out=None):
    """edit = editable & (x0 != tokens) & (prob > editing_threshold)."""
    _bl(prob, "prob", (torch.float32,))
    B, L = prob.shape
    _bl(x0, "x0", (torch.int32,), (B, L))
    _bl(tokens, "tokens", (torch.int32,), (B, L))
    out = _rule_out(prob, editable, out)
    with _on(prob.device):
        _check(load_library().dllm_transfer_edit(
            x0.data_ptr(), prob.data_ptr(), tokens.data_ptr(), editable.data_ptr(), B, L,
            float(editing_threshold), out.data_ptr(), _stream(prob)), "dllm_transfer_edit")
    return out


def transfer_schedule(n_masked, steps, out=None):
    """(B, steps) int32 quotas spreading n_masked[b] evenly, extras first."""
    _bl(n_masked, "n_masked", (torch.int32,))
    B = n_masked.shape[0]
    if out is None:
        out = torch.empty((B, int(steps)), dtype=torch.int32, device=n_masked.device)
    _bl(out, "out", (torch.int32,), (B, int(steps)))
    with _on(n_masked.device):
        _check(load_library().dllm_transfer_schedule(
            n_masked.data_ptr(), B, int(steps), out.data_ptr(), _stream(n_masked)),
            "dllm_transfer_schedule")
    return out


def block_ranges(prompt_len, gen_len, block_len, align=False):
    """List of (start, end) blocks covering [prompt_len, prompt_len + gen_len)."""
    lib = load_library()
    n = _check(lib.dllm_block_ranges(int(prompt_len), int(gen_len), int(block_len),
                                     int(bool(align)), None, 0), "dllm_block_ranges")
    buf = (ctypes.c_int64 * max(2 * n, 2))()
    _check(lib.dllm_block_ranges(int(prompt_len), int(gen_len), int(block_len),
                                 int(bool(align)), buf, n), "dllm_block_ranges")
    return [(buf[2 * i], buf[2 * i + 1]) for i in range(n)]


def block_causal_mask(L, block_len, device="cuda", out=None):
    """(L, L) float32 additive mask: 0 within and below the query's block, -inf above."""
    if out is None:
        out = torch.empty((int(L), int(L)), dtype=torch.float32, device=device)
    _bl(out, "out", (torch.float32,), (int(L), int(L)))
    with _on(out.device):
        _check(load_library().dllm_block_causal_mask(int(L), int(block_len), out.data_ptr(),
                                                     _stream(out)), "dllm_block_causal_mask")
    return out


# ---------------------------------------------------------------- uniform-noise decoding

def linear_temperature(remaining, num_steps, t_min=0.4, t_max=0.8):
    """t_min + (t_max - t_min) * remaining / num_steps."""
    out = ctypes.c_double()
    _check(load_library().dllm_linear_temperature(int(remaining), int(num_steps), float(t_min),
                                                   float(t_max), ctypes.byref(out)),
           "dllm_linear_temperature")
    return out.value


def uniform_canvas(shape, vocab_size, seed, draw, device=None, out=None):
    """(B, L) int32 tokens uniform on [0, vocab_size) (Philox, counter-based)."""
    B, L = shape
    dev = torch.device(device) if device is not None else (out.device if out is not None
                                                           else torch.device("cuda"))
    if out is None:
        out = torch.empty((B, L), dtype=torch.int32, device=dev)
    _bl(out, "out", (torch.int32,), (B, L))
    with _on(out.device):
        _check(load_library().dllm_uniform_canvas(out.data_ptr(), B, L, int(vocab_size),
                                                  int(seed) & 0xFFFFFFFFFFFFFFFF, int(draw),
                                                  _stream(out)), "dllm_uniform_canvas")
    return out


def renoise(sample, accepted, noise, out=None):
    """where(accepted, sample, noise)."""
    _bl(sample, "sample", (torch.int32,))
    B, L = sample.shape
    _bl(accepted, "accepted", _MASK_DTYPES, (B, L))
    _bl(noise, "noise", (torch.int32,), (B, L))
    if out is None:
        out = torch.empty_like(sample)
    _bl(out, "out", (torch.int32,), (B, L))
    with _on(sample.device):
        _check(load_library().dllm_renoise(sample.data_ptr(), accepted.data_ptr(),
                                           noise.data_ptr(), B, L, out.data_ptr(),
                                           _stream(sample)), "dllm_renoise")
    return out


class StableConfidentStopping:
    """Per-row stop of the uniform-noise loop: stability_threshold consecutive
    unchanged argmax canvases and mean entropy <= confidence_threshold.  Call
    with (argmax, entropy); returns the (B,) bool done tensor, which only
    grows."""

    def __init__(self, stability_threshold=1, confidence_threshold=0.005):
        self.k, self.c = int(stability_threshold), float(confidence_threshold)
        self.prev = self.count = self.done = None

    def __call__(self, argmax, entropy):
        _bl(argmax, "argmax", (torch.int32,))
        B, L = argmax.shape
        _bl(entropy, "entropy", (torch.float32,), (B, L))
        first = self.prev is None
        if first:
            dev = argmax.device
            self.prev = torch.empty((B, L), dtype=torch.int32, device=dev)
            self.count = torch.zeros((B,), dtype=torch.int32, device=dev)
            self.done = torch.zeros((B,), dtype=torch.uint8, device=dev)
        with _on(argmax.device):
            _check(load_library().dllm_stable_confident_stop(
                argmax.data_ptr(), entropy.data_ptr(), B, L, self.k, self.c, int(first),
                self.prev.data_ptr(), self.count.data_ptr(), self.done.data_ptr(),
                _stream(argmax)), "dllm_stable_confident_stop")
        return self.done.bool()


# ---------------------------------------------------------------- scores of given tokens
# A call of these has a microsecond or two of device work at its smallest, so
# each argument is looked at once and named only when it is wrong.

def _same(t, name, dtype, shape, device):
    """A contiguous tensor of this dtype and shape on the call's device."""
    if isinstance(t, torch.Tensor) and t.device == device and t.dtype is dtype and \
            t.shape == shape and t.is_contiguous():
        return t
    _dev(t, name)
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    _bl(t, name, (dtype,), torch.Size(shape))
    return t


def _launch(device, what, fn, *args):
    """fn(*args, the device's current stream), with that device current."""
    index = device.index
    if index == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status < 0:
        _check(status, what)


def _logits_args(logits):
    _dev(logits, "logits")
    if logits.dim() != 3:
        raise ValueError("logits must be (B, L, V)")
    if logits.dtype is torch.bfloat16:
        dt = DLLM_BF16
    elif logits.dtype is torch.float32:
        dt = DLLM_F32
    else:
        raise ValueError("logits must be float32 or bfloat16")
    return dt, logits.shape[2] if logits.is_contiguous() else _row_stride(logits)


def _suppress_array(suppress_ids):
    if not len(suppress_ids):
        return None
    return (ctypes.c_int32 * len(suppress_ids))(*[int(s) for s in suppress_ids])


_lp_sizes = {}


def _logprobs_workspace(dev, dt, B, L, V, top):
    key = (dt, B, L, V, top, dev.index)
    need = _lp_sizes.get(key)
    if need is None:
        with _on(dev):
            need = int(load_library().dllm_token_logprobs_workspace_size(dt, B, L, V, top))
        _lp_sizes[key] = need
    if need == 0:
        return None
    if _capturing(dev):
        # a buffer of the graph's own, cleared by a node of the graph, so that
        # graphs captured on one stream and replayed side by side share nothing
        return torch.zeros(need, dtype=torch.uint8, device=dev)
    return _workspace(dev, torch._C._cuda_getCurrentRawStream(dev.index), need)


def _logprobs_call(logits, targets, temperature, suppress_ids, top, workspace):
    dt, row_stride = _logits_args(logits)
    B, L, V = logits.shape
    dev = logits.device
    _same(targets, "targets", torch.int32, (B, L), dev)
    top = int(top)
    if not 0 <= top <= MAX_TOP:
        raise ValueError(f"top must be in [0, {MAX_TOP}]")
    logprob = torch.empty((B, L), dtype=torch.float32, device=dev)
    entropy = torch.empty((B, L), dtype=torch.float32, device=dev)
    norm = torch.empty((B, L, 2), dtype=torch.float32, device=dev)
    ids = lps = ids_p = lps_p = ws_p = None
    ws_n = 0
    if top:
        ids = torch.empty((B, L, top), dtype=torch.int32, device=dev)
        lps = torch.empty((B, L, top), dtype=torch.float32, device=dev)
        ids_p, lps_p = ids.data_ptr(), lps.data_ptr()
    if workspace is None:
        workspace = _logprobs_workspace(dev, dt, B, L, V, top)
    else:
        _bl(workspace, "workspace", (torch.uint8,))
        if workspace.device != dev:
            raise ValueError(f"workspace is on {workspace.device}, not on {dev}")
    if workspace is not None:
        ws_p, ws_n = workspace.data_ptr(), workspace.numel()
    _launch(dev, "dllm_token_logprobs", load_library().dllm_token_logprobs, logits.data_ptr(), dt,
            B, L, V, row_stride, float(temperature), _suppress_array(suppress_ids),
            len(suppress_ids), targets.data_ptr(), top, logprob.data_ptr(), entropy.data_ptr(),
            norm.data_ptr(), ids_p, lps_p, ws_p, ws_n)
    return Logprobs(logprob, entropy, ids, lps, norm)


def _grad_call(logits, targets, norm, entropy, g_logprob, g_entropy, temperature, suppress_ids,
               out):
    dt, row_stride = _logits_args(logits)
    B, L, V = logits.shape
    _launch(logits.device, "dllm_token_logprobs_grad", load_library().dllm_token_logprobs_grad,
            logits.data_ptr(), dt, B, L, V, row_stride, float(temperature),
            _suppress_array(suppress_ids), len(suppress_ids), targets.data_ptr(), norm.data_ptr(),
            entropy.data_ptr(), g_logprob.data_ptr() if g_logprob is not None else None,
            g_entropy.data_ptr() if g_entropy is not None else None, out.data_ptr(),
            V if out.is_contiguous() else _row_stride(out))
    return out


class _LogprobsFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets, temperature, suppress_ids, top, workspace):
        r = _logprobs_call(logits, targets, temperature, suppress_ids, top, workspace)
        ctx.save_for_backward(logits, targets, r.norm, r.entropy)
        ctx.temperature, ctx.suppress_ids = temperature, tuple(suppress_ids)
        if top:
            ctx.mark_non_differentiable(r.norm, r.top_ids, r.top_logprobs)
        else:
            ctx.mark_non_differentiable(r.norm)
        ctx.set_materialize_grads(False)
        return tuple(r)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_logprob, g_entropy, *_):
        if g_logprob is None and g_entropy is None:
            return (None,) * 6
        logits, targets, norm, entropy = ctx.saved_tensors
        grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        _grad_call(logits, targets, norm, entropy,
                   None if g_logprob is None else g_logprob.contiguous(),
                   None if g_entropy is None else g_entropy.contiguous(), ctx.temperature,
                   ctx.suppress_ids, grad)
        return grad, None, None, None, None, None


def _check_leaf(node, device):
    """node: a leaf's gradient accumulator, which all living graphs of the leaf
    share and which runs on the stream it was made on, noted here."""
    stream = torch._C._cuda_getCurrentRawStream(device.index)
    if node.metadata.setdefault("commit_step_amd", stream) != stream and _capturing(device):
        raise RuntimeError("the captured backward pass of a leaf would meet an autograd graph of "
                           "it that lives on another stream; let that go first, or capture "
                           "token_logprobs_grad")


def token_logprobs(logits, targets, temperature=1.0, suppress_ids=(), top=0, workspace=None):
    """Scores of given tokens: for (B, L, V) float32 / bfloat16 logits and (B, L)
    int32 targets, log softmax(logits / temperature) at the target, the
    position's entropy, and its ``top`` most likely ids with their log
    probabilities (decreasing, ties by lower id; -1 and -inf where fewer ids
    have any probability; None when top == 0).  A target outside [0, V), such as
    -1, marks a position that is not scored: logprob and entropy 0, no gradient.

    Differentiable: logprob and entropy carry the gradient to logits that
    require one.  ``norm`` (B, L, 2) is what token_logprobs_grad takes.
    ``workspace``: None, or a zero-filled uint8 tensor that no other call in
    flight uses.

    Under graph capture a leaf's backward pass is refused while an autograd graph
    of the same leaf, made on another stream, lives: torch would join that stream
    to the capture and fail in its own thread.  (The same holds for a model's
    parameters, which this call does not see.)  token_logprobs_grad has no such
    tie.
    """
    if torch.is_grad_enabled() and isinstance(logits, torch.Tensor) and logits.requires_grad:
        r = Logprobs(*_LogprobsFunction.apply(logits, targets, temperature, suppress_ids, top,
                                              workspace))
        if logits.is_leaf:
            _check_leaf(r.logprob.grad_fn.next_functions[0][0], logits.device)
        return r
    return _logprobs_call(logits, targets, temperature, suppress_ids, top, workspace)


def token_logprobs_grad(logits, targets, norm, entropy, grad_logprob, grad_entropy=None,
                        temperature=1.0, suppress_ids=(), out=None):
    """Gradient of sum(grad_logprob * logprob + grad_entropy * entropy) with
    respect to the logits, from token_logprobs' norm and entropy.  Either
    gradient may be None.  ``out`` may be the logits themselves."""
    _logits_args(logits)
    B, L, V = logits.shape
    dev = logits.device
    _same(targets, "targets", torch.int32, (B, L), dev)
    _same(norm, "norm", torch.float32, (B, L, 2), dev)
    _same(entropy, "entropy", torch.float32, (B, L), dev)
    for g, name in ((grad_logprob, "grad_logprob"), (grad_entropy, "grad_entropy")):
        if g is not None:
            _same(g, name, torch.float32, (B, L), dev)
    if out is None:
        out = torch.empty((B, L, V), dtype=logits.dtype, device=dev)
    else:
        _dev(out, "out")
        if out.dtype != logits.dtype or out.shape != logits.shape or out.device != dev:
            raise ValueError("out must have the logits' dtype, shape and device")
        torch.autograd.graph.increment_version(out)      # a graph that saved it must notice
    return _grad_call(logits, targets, norm, entropy, grad_logprob, grad_entropy, temperature,
                      suppress_ids, out)


# ---------------------------------------------------------------- the 8-bit key/value cache

class KVCache:
    """A pool of pages of KV_PAGE tokens: keys and values of ``kv_heads`` heads of
    ``head_dim`` (64, 128 or 256) channels in e4m3, a power-of-two scale per page
    and head.  Sequences are rows of page numbers (int32 page tables), which the
    caller hands out.  The byte layout is the library's (include/dllm_commit.h);
    kv_read gives the values."""

    def __init__(self, num_pages, kv_heads, head_dim, device="cuda"):
        if head_dim not in (64, 128, 256):
            raise ValueError("head_dim must be 64, 128 or 256")
        if num_pages < 1 or kv_heads < 1:
            raise ValueError("num_pages and kv_heads must be positive")
        self.num_pages, self.kv_heads, self.head_dim = int(num_pages), int(kv_heads), int(head_dim)
        shape = (self.num_pages, self.kv_heads, KV_PAGE * self.head_dim)
        self._tensors = (torch.zeros(shape, dtype=torch.uint8, device=device),
                         torch.zeros(shape, dtype=torch.uint8, device=device),
                         torch.ones(shape[:2], dtype=torch.float32, device=device),
                         torch.ones(shape[:2], dtype=torch.float32, device=device))
        self.device = self._tensors[0].device
        self._c = _CCache(*(t.data_ptr() for t in self._tensors), self.num_pages, self.kv_heads,
                          self.head_dim)
        self._ref = ctypes.byref(self._c) if self.device.type == "cuda" else None

    # the pool's memory cannot be exchanged, only written: the calls hold its addresses
    k = property(lambda self: self._tensors[0], doc="e4m3 codes of the keys (uint8)")
    v = property(lambda self: self._tensors[1], doc="e4m3 codes of the values (uint8)")
    k_scale = property(lambda self: self._tensors[2], doc="(num_pages, kv_heads) float32")
    v_scale = property(lambda self: self._tensors[3], doc="(num_pages, kv_heads) float32")


def _cache(cache):
    if not isinstance(cache, KVCache):
        raise ValueError("cache must be a KVCache")
    if cache._ref is None:
        _dev(cache.k, "cache")
    return cache.device, cache._ref


def _table(t, name, B, device):
    """A (B, pages) int32 page table, rows of unit stride (a slice of a larger
    table will do); returns (pages, row stride)."""
    if isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.device == device and \
            t.dim() == 2 and t.is_contiguous() and (B is None or t.shape[0] == B):
        return t.shape[1], t.shape[1]
    _dev(t, name)
    if t.dtype is not torch.int32 or t.dim() != 2 or t.device != device:
        raise ValueError(f"{name} must be a (B, pages) int32 tensor on {device}")
    rows, pages = t.shape
    if B is not None and rows != B:
        raise ValueError(f"{name} has {rows} rows, not {B}")
    if pages > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} rows must have unit stride")
    return pages, t.stride(0) if rows > 1 else pages


_Strides = ctypes.c_int64 * 3


def _heads(t, name, shape, device):
    """A (B, L, heads, head_dim) bfloat16 tensor with unit stride along the last
    dimension; returns its element strides as a C array."""
    if isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.device == device and \
            t.shape == shape:
        sb, sl, sh, sd = t.stride()
        if sd == 1:
            return _Strides(sb, sl, sh)
    _dev(t, name)
    if t.dtype is not torch.bfloat16 or t.shape != shape or t.device != device:
        raise ValueError(f"{name} must be a {tuple(shape)} bfloat16 tensor on {device}, not "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")
    st = t.stride()
    if st[3] != 1 and t.numel():
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return _Strides(st[0], st[1], st[2])


def _apart(t, name):
    """Refuses an output whose elements share memory (an expanded view)."""
    if isinstance(t, torch.Tensor) and not t.is_contiguous():
        reach = 1
        for stride, size in sorted(zip(t.stride(), t.shape)):
            if size > 1:
                if stride < reach:
                    raise ValueError(f"{name} has elements that share memory")
                reach += stride * (size - 1)


def _ints(t, name, B, device):
    return None if t is None else _same(t, name, torch.int32, (B,), device).data_ptr()


def kv_write(cache, k, v, page_table, start, lens=None):
    """Store k, v (B, L, kv_heads, head_dim) bfloat16 as tokens start[b] ..
    start[b] + lens[b] - 1 (lens None: L) of every sequence, whose pages
    page_table (B, pages) names; the sequence then ends there.  Tokens before
    start[b] stay.  start, lens: (B,) int32."""
    dev, c = _cache(cache)
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be (B, L, kv_heads, head_dim)")
    B, L, _, _ = k.shape
    shape = (B, L, cache.kv_heads, cache.head_dim)
    ks = _heads(k, "k", shape, dev)
    vs = _heads(v, "v", shape, dev)
    pages, stride = _table(page_table, "page_table", B, dev)
    s = _ints(start, "start", B, dev)
    if s is None:
        raise ValueError("start must be given")
    _launch(dev, "dllm_kv_write", load_library().dllm_kv_write, c, k.data_ptr(), ks, v.data_ptr(),
            vs, B, L, page_table.data_ptr(), pages, stride, s, _ints(lens, "lens", B, dev))


def kv_read(cache, page_table, lens):
    """(k, v), each (B, KV_PAGE * pages, kv_heads, head_dim) bfloat16: the values
    the cache stands for, 0 past lens[b]."""
    dev, c = _cache(cache)
    pages, stride = _table(page_table, "page_table", None, dev)
    B = page_table.shape[0]
    n = _ints(lens, "lens", B, dev)
    if n is None:
        raise ValueError("lens must be given")
    shape = (B, pages * KV_PAGE, cache.kv_heads, cache.head_dim)
    k = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    v = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    _launch(dev, "dllm_kv_read", load_library().dllm_kv_read, c, B, page_table.data_ptr(), pages,
            stride, n, k.data_ptr(), v.data_ptr())
    return k, v


_attn_sizes = {}


def _attn_size(B, L, Hq, H, D, pages, device):
    """Workspace bytes of (block_attention, its weights)."""
    key = (B, L, Hq, H, D, pages, device.index)
    need = _attn_sizes.get(key)
    if need is None:
        lib = load_library()
        with _on(device):
            need = (int(lib.dllm_block_attention_workspace_size(B, L, Hq, H, D, pages)),
                    int(lib.dllm_attention_weights_workspace_size(B, L, Hq, H, pages)))
        _attn_sizes[key] = need
    return need


def block_attention(q, cache, page_table, kv_lens, q_start=None, q_lens=None, block_len=0,
                    scale=None, weights=None, out=None, lse=None):
    """Attention of q (B, L, q_heads, head_dim) bfloat16 over the cached tokens
    t < kv_lens[b]; with block_len > 0 only t // block_len <= pos // block_len
    for the query at pos = q_start[b] + l (the mask of block_causal_mask;
    block_len = 1 is causal).  Query head h reads key/value head
    h // (q_heads // kv_heads).  scale: 1 / sqrt(head_dim) by default.

    Returns Attention(out, lse): out like q, lse (B, q_heads, L) float32 (natural
    log).  A query that attends to nothing gives 0 and -inf; queries
    l >= q_lens[b] are not written (0 and -inf in outputs allocated here).
    ``weights`` (B, KV_PAGE * pages) float32: every cached token's attention
    weight, summed over queries and heads, is added to it (see kv_evict).  There
    is no gradient.
    """
    dev, c = _cache(cache)
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be (B, L, q_heads, head_dim)")
    if q.requires_grad and torch.is_grad_enabled():
        raise ValueError("block_attention has no gradient: detach q, or call under no_grad")
    B, L, Hq, D = q.shape
    shape = (B, L, Hq, cache.head_dim)
    qs = _heads(q, "q", shape, dev)
    pages, stride = _table(page_table, "page_table", B, dev)
    n = _ints(kv_lens, "kv_lens", B, dev)
    if n is None:
        raise ValueError("kv_lens must be given")
    qstart, qlens = _ints(q_start, "q_start", B, dev), _ints(q_lens, "q_lens", B, dev)
    if out is None:
        out = (torch.empty if q_lens is None else torch.zeros)(shape, dtype=torch.bfloat16,
                                                                device=dev)
    else:
        _apart(out, "out")
    os_ = _heads(out, "out", shape, dev)
    if lse is None:
        lse = torch.empty((B, Hq, L), dtype=torch.float32, device=dev)
        if q_lens is not None:
            lse.fill_(-math.inf)
    else:
        _same(lse, "lse", torch.float32, (B, Hq, L), dev)
    if weights is not None:
        _same(weights, "weights", torch.float32, (B, pages * KV_PAGE), dev)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    need, need_w = _attn_size(B, L, Hq, cache.kv_heads, D, pages, dev)
    if weights is not None:
        need = max(need, need_w)
    # any content will do: a block of torch's allocator per call, so that neither
    # streams nor captured graphs share one
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    ws_p = ws.data_ptr() if need else None
    lib = load_library()
    args = (c, q.data_ptr(), qs, B, L, Hq, page_table.data_ptr(), pages, stride, n, qstart, qlens,
            int(block_len), scale)
    _launch(dev, "dllm_block_attention", lib.dllm_block_attention, *args, out.data_ptr(), os_,
            lse.data_ptr(), ws_p, need)
    if weights is not None:
        _launch(dev, "dllm_attention_weights", lib.dllm_attention_weights, *args, lse.data_ptr(),
                weights.data_ptr(), ws_p, need)
    return Attention(out, lse)


def evict_select(weights, kv_lens, budget, sink=0, recent=0, new_T=None):
    """The tokens that stay when each cache is cut to ``budget`` tokens: all of
    them if there are no more; else the first ``sink``, the last ``recent``, and
    the ones of largest weight (ties: the lower position).  weights (B, T)
    float32, kv_lens (B,) int32.  Returns Evicted(kept (B, budget) int32
    increasing, -1 behind the last; lens (B,) int32; their weights (B, new_T),
    0 behind the last)."""
    _dev(weights, "weights")
    if weights.dtype is not torch.float32 or weights.dim() != 2 or \
            (weights.shape[1] > 1 and weights.stride(1) != 1):
        raise ValueError("weights must be a (B, T) float32 tensor with rows of unit stride")
    B, T = weights.shape
    dev = weights.device
    n = _ints(kv_lens, "kv_lens", B, dev)
    budget = int(budget)
    if budget < 1:
        raise ValueError("budget must be positive")
    new_T = budget if new_T is None else int(new_T)
    return _select(weights, B, T, weights.stride(0) if B > 1 else T, n, budget, int(sink),
                   int(recent), new_T)


def _select(weights, B, T, stride, lens_p, budget, sink, recent, new_T):
    dev = weights.device
    kept = torch.empty((B, budget), dtype=torch.int32, device=dev)
    lens = torch.empty((B,), dtype=torch.int32, device=dev)
    new_w = torch.empty((B, new_T), dtype=torch.float32, device=dev)
    _launch(dev, "dllm_evict_select", load_library().dllm_evict_select, weights.data_ptr(), B, T,
            stride, lens_p, budget, sink, recent, kept.data_ptr(), lens.data_ptr(),
            new_w.data_ptr(), new_T)
    return Evicted(kept, lens, new_w)


def kv_gather(cache, page_table, kept, counts, new_pages):
    """Token j < counts[b] on the pages of new_pages (B, pages) becomes token
    kept[b, j] of the sequence on page_table.  kept increases along its rows; no
    page of new_pages may be in use."""
    dev, c = _cache(cache)
    pages, stride = _table(page_table, "page_table", None, dev)
    B = page_table.shape[0]
    npages, nstride = _table(new_pages, "new_pages", B, dev)
    if not isinstance(kept, torch.Tensor) or kept.dim() != 2:
        raise ValueError("kept must be (B, n)")
    _same(kept, "kept", torch.int32, (B, kept.shape[1]), dev)
    _launch(dev, "dllm_kv_gather", load_library().dllm_kv_gather, c, B, page_table.data_ptr(),
            pages, stride, kept.data_ptr(), kept.shape[1], _ints(counts, "counts", B, dev),
            new_pages.data_ptr(), npages, nstride)


def kv_evict(cache, page_table, kv_lens, weights, budget, new_pages, sink=0, recent=0):
    """Cut every sequence's cache to ``budget`` tokens by accumulated attention
    weight (evict_select) and move the kept tokens to new_pages (B, at least
    ceil(budget / KV_PAGE)), free pages of the same pool (kv_gather); the old
    pages are then free.  Returns Evicted: the kept positions, the new lengths,
    and the kept tokens' weights (B, KV_PAGE * new_pages.shape[1]), which go on
    accumulating."""
    dev, c = _cache(cache)
    pages, stride = _table(page_table, "page_table", None, dev)
    B = page_table.shape[0]
    npages, nstride = _table(new_pages, "new_pages", B, dev)
    budget, T = int(budget), pages * KV_PAGE
    if budget < 1:
        raise ValueError("budget must be positive")
    if npages * KV_PAGE < budget:
        raise ValueError("new_pages cannot hold budget tokens")
    table_p, new_p = page_table.data_ptr(), new_pages.data_ptr()
    if new_p == table_p and pages:
        raise ValueError("new_pages is the page table")
    _same(weights, "weights", torch.float32, (B, T), dev)
    r = _select(weights, B, T, T, _ints(kv_lens, "kv_lens", B, dev), budget, int(sink),
                int(recent), npages * KV_PAGE)
    _launch(dev, "dllm_kv_gather", load_library().dllm_kv_gather, c, B, table_p, pages, stride,
            r.kept.data_ptr(), budget, r.lens.data_ptr(), new_p, npages, nstride)
    return r
