"""Binding of what differs from row to row in a batch that shares its weights: experts, adapters, sampling.

Argument checks and marshalling only, as in ``seq.py``.

    weights, experts = tq.route(logits, 8, score="sigmoid", bias=bias, groups=8, top_groups=4, group_best=2)
    order, offsets = tq.expert_lists(experts, n)
    y = tq.gemm_experts("pq2_0", w, rows, cols, q, d, order, offsets)         # [tokens * 8, rows]
    y = tq.adapter_add(y, x, a, b, index, ranks=ranks, scale=scale, ws=aws)   # in place
    token = tq.sample(logits, u, temperature=t, top_k=k, top_p=p, min_p=m, logprob=logprob, ws=sws)
"""
from __future__ import annotations

import struct

import torch

from . import ERR_SHAPE, FORMATS, TQError, _check, _lib, repacked_bytes
from .seq import _ALL, _HALVES, _bad, _binding, _call, _dtype, _flag, _full, _pack, _some, _stream, _TYPES, _ws, _current_device

_SCORES = {"softmax": 0, "sigmoid": 1}

# the structs of include/tq.h in their field order, native alignment ("0q" pads the end to 8 bytes)
_ROUTE = struct.Struct("@4P2q8if0q")
_EXPERTS = struct.Struct("@7P4q2i0q")
_ADAPTER = struct.Struct("@10P7q5i0q")
_SAMPLE = struct.Struct("@9P4qi0q")


def _matrix(t, dtypes, shape, device, name):
    """A GPU tensor [rows, columns] of one of these types with contiguous rows: its address, row stride and type."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 2 or t.dtype not in dtypes or (device is not None and t.device != device) or (
            shape is not None and t.shape != shape) or (t.stride(1) != 1 and t.shape[1] > 1):
        want = f" of shape {tuple(shape)}" if shape is not None else ""
        _bad(name, t, f"a CUDA tensor [rows, columns]{want} with contiguous rows, of dtype {' or '.join(map(str, dtypes))}")
    return t.data_ptr(), (t.stride(0) if t.shape[0] > 1 else 0), _TYPES[t.dtype]


def route(logits, k: int, *, score: str = "softmax", bias=None, groups: int = 1, top_groups: int = 1, group_best: int = 1, renorm: bool = True,
          scale: float = 1.0, out=None):
    """The k experts of each token and their weights: (weights fp32 [tokens, k], experts int32 [tokens, k]).

    logits [tokens, experts]: fp32, bf16 or fp16, any row stride.  s = softmax or sigmoid of them; s + bias (fp32 [experts]
    or None) chooses, s weighs: scale * s, or scale * s / (sum of the chosen s) with renorm.  groups > 1: only experts of the
    ``top_groups`` groups whose ``group_best`` (1 or 2) largest s + bias sum to most.  Equal ones: the lowest index first.
    Logits of -inf and NaN are never chosen; places without an expert get id -1 and weight 0.  out: (weights, experts) to be
    filled."""
    if _binding and out is not None and score in _SCORES:
        r = _binding.route(logits, k, _SCORES[score], bias, groups, top_groups, group_best, 1 if renorm else 0, scale, out)
        if r is out:
            return out
        if r is not None:
            _check(r, "tq_route")
    lp, stride, code = _matrix(logits, _ALL, None, None, "logits")
    dev, (tokens, experts) = logits.device, logits.shape
    if score not in _SCORES:
        raise ValueError(f"score {score!r} is neither 'softmax' nor 'sigmoid'")
    bp = _some(bias, torch.float32, (experts,), dev, "bias")
    if not isinstance(k, int) or not 1 <= k <= 32:
        raise TQError(ERR_SHAPE, f"route: k {k} is not 1 to 32")
    if out is None:
        out = torch.empty(tokens, k, device=dev), torch.empty(tokens, k, dtype=torch.int32, device=dev)
    weights, ids = out
    wp, ip = _full(weights, torch.float32, (tokens, k), dev, "out[0]"), _full(ids, torch.int32, (tokens, k), dev, "out[1]")
    _call(_lib.tq_route,
          _pack(_ROUTE, "route", lp, bp, wp, ip, stride, tokens, experts, k, groups, top_groups, group_best, _SCORES[score], 1 if renorm else 0, code, scale),
          dev, "tq_route")
    return out


def expert_lists(experts, n: int, *, out=None):
    """The pairs of a choice sorted by expert: (order int32 [pairs], offsets int32 [n + 1]); expert e has the pairs
    order[offsets[e]:offsets[e + 1]], in their own order.  experts int32, any shape (its values, flattened, are the pairs');
    pairs whose expert is not in [0, n) come last."""
    if _binding and out is not None:
        r = _binding.expert_lists(experts, n, out)
        if r is out:
            return out
        if r is not None:
            _check(r, "tq_expert_lists")
    if not isinstance(experts, torch.Tensor) or not experts.is_cuda or experts.dtype != torch.int32 or not experts.is_contiguous():
        _bad("experts", experts, "a contiguous int32 CUDA tensor")
    if not isinstance(n, int) or not 1 <= n <= 65536:
        raise TQError(ERR_SHAPE, f"expert_lists: {n} experts are not 1 to 65536")
    dev, pairs = experts.device, experts.numel()
    if out is None:
        out = torch.empty(pairs, dtype=torch.int32, device=dev), torch.empty(n + 1, dtype=torch.int32, device=dev)
    order, offsets = out
    op, fp = _full(order, torch.int32, (pairs,), dev, "out[0]"), _full(offsets, torch.int32, (n + 1,), dev, "out[1]")
    other = dev.index is not None and dev.index != _current_device()
    if other:
        with torch.cuda.device(dev):
            _check(_lib.tq_expert_lists(experts.data_ptr(), pairs, n, op, fp, _stream(dev.index)), "tq_expert_lists")
    else:
        _check(_lib.tq_expert_lists(experts.data_ptr(), pairs, n, op, fp, _stream(dev.index)), "tq_expert_lists")
    return out


def gemm_experts(fmt, w, rows: int, cols: int, q, d, order, offsets, *, out=None, bad_flag=None) -> torch.Tensor:
    """y fp32 [pairs, rows]: pair p times the matrix of its expert, bit-identical to ``gemv`` of that matrix without a workspace.

    w uint8 [experts, repacked_bytes(fmt, rows, cols)] (stacked ``repack`` results); q int8 [inputs, cols] and d fp32
    [inputs, cols / 256] from ``quantize_q8k``; order and offsets from ``expert_lists``.  inputs divides the pairs: pair p
    reads input p // (pairs // inputs), so that a token's experts share its activations, or every pair has its own.  Pairs
    without an expert get zeros.  pq2_0 only."""
    if isinstance(fmt, str) and fmt not in FORMATS:
        raise ValueError(f"unknown format {fmt!r}")
    code = FORMATS[fmt] if isinstance(fmt, str) else int(fmt)
    if _binding and out is not None:
        r = _binding.gemm_experts(code, w, rows, cols, q, d, order, offsets, out, bad_flag)
        if r is out:
            return out
        if r is not None:
            _check(r, "tq_gemm_experts")
    if not isinstance(w, torch.Tensor) or not w.is_cuda or w.dtype != torch.uint8 or w.dim() != 2 or not w.is_contiguous():
        _bad("w", w, "a contiguous uint8 CUDA tensor [experts, bytes of a repacked matrix]")
    need = repacked_bytes(code, rows, cols)
    if need <= 0 or w.shape[1] != need:
        raise TQError(ERR_SHAPE, f"gemm_experts: w has {w.shape[1]} bytes per expert, {rows} x {cols} needs {need}")
    dev, experts = w.device, w.shape[0]
    if not isinstance(order, torch.Tensor) or order.dim() != 1:
        _bad("order", order, "an int32 CUDA tensor [pairs]")
    pairs = order.shape[0]
    if not isinstance(q, torch.Tensor) or q.dim() != 2:
        _bad("q", q, "an int8 CUDA tensor [inputs, cols]")
    inputs = q.shape[0]
    qp, dp = _full(q, torch.int8, (inputs, cols), dev, "q"), _full(d, torch.float32, (inputs, cols // 256), dev, "d")
    op, fp = _full(order, torch.int32, (pairs,), dev, "order"), _full(offsets, torch.int32, (experts + 1,), dev, "offsets")
    if out is None:
        out = torch.empty(pairs, rows, device=dev)
    yp = _full(out, torch.float32, (pairs, rows), dev, "out")
    _call(_lib.tq_gemm_experts, _pack(_EXPERTS, "gemm_experts", w.data_ptr(), qp, dp, op, fp, yp, _flag(bad_flag, dev), rows, cols, pairs, inputs, experts, code),
          dev, "tq_gemm_experts")
    return out


def adapter_workspace_bytes(tokens: int, adapters: int, rank: int, cols: int) -> int:
    return _lib.tq_adapter_workspace_bytes(tokens, adapters, rank, cols)


def adapter_workspace(tokens: int, adapters: int, rank: int, cols: int, device="cuda") -> torch.Tensor:
    """Scratch for ``adapter_add`` calls of these sizes and of smaller ones (needs no clearing)."""
    return torch.empty(max(16, adapter_workspace_bytes(tokens, adapters, rank, cols)), dtype=torch.uint8, device=device)


def adapter_add(y, x, a, b, index, *, ranks=None, scale=None, out=None, ws=None, bad_flag=None) -> torch.Tensor:
    """out[t] = y[t] + scale_i B_i (A_i x[t]) with i = index[t]; a token of index -1 keeps its y.  In place without ``out``.

    y [tokens, rows]: fp32, bf16 or fp16, any row stride; x [tokens, cols]: fp32, or a's type; a [adapters, rank, cols] and b
    [adapters, rows, rank]: bf16 or fp16, rank and cols multiples of 8; index int32 [tokens]; ranks int32 [adapters] (how many
    rows of A and columns of B an adapter uses) or None; scale fp32 [adapters] or None.  ws: see ``adapter_workspace``, made
    for the call where none is given."""
    if out is None:
        out = y
    if _binding and ws is not None:
        r = _binding.adapter_add(y, x, a, b, index, ranks, scale, out, ws, bad_flag)
        if r is out:
            return out
        if r is not None:
            _check(r, "tq_adapter_add")
    yp, ys, ycode = _matrix(y, _ALL, None, None, "y")
    dev, (tokens, rows) = y.device, y.shape
    if not isinstance(a, torch.Tensor) or a.dim() != 3:
        _bad("a", a, "a CUDA tensor [adapters, rank, cols]")
    adapters, rank, cols = a.shape
    wt = a.dtype
    wcode = _dtype(wt, _HALVES, "a")
    xp, xs, xcode = _matrix(x, _ALL, (tokens, cols), dev, "x")
    ap, bp = _full(a, wt, (adapters, rank, cols), dev, "a"), _full(b, wt, (adapters, rows, rank), dev, "b")
    ip = _full(index, torch.int32, (tokens,), dev, "index")
    rp, sp = _some(ranks, torch.int32, (adapters,), dev, "ranks"), _some(scale, torch.float32, (adapters,), dev, "scale")
    op, os, _ = _matrix(out, (y.dtype,), (tokens, rows), dev, "out")
    if out.stride(0) == 0 and tokens > 1:
        raise ValueError("out's rows overlap")
    need = adapter_workspace_bytes(tokens, adapters, rank, cols)
    if ws is None:
        ws = torch.empty(max(16, need), dtype=torch.uint8, device=dev)
    wp, wn = _ws(ws, need, dev)
    _call(_lib.tq_adapter_add,
          _pack(_ADAPTER, "adapter_add", xp, yp, ap, bp, op, ip, rp, sp, wp, _flag(bad_flag, dev), xs, ys, os, tokens, cols, rows, wn, adapters, rank, xcode,
                wcode, ycode),
          dev, "tq_adapter_add")
    return out


def sample_workspace_bytes(rows: int, vocab: int) -> int:
    return _lib.tq_sample_workspace_bytes(rows, vocab)


def sample_workspace(rows: int, vocab: int, device="cuda") -> torch.Tensor:
    """Scratch for ``sample`` calls of these sizes and of smaller ones (needs no clearing)."""
    return torch.empty(max(16, sample_workspace_bytes(rows, vocab)), dtype=torch.uint8, device=device)


def sample(logits, u, *, temperature=None, top_k=None, top_p=None, min_p=None, out=None, logprob=None, ws=None) -> torch.Tensor:
    """One token (int32 [rows]) for each row of logits [rows, vocab] (fp32, bf16 or fp16, any row stride), drawn with the random
    numbers u (fp32 [rows], in [0, 1)).

    Each request its own: temperature fp32 [rows] (0: the largest logit), top_k int32 (0: off), top_p fp32 (1: off), min_p fp32
    (0: off), or None.  top_k keeps the largest logits, top_p of these the shortest beginning with that share of their
    probability, min_p of these the tokens with that share of the largest probability.  logprob: fp32 [rows] to be filled with
    the token's log probability before any filter.  A row of nothing but -inf and NaN gives -1.  ws: see ``sample_workspace``,
    made for the call where none is given."""
    if _binding and out is not None and ws is not None:
        r = _binding.sample(logits, u, temperature, top_k, top_p, min_p, out, logprob, ws)
        if r is out:
            return out
        if r is not None:
            _check(r, "tq_sample")
    lp, stride, code = _matrix(logits, _ALL, None, None, "logits")
    dev, (rows, vocab) = logits.device, logits.shape
    f32, i32, one = torch.float32, torch.int32, (rows,)
    up, tp, kp = _full(u, f32, one, dev, "u"), _some(temperature, f32, one, dev, "temperature"), _some(top_k, i32, one, dev, "top_k")
    pp, mp, gp = _some(top_p, f32, one, dev, "top_p"), _some(min_p, f32, one, dev, "min_p"), _some(logprob, f32, one, dev, "logprob")
    if out is None:
        out = torch.empty(rows, dtype=i32, device=dev)
    op = _full(out, i32, one, dev, "out")
    need = sample_workspace_bytes(rows, vocab)
    if ws is None:
        ws = sample_workspace(rows, vocab, device=dev)
    wp, wn = _ws(ws, need, dev)
    _call(_lib.tq_sample, _pack(_SAMPLE, "sample", lp, up, tp, kp, pp, mp, op, gp, wp, stride, rows, vocab, wn, code), dev, "tq_sample")
    return out
