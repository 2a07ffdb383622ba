"""Binding of the operators between a block's projections: rotary append, paged attention, gated delta rule.

Argument checks and marshalling only, as in the package; the arguments go to the C ABI as the structs of
``include/tq.h``, packed field by field.

    freq, rope_scale = tq.rope_frequencies(64, 1e6, scaling="yarn", factor=4, original=32768, device="cuda")
    kc, vc = tq.kv_cache(pages, kv_heads, page, dim, torch.bfloat16)
    q = tq.rope_append(q, k, v, positions, slots, freq, kc, vc, q_norm=wq, k_norm=wk, rope_scale=rope_scale)
    y = tq.paged_attn(q, kc, vc, block_table, kv_len, cu, out_dtype=torch.float32, ws=ws)
    y = tq.gdn(q, k, v, g, beta, state, cu, l2norm=True, ws=gws)
"""
from __future__ import annotations

import contextlib
import math
import struct
import warnings

import torch

from . import ERR_SHAPE, TQError, _check, _lib


def _load_binding():
    """The checks of the ordinary call in C++: where these checks have to say what is wrong or serve what is rare, its calls
    return None.  Where it is not there, or was built for another torch (whose classes it reads), these checks serve every call."""
    try:
        from . import _binding as b
    except ImportError as e:
        why = str(e)
    else:
        built = getattr(b, "torch_version", None)
        if built == torch.__version__:
            return b
        why = f"it was built for torch {built}"
    warnings.warn(f"_binding.so is not used ({why}): each of these operators' calls takes the host some 6 us more; build.py builds it", stacklevel=3)
    return None


_binding = _load_binding()

_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_LAYOUTS = {"half": 0, "interleaved": 1}

# the structs of include/tq.h in their field order, native alignment ("0q" pads the end to 8 bytes)
_ROPE = struct.Struct("@3P6q3P2P1P2P1P2q8i2f0q")
_ATTN = struct.Struct("@P2q2P3P3P1P7q7if0q")
_GDN = struct.Struct("@3P6q2P2P2P2P1P5q7i2f0q")

_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _pack(form: struct.Struct, where: str, *fields) -> bytes:
    try:
        return form.pack(*fields)
    except (struct.error, OverflowError) as e:  # what no field holds
        raise ValueError(f"{where}: an argument that is no number, or out of its type's range ({e})") from None


def _call(f, args: bytes, device, where: str) -> None:
    """A call of the library on the tensors' device and that device's current stream."""
    other = device.index is not None and device.index != _current_device()
    with torch.cuda.device(device) if other else contextlib.nullcontext():
        _check(f(args, _stream(device.index)), where)


def _bad(name: str, t, want: str):
    got = type(t).__name__ if not isinstance(t, torch.Tensor) else f"{t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}"
    raise ValueError(f"{name} must be {want} (got {got})")


def _full(t, dtype, shape, device, name):
    """A contiguous GPU tensor of this dtype and shape on this device."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        _bad(name, t, f"a contiguous CUDA tensor of dtype {dtype} and shape {tuple(shape)} on {device}")
    return t.data_ptr()


def _some(t, dtype, shape, device, name):
    return 0 if t is None else _full(t, dtype, shape, device, name)


def _heads3(t, dtype, device, name):
    """A GPU tensor [tokens, heads, dim] with a contiguous last dimension: shape and strides."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 3 or (dtype is not None and t.dtype != dtype) or (
            device is not None and t.device != device):
        _bad(name, t, f"a CUDA tensor [tokens, heads, dim]{f' of dtype {dtype}' if dtype else ''}")
    s = t.stride()
    if s[2] != 1 and t.shape[2] > 1:
        _bad(name, t, "contiguous in its last dimension")
    # the stride of a dimension of one is never used, whatever it holds
    n = t.shape
    return n, (s[0] if n[0] > 1 else 0), (s[1] if n[1] > 1 else 0)


def _dtype(t, allowed, name):
    if t not in allowed:
        raise ValueError(f"{name} has dtype {t}, not one of {', '.join(map(str, allowed))}")
    return _TYPES[t]


def _ws(ws, need: int, device):
    if ws is None:
        return 0, 0
    if not isinstance(ws, torch.Tensor) or not ws.is_cuda or ws.dtype != torch.uint8 or ws.device != device or not ws.is_contiguous():
        _bad("ws", ws, f"a contiguous uint8 CUDA tensor on {device}")
    n = ws.numel()
    if n < need:
        raise ValueError(f"ws holds {n} bytes, needs {need}")
    return (ws.data_ptr(), n) if n else (0, 0)


def _result(out, out_dtype, default, shape, device):
    """The output tensor (made here if none is given), its address and its type's code."""
    if out is None:
        dt = default if out_dtype is None else out_dtype
        code = _dtype(dt, _ALL, "out")
        out = torch.empty(shape, dtype=dt, device=device)
        return out, out.data_ptr(), code
    if not isinstance(out, torch.Tensor) or (out_dtype is not None and out.dtype != out_dtype):
        _bad("out", out, f"a tensor of dtype {default if out_dtype is None else out_dtype}")
    return out, _full(out, out.dtype, shape, device, "out"), _dtype(out.dtype, _ALL, "out")


def _flag(bad_flag, device):
    return 0 if bad_flag is None else _full(bad_flag, torch.int32, (1,), device, "bad_flag")


_HALVES = (torch.bfloat16, torch.float16)
_ALL = (torch.float32, torch.bfloat16, torch.float16)


def rope_frequencies(rot: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0, original: int = 0,
                     beta_fast: float = 32.0, beta_slow: float = 1.0, low: float = 1.0, high: float = 4.0, device=None):
    """Rotary frequencies (float64 [rot / 2]) and the factor on cosines and sines, for ``rope_append``.

    ``scaling`` for contexts of ``factor`` times the ``original`` length:
      none    base^(-2i/rot)
      linear  every frequency divided by factor
      ntk     base * factor^(rot/(rot-2)): the slowest divided by factor, the fastest kept
      yarn    between kept (at least beta_fast turns over ``original``) and divided (at most beta_slow turns) on a
              ramp over i, and cosines and sines times 0.1 ln(factor) + 1
      bands   wavelengths above original / low divided, below original / high kept, in between interpolated
    """
    if rot < 2 or rot % 2 or not base > 1 or not factor > 0:
        raise ValueError("rope_frequencies: rot even and at least 2, base > 1, factor > 0")
    if scaling in ("yarn", "bands") and original < 1:
        raise ValueError(f"rope_frequencies: {scaling} needs the original length")
    if scaling == "ntk":
        if rot == 2:
            raise ValueError("rope_frequencies: ntk needs rot of at least 4")
        base = base * factor ** (rot / (rot - 2))
    inv = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    scale = 1.0
    if scaling == "linear":
        inv = [f / factor for f in inv]
    elif scaling == "yarn":
        def place(turns):
            return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo, hi = max(math.floor(place(beta_fast)), 0), min(math.ceil(place(beta_slow)), rot - 1)
        ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(rot // 2)]
        inv = [f * (1 - r) + f / factor * r for f, r in zip(inv, ramp)]
        scale = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    elif scaling == "bands":
        def band(f):
            turns = original * f / (2 * math.pi)
            s = min(1.0, max(0.0, (turns - low) / (high - low)))
            return f * s + f / factor * (1 - s)

        inv = [band(f) for f in inv]
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"rope_frequencies: unknown scaling {scaling!r}")
    return torch.tensor(inv, dtype=torch.float64, device=device), scale


def kv_cache(pages: int, kv_heads: int, page: int, dim: int, dtype=torch.bfloat16, device="cuda"):
    """A zeroed paged cache: K [pages, kv_heads, page, dim] and V [pages, kv_heads, dim, page]."""
    _dtype(dtype, _HALVES, "the cache")
    return (torch.zeros(pages, kv_heads, page, dim, dtype=dtype, device=device),
            torch.zeros(pages, kv_heads, dim, page, dtype=dtype, device=device))


def _cache(k_cache, v_cache, device):
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        _bad("k_cache", k_cache, "a CUDA tensor [pages, kv_heads, page, dim]")
    pages, heads, page, dim = n = k_cache.shape
    dt = k_cache.dtype
    code = _dtype(dt, _HALVES, "k_cache")
    return pages, heads, page, dim, dt, code, _full(k_cache, dt, n, device, "k_cache"), _full(v_cache, dt, (pages, heads, dim, page), device, "v_cache")


def rope_append(q, k, v, positions, slots, inv_freq, k_cache, v_cache, *, q_norm=None, k_norm=None, eps: float = 1e-6,
                layout: str = "half", rope_scale: float = 1.0, out=None, bad_flag=None) -> torch.Tensor:
    """Norm and rotate q and k per head, append k and v to the paged cache; returns the rotated q in the cache's type.

    q [tokens, heads, dim], k and v [tokens, kv_heads, dim]: fp32, bf16 or fp16, any token and head strides (views of
    a fused projection's rows).  positions int32 [tokens]; slots int64 [tokens] (page * page size + place, negative:
    not stored); inv_freq float64 [rot / 2] or None; q_norm and k_norm fp32 [dim] or None."""
    if _binding and out is not None and layout in _LAYOUTS:
        r = _binding.rope_append(q, k, v, positions, slots, inv_freq, k_cache, v_cache, q_norm, k_norm, eps, _LAYOUTS[layout], rope_scale, out, bad_flag)
        if r is out:
            return out
        if r is not None:
            _check(r, "tq_rope_append")
    dt = q.dtype if isinstance(q, torch.Tensor) else None
    (tokens, heads, dim), q0, q1 = _heads3(q, None, None, "q")
    dev = q.device
    kn, k0, k1 = _heads3(k, dt, dev, "k")
    vn, v0, v1 = _heads3(v, dt, dev, "v")
    pages, kv_heads, page, cdim, cdt, ccode, kp, vp = _cache(k_cache, v_cache, dev)
    code = _dtype(dt, _ALL, "q")
    if cdim != dim or kn != (tokens, kv_heads, dim) or vn != kn:
        raise TQError(ERR_SHAPE, f"rope_append: q {tuple(q.shape)}, k {tuple(kn)}, v {tuple(vn)} and k_cache {tuple(k_cache.shape)} do not fit")
    rot = 0
    if inv_freq is not None:
        if not isinstance(inv_freq, torch.Tensor):
            _bad("inv_freq", inv_freq, "a float64 CUDA tensor [rot / 2], or None")
        rot = 2 * inv_freq.numel()
    if layout not in _LAYOUTS:
        raise ValueError(f"layout {layout!r} is neither 'half' nor 'interleaved'")
    row = (tokens,)
    freq = _some(inv_freq, torch.float64, (rot // 2,), dev, "inv_freq")
    pos = _some(positions, torch.int32, row, dev, "positions")
    slot = _full(slots, torch.int64, row, dev, "slots")
    wq = _some(q_norm, torch.float32, (dim,), dev, "q_norm")
    wk = _some(k_norm, torch.float32, (dim,), dev, "k_norm")
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=cdt, device=dev)
        o = out.data_ptr()
    else:
        o = _full(out, cdt, (tokens, heads, dim), dev, "out")
    _call(_lib.tq_rope_append,
          _pack(_ROPE, "rope_append", q.data_ptr(), k.data_ptr(), v.data_ptr(), q0, q1, k0, k1, v0, v1, pos, slot, freq, wq, wk, o, kp, vp,
                _flag(bad_flag, dev), tokens, pages, heads, kv_heads, dim, rot, page, code, ccode, _LAYOUTS[layout], eps, rope_scale),
          dev, "tq_rope_append")
    return out


def attn_workspace_bytes(tokens: int, seqs: int, heads: int, kv_heads: int, dim: int) -> int:
    return _lib.tq_paged_attn_workspace_bytes(tokens, seqs, heads, kv_heads, dim)


def attn_workspace(tokens: int, seqs: int, heads: int, kv_heads: int, dim: int, device="cuda") -> torch.Tensor:
    """A zeroed workspace for ``paged_attn`` calls of these sizes; every call leaves it ready for the next."""
    return torch.zeros(max(16, attn_workspace_bytes(tokens, seqs, heads, kv_heads, dim)), dtype=torch.uint8, device=device)


def paged_attn(q, k_cache, v_cache, block_table, kv_len, cu=None, *, scale=None, window: int = 0, max_len: int = 0, out=None,
               out_dtype=None, lse=None, ws=None, bad_flag=None) -> torch.Tensor:
    """Causal attention of new tokens over a paged cache that holds their keys and values already.

    q [tokens, heads, dim] in the cache's type; block_table int32 [seqs, width]; kv_len int32 [seqs], new tokens
    included; cu int32 [seqs + 1] or None (one token each); scale defaults to dim^-1/2; window 0 = all earlier keys;
    max_len: the longest sequence's new tokens, if known.  out in the cache's type or fp32; lse: fp32 [tokens, heads]
    to be filled, or None.  ws: see ``attn_workspace``; without one no sequence's keys are split over workgroups
    (one stream over 131075 keys 3.5 ms instead of 0.07, over 1000 keys 40 us instead of 18)."""
    if _binding and out is not None and out_dtype is None:
        r = _binding.paged_attn(q, k_cache, v_cache, block_table, kv_len, cu, scale, window, max_len, out, lse, ws, bad_flag)
        if r is out:
            return out
        if r is not None:
            _check(r, "tq_paged_attn")
    dt = q.dtype if isinstance(q, torch.Tensor) else None
    (tokens, heads, dim), q0, q1 = _heads3(q, None, None, "q")
    dev = q.device
    pages, kv_heads, page, cdim, cdt, ccode, kp, vp = _cache(k_cache, v_cache, dev)
    if cdim != dim or dt != cdt:
        raise TQError(ERR_SHAPE, f"paged_attn: q {tuple(q.shape)} {dt} and k_cache {tuple(k_cache.shape)} {cdt} do not fit")
    if not isinstance(block_table, torch.Tensor) or not block_table.is_cuda or block_table.dtype != torch.int32 or block_table.dim() != 2 or (
            block_table.device != dev or (block_table.stride(1) != 1 and block_table.shape[1] > 1)):
        _bad("block_table", block_table, "an int32 CUDA tensor [seqs, width] with contiguous rows")
    seqs, width = block_table.shape
    stride = block_table.stride(0) if seqs > 1 else width
    lens = _full(kv_len, torch.int32, (seqs,), dev, "kv_len")
    cup = _some(cu, torch.int32, (seqs + 1,), dev, "cu")
    out, o, ocode = _result(out, out_dtype, cdt, (tokens, heads, dim), dev)
    lp = _some(lse, torch.float32, (tokens, heads), dev, "lse")
    wp, wn = _ws(ws, 0 if ws is None else attn_workspace_bytes(tokens, seqs, heads, kv_heads, dim), dev)
    _call(_lib.tq_paged_attn,
          _pack(_ATTN, "paged_attn", q.data_ptr(), q0, q1, kp, vp, block_table.data_ptr(), lens, cup, o, lp, wp, _flag(bad_flag, dev), width, stride,
                tokens, seqs, pages, max_len, wn, heads, kv_heads, dim, page, ccode, ocode, window, dim**-0.5 if scale is None else scale),
          dev, "tq_paged_attn")
    return out


def gdn_workspace_bytes(tokens: int, seqs: int, v_heads: int, dk: int, dv: int, max_len: int = 0) -> int:
    return _lib.tq_gdn_workspace_bytes(tokens, seqs, max_len, v_heads, dk, dv)


def gdn_workspace(tokens: int, seqs: int, v_heads: int, dk: int, dv: int, max_len: int = 0, device="cuda"):
    """Scratch for ``gdn`` calls of these sizes (needs no clearing), or None where they use none."""
    n = gdn_workspace_bytes(tokens, seqs, v_heads, dk, dv, max_len)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def gdn(q, k, v, g, beta, state, cu=None, *, slots=None, scale=None, l2norm: bool = False, eps: float = 1e-6, max_len: int = 0, out=None,
        out_dtype=None, state_out=None, ws=None, bad_flag=None) -> torch.Tensor:
    """Gated delta rule over the sequences of the token axis; updates ``state`` in place unless ``state_out`` is given.

    q and k [tokens, k_heads, dk], v [tokens, v_heads, dv]: fp32, bf16 or fp16, any token and head strides; g (log
    decay, <= 0) and beta fp32 [tokens, v_heads]; state fp32 [states, v_heads, dk, dv]; cu int32 [seqs + 1] or None
    (one token each); slots int32 [seqs] into the states, or None (sequence b has state b); scale defaults to
    dk^-1/2; l2norm: q and k are normalised per head first.  ws: see ``gdn_workspace``; without one long sequences go
    token after token (4096 tokens in 5.6 ms instead of 0.19).  max_len: the longest sequence's tokens; without it the
    call is taken for one long sequence, which several short ones pay for (8 of 4 tokens 59 us instead of 23).  Returns
    out [tokens, v_heads, dv] in the inputs' type or fp32."""
    if _binding and out is not None and out_dtype is None:
        r = _binding.gdn(q, k, v, g, beta, state, cu, slots, scale, 1 if l2norm else 0, eps, max_len, out, state_out, ws, bad_flag)
        if r is out:
            return out
        if r is not None:
            _check(r, "tq_gdn")
    dt = q.dtype if isinstance(q, torch.Tensor) else None
    (tokens, k_heads, dk), q0, q1 = _heads3(q, None, None, "q")
    dev = q.device
    kn, k0, k1 = _heads3(k, dt, dev, "k")
    (vt, v_heads, dv), v0, v1 = _heads3(v, dt, dev, "v")
    code = _dtype(dt, _ALL, "q")
    if kn != (tokens, k_heads, dk) or vt != tokens or not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise TQError(ERR_SHAPE, f"gdn: q {tuple(q.shape)}, k {tuple(kn)} and v {tuple(v.shape)} do not fit, or state is not [states, heads, dk, dv]")
    states = state.shape[0]
    sshape = (states, v_heads, dk, dv)
    sp = _full(state, torch.float32, sshape, dev, "state")
    so = sp if state_out is None else _full(state_out, torch.float32, sshape, dev, "state_out")
    if cu is not None:
        if not isinstance(cu, torch.Tensor) or cu.dim() != 1 or cu.shape[0] < 1:
            _bad("cu", cu, "an int32 CUDA tensor [seqs + 1]")
        seqs = cu.shape[0] - 1
        cup = _full(cu, torch.int32, (seqs + 1,), dev, "cu")
    else:
        seqs, cup = tokens, 0
    slot = _some(slots, torch.int32, (seqs,), dev, "slots")
    row = (tokens, v_heads)
    gp, bp = _full(g, torch.float32, row, dev, "g"), _full(beta, torch.float32, row, dev, "beta")
    out, o, ocode = _result(out, out_dtype, dt, (tokens, v_heads, dv), dev)
    wp, wn = _ws(ws, 0 if ws is None else gdn_workspace_bytes(tokens, seqs, v_heads, dk, dv, max_len), dev)
    _call(_lib.tq_gdn,
          _pack(_GDN, "gdn", q.data_ptr(), k.data_ptr(), v.data_ptr(), q0, q1, k0, k1, v0, v1, gp, bp, sp, so, slot, cup, o, wp,
                _flag(bad_flag, dev), tokens, seqs, states, max_len, wn, k_heads, v_heads, dk, dv, code, ocode, 1 if l2norm else 0,
                dk**-0.5 if scale is None else scale, eps),
          dev, "tq_gdn")
    return out
