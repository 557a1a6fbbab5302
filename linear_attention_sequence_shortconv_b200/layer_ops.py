"""ctypes binding of the operators around the mixer (argument marshalling only): the gated
norm of its readout, the norm at the border of a residual block, the embedding and the AdamW
step.  As in the mixer's binding, every step runs in the library's CUDA kernels; there is no
CPU path, and a call runs on the device of its tensors, on torch's current stream or on
``stream``.  With ``stream`` given, what the call allocates belongs to that stream, and the
caller orders the stream behind the work that made the inputs.  Tensors of the caller that a call
writes get a new version, so that an autograd graph that needs their old values fails.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import functools
import itertools
from typing import Dict, List, Optional, Sequence, Union

import torch
from torch.autograd.graph import increment_version

from ._lib import LIB_PATH, PRISM_BF16, PRISM_FP32, PrismError, _call_device, _dtype_code, _wrote, lib
from ._lib import _check as _check_slow

PRISM_ACT_SILU = 0
PRISM_ACT_SIGMOID = 1
ACTS = {"silu": PRISM_ACT_SILU, "sigmoid": PRISM_ACT_SIGMOID}
STATE_BLOCK = 256  # elements under one scale of the 8-bit AdamW states
PRISM_ERR_UNSUPPORTED = 2


def _act_code(act: str) -> int:
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}, got {act!r}")
    return ACTS[act]


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _check(t, name, dtype=None, required=True, shape=None, device=None):
    """The mixer's check of one tensor argument, with a short way for a tensor that is fine."""
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return
    if (t.is_cuda and (dtype is None or t.dtype == dtype) and (shape is None or t.shape == shape)
            and (device is None or t.get_device() == device.index) and t.is_contiguous()):
        return
    _check_slow(t, name, dtype, required, shape, device)


_STAY = contextlib.nullcontext()


def _on(dev: torch.device, stream, tensors=()):
    """Context in which a call allocates and launches: the tensors' device, and `stream` where
    the caller names one (its inputs are then kept until the stream is through with them)."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        return torch.cuda.stream(stream)
    if torch._C._cuda_getDevice() == dev.index:
        return _STAY
    return torch.cuda.device(dev)


def _here(dev: torch.device):
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _done(rc: int, what: str) -> None:
    if rc != 0:
        raise PrismError(rc, what)


def _workspace(workspace, need: int, dev: torch.device):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    _check(workspace, "workspace", torch.uint8, device=dev)
    return workspace


INT_MAX = 0x7FFFFFFF


def _fit(what: str, sizes) -> None:
    """Refuses sizes beyond the C interface's int, which ctypes would cut off without an error."""
    if any(n > INT_MAX for n in sizes):
        raise PrismError(PRISM_ERR_UNSUPPORTED, f"{what} with {tuple(sizes)}")


def _heads(o: torch.Tensor):
    """Sizes (B, T, H, d) of [B, T, H, d], or of one decoded token [B, H, d]."""
    if o.numel() > INT_MAX:
        _fit("o", o.shape)
    if o.dim() == 4:
        return tuple(o.shape)
    if o.dim() == 3:
        return o.shape[0], 1, o.shape[1], o.shape[2]
    raise ValueError(f"o must be [B, T, H, d] or [B, H, d], got {tuple(o.shape)}")


def _gate_stride(gate, o, sizes) -> int:
    """Elements between the gate rows of two tokens: the last two dimensions are dense, and
    tokens stand at one distance (a slice of a wider projection)."""
    B, T, H, d = sizes
    if gate is None:
        return H * d
    if gate.dtype == o.dtype and gate.shape == o.shape and gate.get_device() == o.get_device() and gate.is_contiguous():
        return H * d
    if not gate.is_cuda or gate.device != o.device:
        raise ValueError(f"gate is on {gate.device}, but the call's tensors are on {o.device}")
    if gate.dtype != o.dtype:
        raise TypeError(f"gate must be {o.dtype}, got {gate.dtype}")
    if gate.shape != o.shape:
        raise ValueError(f"gate must have shape {tuple(o.shape)}, got {tuple(gate.shape)}")
    st = gate.stride()
    step = st[-3] if T > 1 or gate.dim() == 3 else st[0]
    if B * T == 1:
        step = H * d
    dense = (st[-1] == 1 or d == 1) and (st[-2] == d or H == 1)
    even = gate.dim() == 3 or T == 1 or B == 1 or st[0] == T * step
    if not dense or not even or step < H * d:
        raise ValueError(f"gate must be dense in its last two dimensions with tokens at one distance, got strides {st}")
    return step


def gated_norm_fwd(o, gate, weight, lengths=None, eps: float = 1e-5, act: str = "silu", y=None, stream=None):
    """y = o / sqrt(mean(o^2) + eps) * weight * act(gate), the mean over the last dimension
    (one head of one token): the norm of the mixer's readout with its output gate.

    o [B,T,H,d], or [B,H,d] for one decoded token; gate like o or None (no gate), possibly a
    slice of a wider projection (dense in H and d); weight [d] fp32; lengths [B] int32 or None
    (rows t >= lengths[b] give zero).  ``act`` is "silu" or "sigmoid".  y may be o.
    """
    act_code = _act_code(act)
    dev = _call_device(o, stream)
    code = _dtype_code(o, "o")
    sizes = B, T, H, d = _heads(o)
    _check(o, "o", device=dev)
    stride = _gate_stride(gate, o, sizes)
    _check(weight, "weight", torch.float32, shape=(d,), device=dev)
    _check(lengths, "lengths", torch.int32, required=False, shape=(B,), device=dev)
    _check(y, "y", o.dtype, required=False, shape=o.shape, device=dev)
    given = y
    with _on(dev, stream, (o, gate, weight, lengths, y)):
        if y is None:
            y = torch.empty_like(o)
        _done(lib().prism_gated_norm_fwd(_ptr(o), _ptr(gate), _ptr(weight), _ptr(lengths), B, T, H, d, stride, eps,
                                         act_code, code, _ptr(y), _here(dev)), "prism_gated_norm_fwd")
    if given is not None:
        _wrote(given)
    return y


def gated_norm_bwd(o, gate, weight, dy, lengths=None, eps: float = 1e-5, act: str = "silu", workspace=None,
                   stream=None) -> Dict[str, Optional[torch.Tensor]]:
    """Gradients of <y, dy> of gated_norm_fwd: a dict with keys o, gate (None without a gate),
    both in o's dtype, and weight (fp32).  "o" is what scan_bwd takes as dO."""
    act_code = _act_code(act)
    dev = _call_device(o, stream)
    code = _dtype_code(o, "o")
    sizes = B, T, H, d = _heads(o)
    _check(o, "o", device=dev)
    stride = _gate_stride(gate, o, sizes)
    _check(weight, "weight", torch.float32, shape=(d,), device=dev)
    _check(dy, "dy", o.dtype, shape=o.shape, device=dev)
    _check(lengths, "lengths", torch.int32, required=False, shape=(B,), device=dev)
    with _on(dev, stream, (o, gate, weight, dy, lengths, workspace)):
        workspace = _workspace(workspace, lib().prism_gated_norm_bwd_workspace_size(B, T, H, d), dev)
        g = {"o": torch.empty_like(o),
             "gate": None if gate is None else torch.empty(o.shape, dtype=o.dtype, device=dev),
             "weight": torch.empty_like(weight)}
        _done(lib().prism_gated_norm_bwd(_ptr(o), _ptr(gate), _ptr(weight), _ptr(dy), _ptr(lengths), B, T, H, d,
                                         stride, eps, act_code, code, _ptr(g["o"]), _ptr(g["gate"]),
                                         _ptr(g["weight"]), _ptr(workspace), workspace.numel(), _here(dev)),
              "prism_gated_norm_bwd")
    return g


def _stream_rows(x: torch.Tensor):
    """Sizes (B, T, D) of [B, T, D], or of one decoded token [B, D]."""
    if x.numel() > INT_MAX:
        _fit("x", x.shape)
    if x.dim() == 3:
        return tuple(x.shape)
    if x.dim() == 2:
        return x.shape[0], 1, x.shape[1]
    raise ValueError(f"x must be [B, T, D] or [B, D], got {tuple(x.shape)}")


def _block_checks(x, weight, y, post_weight, scale, lengths, dev):
    B, T, D = _stream_rows(x)
    _check(x, "x", device=dev)
    _check(weight, "weight", torch.float32, shape=(D,), device=dev)
    if y is None and (post_weight is not None or scale is not None):
        raise ValueError("post_weight and scale belong to y, which is not given")
    _check(y, "y", required=False, shape=x.shape, device=dev)
    _check(post_weight, "post_weight", torch.float32, required=False, shape=(D,), device=dev)
    _check(scale, "scale", torch.float32, required=False, shape=(D,), device=dev)
    _check(lengths, "lengths", torch.int32, required=False, shape=(B,), device=dev)
    return B, T, D


def block_norm_fwd(x, weight, y=None, post_weight=None, scale=None, res_scale: float = 1.0, lengths=None,
                   eps: float = 1e-5, h_dtype: Optional[torch.dtype] = None, x_out=None, h=None, stream=None):
    """The border between two blocks: x_out = x + res_scale * scale * z and h = RMSNorm(x_out)
    * weight, where z is the block's output y, or its RMSNorm * post_weight; returns (x_out, h).

    x [B,T,D], or [B,D] for one decoded token: the residual stream.  y like x; without it
    (before the first block) h is the norm of x and x itself is returned.  weight, post_weight,
    scale [D] fp32.  h has y's dtype, or ``h_dtype`` without y (None: x's); x and y may both be
    bf16 or both fp32, or x fp32 and y bf16.  x_out may be x.
    """
    dev = _call_device(x, stream)
    B, T, D = _block_checks(x, weight, y, post_weight, scale, lengths, dev)
    dt = y.dtype if y is not None else (h_dtype or x.dtype)
    if h_dtype is not None and h_dtype != dt:
        raise TypeError(f"h has y's dtype {dt}, got h_dtype={h_dtype}")
    x_code = _dtype_code(x, "x")
    if dt not in (torch.bfloat16, torch.float32):
        raise TypeError(f"y and h must be bfloat16 or float32, got {dt}")
    code = PRISM_BF16 if dt == torch.bfloat16 else PRISM_FP32
    _check(x_out, "x_out", x.dtype, required=False, shape=x.shape, device=dev)
    _check(h, "h", dt, required=False, shape=x.shape, device=dev)
    given = (None if y is None else x_out, h)
    with _on(dev, stream, (x, weight, y, post_weight, scale, lengths, x_out, h)):
        if y is None:
            x_out = x
        elif x_out is None:
            x_out = torch.empty_like(x)
        if h is None:
            h = torch.empty(x.shape, dtype=dt, device=dev)
        _done(lib().prism_block_norm_fwd(_ptr(x), _ptr(y), _ptr(post_weight), _ptr(scale), _ptr(weight),
                                         _ptr(lengths), B, T, D, res_scale, eps, x_code, code,
                                         _ptr(x_out if y is not None else None), _ptr(h), _here(dev)),
              "prism_block_norm_fwd")
    if any(t is not None for t in given):
        _wrote(*given)
    return x_out, h


def block_norm_bwd(x_out, weight, dh, y=None, post_weight=None, scale=None, res_scale: float = 1.0, dx_out=None,
                   lengths=None, eps: float = 1e-5, workspace=None,
                   stream=None) -> Dict[str, Optional[torch.Tensor]]:
    """Gradients of <x_out, dx_out> + <h, dh> of block_norm_fwd, from the x_out it returned (x
    without y) and the same y and vectors: a dict with keys x (x_out's dtype), y (dh's dtype),
    weight, post_weight and scale (fp32); None for what was not given.  dx_out None is zero."""
    dev = _call_device(x_out, stream)
    B, T, D = _block_checks(x_out, weight, y, post_weight, scale, lengths, dev)
    x_code, code = _dtype_code(x_out, "x_out"), _dtype_code(dh, "dh")
    _check(dh, "dh", None if y is None else y.dtype, shape=x_out.shape, device=dev)
    _check(dx_out, "dx_out", x_out.dtype, required=False, shape=x_out.shape, device=dev)
    with _on(dev, stream, (x_out, weight, dh, y, post_weight, scale, dx_out, lengths, workspace)):
        workspace = _workspace(workspace, lib().prism_block_norm_bwd_workspace_size(B, T, D), dev)
        g = {"x": torch.empty_like(x_out), "y": None if y is None else torch.empty_like(y),
             "weight": torch.empty_like(weight),
             "post_weight": None if post_weight is None else torch.empty_like(post_weight),
             "scale": None if scale is None else torch.empty_like(scale)}
        _done(lib().prism_block_norm_bwd(_ptr(x_out), _ptr(y), _ptr(post_weight), _ptr(scale), _ptr(weight), _ptr(dh),
                                         _ptr(dx_out), _ptr(lengths), B, T, D, res_scale, eps, x_code, code,
                                         _ptr(g["x"]), _ptr(g["y"]), _ptr(g["weight"]), _ptr(g["post_weight"]),
                                         _ptr(g["scale"]), _ptr(workspace), workspace.numel(), _here(dev)),
              "prism_block_norm_bwd")
    return g


def _id_sizes(ids: torch.Tensor, lengths):
    """(B, T, bits) of ids [B, T], or of one decoded token each, [B]."""
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids must be int32 or int64, got {ids.dtype}")
    if ids.dim() not in (1, 2):
        raise ValueError(f"ids must be [B, T] or [B], got {tuple(ids.shape)}")
    if ids.numel() > INT_MAX:
        _fit("ids", ids.shape)
    B, T = ids.shape if ids.dim() == 2 else (ids.shape[0], 1)
    return B, T, 32 if ids.dtype == torch.int32 else 64


def _table_sizes(V: int, D: int):
    """(V, D) of an embedding table."""
    if V > INT_MAX or D > INT_MAX:
        _fit("table", (V, D))
    return V, D


def embed_fwd(ids, table, scale: float = 1.0, lengths=None, dtype: Optional[torch.dtype] = None, out=None,
              stream=None):
    """out = scale * table[ids]: ids [B,T] or [B] (int32 or int64), table [V,D] (bf16 or fp32);
    returns [B,T,D] or [B,D] in ``dtype`` (None: the table's; bf16 of an fp32 table is
    possible).  Rows t >= lengths[b] are zero and their ids are not read.  An id outside the
    table gives a zero row, and stream_status() reports PRISM_ERR_BOUNDS."""
    dev = _call_device(ids, stream)
    B, T, bits = _id_sizes(ids, lengths)
    _check(ids, "ids", device=dev)
    _check(table, "table", device=dev)
    if table.dim() != 2:
        raise ValueError(f"table must be [V, D], got {tuple(table.shape)}")
    V, D = _table_sizes(*table.shape)
    table_code = _dtype_code(table, "table")
    dt = dtype or (table.dtype if out is None else out.dtype)
    if dt not in (torch.bfloat16, torch.float32):
        raise TypeError(f"dtype must be bfloat16 or float32, got {dt}")
    _check(lengths, "lengths", torch.int32, required=False, shape=(B,), device=dev)
    _check(out, "out", dt, required=False, shape=tuple(ids.shape) + (D,), device=dev)
    given = out
    with _on(dev, stream, (ids, table, lengths, out)):
        if out is None:
            out = torch.empty(tuple(ids.shape) + (D,), dtype=dt, device=dev)
        _done(lib().prism_embed_fwd(_ptr(ids), _ptr(table), _ptr(lengths), B, T, V, D, scale, bits, table_code,
                                    PRISM_BF16 if dt == torch.bfloat16 else PRISM_FP32, _ptr(out), _here(dev)),
              "prism_embed_fwd")
    if given is not None:
        _wrote(given)
    return out


def embed_bwd(ids, d_out, V: int, scale: float = 1.0, lengths=None, d_table=None, accumulate: bool = False,
              workspace=None, stream=None):
    """Gradient of embed_fwd's table, [V,D] fp32: d_table[v] = scale * the sum of d_out over the
    tokens with id v, in the order of the tokens.  ``d_table`` may be given; with ``accumulate``
    (which needs it) the sums are added to it and only rows that a token names are touched."""
    dev = _call_device(ids, stream)
    B, T, bits = _id_sizes(ids, lengths)
    _check(ids, "ids", device=dev)
    V, D = _table_sizes(V, d_out.shape[-1])
    code = _dtype_code(d_out, "d_out")
    _check(d_out, "d_out", shape=tuple(ids.shape) + (D,), device=dev)
    _check(lengths, "lengths", torch.int32, required=False, shape=(B,), device=dev)
    _check(d_table, "d_table", torch.float32, required=accumulate, shape=(V, D), device=dev)
    given = d_table
    with _on(dev, stream, (ids, d_out, lengths, d_table, workspace)):
        if d_table is None:
            d_table = torch.empty((V, D), dtype=torch.float32, device=dev)
        workspace = _workspace(workspace, lib().prism_embed_bwd_workspace_size(B, T, V, D), dev)
        _done(lib().prism_embed_bwd(_ptr(ids), _ptr(d_out), _ptr(lengths), B, T, V, D, scale, bits, code,
                                    int(accumulate), _ptr(d_table), _ptr(workspace), workspace.numel(), _here(dev)),
              "prism_embed_bwd")
    if given is not None:
        _wrote(given)
    return d_table


def adamw_state(params: Sequence[torch.Tensor], bits: int = 32) -> Dict[str, List[torch.Tensor]]:
    """Zero moments for adamw_step (pass as ``**state``): fp32, or with bits = 8 e4m3 codes
    with one fp32 scale per 256 elements."""
    if bits not in (8, 32):
        raise ValueError(f"bits must be 8 or 32, got {bits}")
    dt = torch.float32 if bits == 32 else torch.float8_e4m3fn
    state = {n: [torch.zeros(p.shape, dtype=torch.float32, device=p.device).to(dt) for p in params]
             for n in ("exp_avg", "exp_avg_sq")}
    if bits == 8:
        for n in ("exp_avg_scale", "exp_avg_sq_scale"):
            state[n] = [torch.zeros(-(-p.numel() // STATE_BLOCK), dtype=torch.float32, device=p.device)
                        for p in params]
    return state


def _list_checks(tensors, name, dtype, params, dev, shapes=True):
    if len(tensors) != len(params):
        raise ValueError(f"{name} must have {len(params)} tensors, got {len(tensors)}")
    at = dev.index
    for t, p in zip(tensors, params):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must hold tensors, got {type(t).__name__}")
        if t.dtype == dtype and t.get_device() == at and t.is_contiguous() and (not shapes or t.shape == p.shape):
            continue
        if t.dtype != dtype:
            raise TypeError(f"{name} must all be {dtype}, got {t.dtype}")
        if t.device != dev:
            raise ValueError(f"{name} holds a tensor on {t.device}, but the call's tensors are on {dev}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        raise ValueError(f"{name} must have the parameters' shapes, got {tuple(t.shape)} for {tuple(p.shape)}")


def _step_number(step: int) -> int:
    step = int(step)
    if abs(step) > INT_MAX:
        _fit("step", (abs(step),))
    return step


def _scalar(x, name, dtype, dev):
    """(host value, device pointer) of a number, or of a one-element CUDA tensor."""
    if not isinstance(x, torch.Tensor):
        return x, None
    _check(x, name, dtype, device=dev)
    if x.numel() != 1:
        raise ValueError(f"{name} must have one element, got {tuple(x.shape)}")
    return None, _ptr(x)


_ADAMW_TENSOR = 72  # bytes of prism_adamw_tensor: seven pointers, a count and a double
_DL_TENSOR = 48      # bytes of prism_dl_tensor
_DL_TYPES = {torch.float32: (2, 32), torch.bfloat16: (4, 16), torch.float8_e4m3fn: (10, 8)}


@functools.lru_cache(maxsize=None)
def _dl_exchange():
    """(prism_dl_pointers, torch's DLPack exchange function), or None where torch has none.  The
    function runs with the interpreter's lock held, since it looks at Python objects."""
    capsule = getattr(torch.Tensor, "__dlpack_c_exchange_api__", None)
    if capsule is None:
        return None
    get = ctypes.pythonapi.PyCapsule_GetPointer
    get.restype, get.argtypes = ctypes.c_void_p, [ctypes.py_object, ctypes.c_char_p]
    api = get(capsule, b"dlpack_exchange_api")
    # DLPackExchangeAPI: the version (two 32-bit numbers), an older table, then the functions; the
    # one that views an object as a tensor is the fourth
    if (ctypes.c_uint32 * 1).from_address(api)[0] != 1:
        return None
    view = (ctypes.c_void_p * 4).from_address(api + 16)[3]
    if not view:
        return None
    gather = ctypes.PyDLL(LIB_PATH).prism_dl_pointers
    vp, ci = ctypes.c_void_p, ctypes.c_int
    gather.restype = ci
    gather.argtypes = [ci, vp, ci, vp, vp, ci, vp, vp, ctypes.c_size_t, ctypes.c_size_t]
    return gather, view


def _adamw_table(n, lists, decay, dev):
    """The host array of prism_adamw_tensor of a step, its tensors checked."""
    table = ctypes.create_string_buffer(_ADAMW_TENSOR * n)
    memoryview(table).cast("B").cast("d")[8::9] = memoryview(decay)
    exchange = _dl_exchange()
    if exchange is not None:
        gather, view = exchange
        given = [tensors for _, tensors, _, _ in lists if tensors is not None]
        spec = array.array("i", [x for _, tensors, dtype, blocks in lists
                                 for x in (*(_DL_TYPES[dtype] if tensors is not None else (0, 0)),
                                           STATE_BLOCK if blocks else 0)])
        objects = array.array("Q", map(id, itertools.chain.from_iterable(given)))
        try:
            if gather(len(lists), spec.buffer_info()[0], n, objects.buffer_info()[0], view, dev.index,
                      ctypes.create_string_buffer(_DL_TENSOR * n), table, _ADAMW_TENSOR, 56) < 0:
                return table
        except Exception:  # torch's function says so of an object that is no tensor
            pass
        # the checks below say what is wrong with which
    fields = memoryview(table).cast("B").cast("Q")
    params = lists[0][1]
    for field, (name, tensors, dtype, blocks) in enumerate(lists):
        if tensors is None:
            continue
        _list_checks(tensors, name, dtype, params, dev, shapes=not blocks)
        if blocks and any(s.numel() != -(-p.numel() // STATE_BLOCK) for s, p in zip(tensors, params)):
            raise ValueError(f"{name} must have one element per {STATE_BLOCK} of its parameter")
        fields[field::9] = memoryview(array.array("Q", [t.data_ptr() for t in tensors]))
    fields[7::9] = memoryview(array.array("Q", [p.numel() for p in params]))
    return table


def adamw_step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], exp_avg: Sequence[torch.Tensor],
               exp_avg_sq: Sequence[torch.Tensor], step: Union[int, torch.Tensor] = 1,
               lr: Union[float, torch.Tensor] = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
               weight_decay: Union[float, Sequence[float]] = 0.01, grad_scale: Optional[torch.Tensor] = None,
               copies: Optional[Sequence[torch.Tensor]] = None, exp_avg_scale=None, exp_avg_sq_scale=None,
               stream=None) -> None:
    """One AdamW step over all tensors, in place (see prism_adamw_step for the formulas).

    params fp32 or bf16, grads fp32 or bf16 (one dtype each); exp_avg, exp_avg_sq and the scales
    as adamw_state makes them, updated in place.  ``step`` counts from 1; ``step`` (int32) and
    ``lr`` (fp32) may be one-element CUDA tensors, which the kernel reads, so that a captured
    graph follows them.  ``grad_scale``: one-element fp32 CUDA tensor that multiplies the
    gradients.  ``weight_decay``: one number, or one per tensor.  ``copies``: bf16 tensors that
    receive the new fp32 parameters.  Tensors of the call must not overlap.
    """
    # kept as they are for the length of the call
    params, grads, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, copies = (
        x if x is None or isinstance(x, (list, tuple)) else list(x)
        for x in (params, grads, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, copies))
    n = len(params)
    if n == 0:
        return
    dev = _call_device(params[0], stream)
    p_code = _dtype_code(params[0], "params")
    if len(grads) != n:
        raise ValueError(f"grads must have {n} tensors, got {len(grads)}")
    g_code = _dtype_code(grads[0], "grads")
    state_dtype = exp_avg[0].dtype if len(exp_avg) else None
    if state_dtype not in (torch.float32, torch.float8_e4m3fn):
        raise TypeError(f"exp_avg must be float32 or float8_e4m3fn, got {state_dtype}")
    bits = 32 if state_dtype == torch.float32 else 8
    if bits == 8 and (exp_avg_scale is None or exp_avg_sq_scale is None):
        raise ValueError("8-bit states need exp_avg_scale and exp_avg_sq_scale")
    if bits == 32 and (exp_avg_scale is not None or exp_avg_sq_scale is not None):
        raise ValueError("fp32 states take no scales")
    if copies is not None and p_code != PRISM_FP32:
        raise ValueError("copies go with fp32 parameters")
    if isinstance(weight_decay, (int, float)):
        decay = array.array("d", (weight_decay,)) * n
    else:
        decay = array.array("d", weight_decay)
        if len(decay) != n:
            raise ValueError(f"weight_decay must be a number or {n} of them, got {len(decay)}")
    step_host, step_dev = _scalar(step, "step", torch.int32, dev)
    lr_host, lr_dev = _scalar(lr, "lr", torch.float32, dev)
    if grad_scale is not None:
        _, grad_scale_dev = _scalar(grad_scale, "grad_scale", torch.float32, dev)
        if grad_scale_dev is None:
            raise TypeError("grad_scale must be a CUDA tensor")
    else:
        grad_scale_dev = None
    # the tensors in the order of prism_adamw_tensor's fields, with their types
    lists = [("params", params, params[0].dtype, False), ("grads", grads, grads[0].dtype, False),
             ("exp_avg", exp_avg, state_dtype, False), ("exp_avg_sq", exp_avg_sq, state_dtype, False),
             ("exp_avg_scale", exp_avg_scale, torch.float32, True),
             ("exp_avg_sq_scale", exp_avg_sq_scale, torch.float32, True), ("copies", copies, torch.bfloat16, False)]
    for name, tensors, _, _ in lists:
        if tensors is not None and len(tensors) != n:
            raise ValueError(f"{name} must have {n} tensors, got {len(tensors)}")
    table = _adamw_table(n, lists, decay, dev)
    used = ()
    if stream is not None:
        used = (*params, *grads, *exp_avg, *exp_avg_sq, *(exp_avg_scale or ()), *(exp_avg_sq_scale or ()),
                *(copies or ()), *(x for x in (step, lr, grad_scale) if isinstance(x, torch.Tensor)))
    with _on(dev, stream, used):
        _done(lib().prism_adamw_step(table, n, 0 if step_host is None else _step_number(step_host), step_dev,
                                     0.0 if lr_host is None else float(lr_host), lr_dev, betas[0], betas[1], eps,
                                     grad_scale_dev, p_code, g_code, bits, _here(dev)), "prism_adamw_step")
    increment_version([*params, *exp_avg, *exp_avg_sq, *(exp_avg_scale or ()), *(exp_avg_sq_scale or ()),
                       *(copies or ())])
