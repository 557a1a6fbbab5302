"""Host-side checks of the operators around the mixer (no GPU): the C entry points reject bad
arguments before any CUDA call, and report the workspaces that their documentation states."""
import ctypes
import struct

import pytest
import torch

import linear_attention_sequence_shortconv_b200 as prism
from linear_attention_sequence_shortconv_b200 import build as prism_build
from linear_attention_sequence_shortconv_b200 import layer_ops

FAKE = [0x100000000 + (i << 32) for i in range(16)]  # aligned, far apart, never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
BIG = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def built():
    prism_build.build()


def _gated(bwd=False, **kw):
    a = dict(o=FAKE[0], gate=FAKE[1], weight=FAKE[2], lengths=None, B=2, T=8, H=2, d=64, stride=128, eps=1e-5, act=0,
             dtype=0, y=FAKE[3], dy=FAKE[4], d_gate=FAKE[5], d_weight=FAKE[6], ws=FAKE[7], ws_bytes=BIG)
    a.update(kw)
    sizes = (a["B"], a["T"], a["H"], a["d"], a["stride"], a["eps"], a["act"], a["dtype"])
    if bwd:
        return prism.lib().prism_gated_norm_bwd(a["o"], a["gate"], a["weight"], a["dy"], a["lengths"], *sizes, a["y"],
                                                a["d_gate"], a["d_weight"], a["ws"], a["ws_bytes"], None)
    return prism.lib().prism_gated_norm_fwd(a["o"], a["gate"], a["weight"], a["lengths"], *sizes, a["y"], None)


COMMON_GATED = [
    (dict(o=None), INVALID), (dict(weight=None), INVALID), (dict(y=None), INVALID), (dict(B=0), INVALID),
    (dict(T=0), INVALID), (dict(H=0), INVALID), (dict(d=0), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(act=2), INVALID),
    (dict(dtype=9), INVALID), (dict(stride=127), INVALID), (dict(stride=132), UNSUPPORTED), (dict(d=48), UNSUPPORTED),
    (dict(o=FAKE[0] + 8), UNSUPPORTED), (dict(gate=FAKE[1] + 2), UNSUPPORTED), (dict(lengths=FAKE[8] + 4), UNSUPPORTED),
    (dict(H=1 << 30, d=128, stride=1 << 40), UNSUPPORTED),
    (dict(y=FAKE[0] + 16), INVALID), (dict(y=FAKE[1]), INVALID), (dict(y=FAKE[2]), INVALID),
    (dict(T=16, stride=144, y=FAKE[1] + 16 * 144), INVALID),  # inside a strided gate
]


@pytest.mark.parametrize("kw,code", COMMON_GATED)
def test_gated_norm_refusals(kw, code):
    assert _gated(**kw) == code
    assert _gated(bwd=True, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), INVALID), (dict(d_weight=None), INVALID), (dict(d_gate=None), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=255), WORKSPACE), (dict(y=FAKE[5]), INVALID),
    (dict(y=FAKE[0]), INVALID), (dict(d_gate=FAKE[1]), INVALID), (dict(d_weight=FAKE[2]), INVALID),
    (dict(ws=FAKE[0]), INVALID),
])
def test_gated_norm_bwd_refusals(kw, code):
    assert _gated(bwd=True, **kw) == code


def _block(bwd=False, **kw):
    a = dict(x=FAKE[0], y=FAKE[1], post=FAKE[2], scale=FAKE[3], weight=FAKE[4], lengths=None, B=2, T=8, D=96,
             res=1.0, eps=1e-5, x_dtype=1, dtype=0, x_out=FAKE[5], h=FAKE[6], dh=FAKE[7], dx_out=FAKE[8],
             dw=FAKE[9], dpost=FAKE[10], dscale=FAKE[11], ws=FAKE[12], ws_bytes=BIG)
    a.update(kw)
    sizes = (a["B"], a["T"], a["D"], a["res"], a["eps"], a["x_dtype"], a["dtype"])
    vecs = (a["x"], a["y"], a["post"], a["scale"], a["weight"])
    if bwd:
        return prism.lib().prism_block_norm_bwd(*vecs, a["dh"], a["dx_out"], a["lengths"], *sizes, a["x_out"], a["h"],
                                                a["dw"], a["dpost"], a["dscale"], a["ws"], a["ws_bytes"], None)
    return prism.lib().prism_block_norm_fwd(*vecs, a["lengths"], *sizes, a["x_out"], a["h"], None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INVALID), (dict(weight=None), INVALID), (dict(h=None), INVALID), (dict(x_out=None), INVALID),
    (dict(y=None), INVALID), (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(D=0), INVALID),
    (dict(eps=-1.0), INVALID), (dict(res=float("nan")), INVALID), (dict(dtype=2), INVALID), (dict(x_dtype=2), INVALID),
    (dict(D=8193), UNSUPPORTED), (dict(x_dtype=0, dtype=1), UNSUPPORTED), (dict(x=FAKE[0] + 4), UNSUPPORTED),
    (dict(post=FAKE[2] + 4), UNSUPPORTED), (dict(h=FAKE[1]), INVALID), (dict(h=FAKE[0]), INVALID),
    (dict(x_out=FAKE[6]), INVALID), (dict(x_out=FAKE[1]), INVALID),
])
def test_block_norm_refusals(bwd, kw, code):
    assert _block(bwd, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dh=None), INVALID), (dict(dw=None), INVALID), (dict(dpost=None), INVALID), (dict(dscale=None), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=1), WORKSPACE), (dict(x_out=FAKE[7]), INVALID),
    (dict(x_out=FAKE[0]), INVALID), (dict(dw=FAKE[10]), INVALID), (dict(ws=FAKE[8]), INVALID),
    (dict(dx_out=FAKE[8] + 4), UNSUPPORTED),
])
def test_block_norm_bwd_refusals(kw, code):
    assert _block(True, **kw) == code


def _embed(bwd=False, **kw):
    a = dict(ids=FAKE[0], table=FAKE[1], lengths=None, B=2, T=8, V=100, D=96, scale=1.0, bits=64, table_dtype=1,
             dtype=0, out=FAKE[2], acc=0, ws=FAKE[3], ws_bytes=BIG)
    a.update(kw)
    sizes = (a["B"], a["T"], a["V"], a["D"], a["scale"], a["bits"])
    if bwd:
        return prism.lib().prism_embed_bwd(a["ids"], a["table"], a["lengths"], *sizes, a["dtype"], a["acc"], a["out"],
                                           a["ws"], a["ws_bytes"], None)
    return prism.lib().prism_embed_fwd(a["ids"], a["table"], a["lengths"], *sizes, a["table_dtype"], a["dtype"],
                                       a["out"], None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(ids=None), INVALID), (dict(table=None), INVALID), (dict(out=None), INVALID), (dict(B=0), INVALID),
    (dict(T=0), INVALID), (dict(V=0), INVALID), (dict(D=0), INVALID), (dict(bits=16), INVALID),
    (dict(dtype=3), INVALID), (dict(scale=float("inf")), INVALID), (dict(D=8193), UNSUPPORTED),
    (dict(V=BIG + 1), UNSUPPORTED), (dict(B=1 << 16, T=1 << 15), UNSUPPORTED), (dict(ids=FAKE[0] + 8), UNSUPPORTED),
    (dict(out=FAKE[2] + 4), UNSUPPORTED), (dict(out=FAKE[1]), INVALID), (dict(out=FAKE[0]), INVALID),
])
def test_embed_refusals(bwd, kw, code):
    assert _embed(bwd, **kw) == code


def test_embed_more_refusals():
    assert _embed(table_dtype=0, dtype=1) == UNSUPPORTED
    assert _embed(True, ws=None) == WORKSPACE
    need = prism.lib().prism_embed_bwd_workspace_size(2, 8, 100, 96)
    assert need > 0 and _embed(True, ws_bytes=need - 1) == WORKSPACE
    assert _embed(True, ws=FAKE[2]) == INVALID


def test_workspace_sizes():
    L = prism.lib()
    assert L.prism_gated_norm_bwd_workspace_size(0, 1, 1, 64) == 0
    assert L.prism_block_norm_bwd_workspace_size(1, 1, 9000) == 0
    assert L.prism_embed_bwd_workspace_size(1, 1, 0, 8) == 0
    # partial sums: a bounded number of blocks, whatever the length of the batch
    assert L.prism_gated_norm_bwd_workspace_size(1 << 10, 1 << 14, 8, 128) <= 1 << 20
    assert L.prism_block_norm_bwd_workspace_size(1 << 10, 1 << 14, 768) <= 32 << 20
    # 16 bytes a token, the counts, a bit per row, and two rows for each chunk of at least 16 sorted tokens
    for B, T, V, D in ((1, 1, 1, 1), (16, 2048, 32000, 768), (128, 1024, 1000003, 128), (1, 1 << 22, 1 << 30, 64)):
        need, N = L.prism_embed_bwd_workspace_size(B, T, V, D), B * T
        assert 16 * N <= need <= 16 * N + (2 << 20) + V // 8 + 8 * D * (N // 16 + 1) + 2048


def _adam(tensors, step=1, step_dev=None, lr=1e-3, lr_dev=None, b1=0.9, b2=0.99, eps=1e-8, gs=None, p=1, g=1, bits=32,
          count=None):
    table = b"".join(struct.pack("@7PQd", *t) for t in tensors)
    return prism.lib().prism_adamw_step(table, len(tensors) if count is None else count, step, step_dev, lr, lr_dev, b1,
                                        b2, eps, gs, p, g, bits, None)


def _tensor(n=100, **kw):
    a = dict(p=FAKE[0], g=FAKE[1], m=FAKE[2], v=FAKE[3], ms=FAKE[4], vs=FAKE[5], c=0, n=n, wd=0.1)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(p=0), INVALID), (dict(g=0), INVALID), (dict(m=0), INVALID), (dict(v=0), INVALID),
    (dict(wd=float("nan")), INVALID), (dict(p=FAKE[0] + 4), UNSUPPORTED), (dict(v=FAKE[3] + 8), UNSUPPORTED),
    (dict(c=FAKE[6] + 8), UNSUPPORTED), (dict(g=FAKE[0]), INVALID), (dict(m=FAKE[3]), INVALID),
    (dict(c=FAKE[1]), INVALID), (dict(m=FAKE[0] + 384), INVALID),
])
def test_adamw_tensor_refusals(kw, code):
    assert _adam([_tensor(**kw)]) == code
    # the same behind other tensors
    ok = _tensor(p=FAKE[8], g=FAKE[9], m=FAKE[10], v=FAKE[11])
    assert _adam([ok, _tensor(**kw)]) == code


def test_adamw_refusals():
    t = _tensor()
    assert _adam([t], bits=16) == INVALID
    assert _adam([t], step=0) == INVALID
    assert _adam([t], b1=1.0) == INVALID
    assert _adam([t], b2=-0.1) == INVALID
    assert _adam([t], eps=float("nan")) == INVALID
    assert _adam([t], lr=float("inf")) == INVALID
    assert _adam([t], p=5) == INVALID
    assert _adam([t], g=-1) == INVALID
    assert _adam([t], count=-1) == INVALID
    assert _adam([t], gs=FAKE[9] + 2) == UNSUPPORTED
    assert _adam([t], gs=FAKE[0] + 4) == INVALID                       # a scalar inside a parameter
    assert _adam([_tensor(c=FAKE[6])], p=0) == INVALID                 # a copy of a bf16 parameter
    assert _adam([_tensor(ms=0)], bits=8) == INVALID
    assert _adam([_tensor(vs=FAKE[5] + 2)], bits=8) == UNSUPPORTED
    assert _adam([_tensor(vs=FAKE[4])], bits=8) == INVALID
    assert _adam([t, t]) == INVALID                                    # the same tensor twice
    assert _adam([t, _tensor(p=FAKE[8], m=FAKE[10], v=FAKE[11] + 0, g=FAKE[2])]) == INVALID  # a gradient in a moment
    assert _adam([_tensor(n=1 << 43)]) == UNSUPPORTED


def test_python_checks_need_no_device():
    x = torch.zeros(2, 3, 4, 16)
    for call in (lambda: prism.gated_norm_fwd(x, None, torch.ones(16)),
                 lambda: prism.block_norm_fwd(torch.zeros(2, 3, 8), torch.ones(8)),
                 lambda: prism.embed_fwd(torch.zeros(2, 3, dtype=torch.int64), torch.zeros(4, 8)),
                 lambda: prism.embed_bwd(torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, 3, 8), 4),
                 lambda: prism.adamw_step([x], [x], [x], [x])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="act"):
        prism.gated_norm_fwd(x, None, torch.ones(16), act="relu")
    with pytest.raises(ValueError, match="bits"):
        prism.adamw_state([x], bits=4)
    assert prism.adamw_step([], [], [], []) is None


def test_adamw_state_shapes():
    params = [torch.zeros(3, 100), torch.zeros(0), torch.zeros(256)]
    s = prism.adamw_state(params)
    assert [t.dtype for t in s["exp_avg"]] == [torch.float32] * 3 and set(s) == {"exp_avg", "exp_avg_sq"}
    s = prism.adamw_state(params, bits=8)
    assert [tuple(t.shape) for t in s["exp_avg_sq"]] == [(3, 100), (0,), (256,)]
    assert [t.numel() for t in s["exp_avg_scale"]] == [2, 0, 1]
    assert s["exp_avg"][0].dtype == torch.float8_e4m3fn


def test_struct_matches_the_header():
    # seven pointers, a 64-bit count and a double, no padding
    class T(ctypes.Structure):
        _fields_ = [(n, ctypes.c_void_p) for n in "pgmvabc"] + [("n", ctypes.c_longlong), ("wd", ctypes.c_double)]

    assert ctypes.sizeof(T) == struct.calcsize("@7PQd") == 72


class DL(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("device_type", ctypes.c_int32), ("device_id", ctypes.c_int32),
                ("ndim", ctypes.c_int32), ("code", ctypes.c_uint8), ("bits", ctypes.c_uint8),
                ("lanes", ctypes.c_uint16), ("shape", ctypes.POINTER(ctypes.c_int64)),
                ("strides", ctypes.POINTER(ctypes.c_int64)), ("offset", ctypes.c_uint64)]


def _dl(shape, strides=None, device=(2, 0), code=2, bits=32, lanes=1, data=0x1000, offset=0):
    arr = lambda x: (ctypes.c_int64 * max(1, len(x)))(*x)  # noqa: E731
    return DL(data, *device, len(shape), code, bits, lanes, arr(shape), None if strides is None else arr(strides), offset)


def _gather(*fields, block=0, code=2, bits=32, fail=None, skip=()):
    """prism_dl_pointers over described tensors: (returned, pointers per field, counts)."""
    flat = [t for f, ts in enumerate(fields) if f not in skip for t in ts]
    view = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.POINTER(DL))

    def look(obj, out):
        i = (obj or 0) - 1
        if i == fail:
            return -1
        ctypes.memmove(out, ctypes.byref(flat[i]), ctypes.sizeof(DL))
        return 0

    n = len(fields[0])
    spec = [x for f in range(len(fields)) for x in ((0, 0, 0) if f in skip else (code, bits, block if f else 0))]
    out = (ctypes.c_uint64 * (9 * n))()
    got = prism.lib().prism_dl_pointers(
        len(fields), (ctypes.c_int * len(spec))(*spec), n, (ctypes.c_void_p * len(flat))(*range(1, len(flat) + 1)),
        view(look), 0, (DL * n)(), out, ctypes.c_size_t(72), ctypes.c_size_t(56))
    return got, [list(out[f::9]) for f in range(len(fields))], list(out[7::9])


def test_dl_pointers():
    assert ctypes.sizeof(DL) == 48
    ok = [_dl([2, 3], [3, 1]), _dl([], [], data=0x2000), _dl([4, 1, 5], [5, 99, 1], data=0x3000, offset=64),
          _dl([0, 7], [7, 1]), _dl([6])]
    where = [0x1000, 0x2000, 0x3040, 0x1000, 0x1000]
    assert _gather(ok) == (-1, [where], [6, 1, 20, 0, 6])
    assert _gather(ok, ok, ok, skip=(1,)) == (-1, [where, [0] * 5, where], [6, 1, 20, 0, 6])
    bad = [_dl([2, 3], [1, 2]), _dl([2, 3], [4, 1]), _dl([3], [0]), _dl([2], device=(1, 0)), _dl([2], device=(2, 1)),
           _dl([2], code=4, bits=16), _dl([2], bits=64), _dl([2], lanes=2)]
    for b in bad:
        assert _gather([ok[0], ok[4], b])[0] == 2
    assert _gather(ok, fail=3)[0] == 3 and _gather(ok, ok, fail=7)[0] == 7
    # shapes are compared, or the numbers of blocks
    assert _gather([_dl([2, 3])], [_dl([6])])[0] == 1
    assert _gather([_dl([2, 3])], [_dl([3, 2])])[0] == 1
    many = [_dl([257]), _dl([16, 16]), _dl([0, 3])]
    assert _gather(many, [_dl([2]), _dl([1]), _dl([0])], block=256)[0] == -1
    assert _gather(many, [_dl([1]), _dl([1]), _dl([0])], block=256)[0] == 3


def test_sizes_beyond_32_bits_are_refused():
    # the C entry points take them as int: they must not arrive cut off
    big = (1 << 32) + 5
    meta = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="meta")  # noqa: E731
    for call in (lambda: layer_ops._heads(meta(big, 1, 1, 16)), lambda: layer_ops._heads(meta(1, big, 1, 16)),
                 lambda: layer_ops._heads(meta(big, 1, 16)), lambda: layer_ops._stream_rows(meta(big, 1, 8)),
                 lambda: layer_ops._stream_rows(meta(1, 1 << 31, 8)), lambda: layer_ops._stream_rows(meta(big, 1)),
                 lambda: layer_ops._id_sizes(meta(big, dtype=torch.int64), None),
                 lambda: layer_ops._id_sizes(meta(2, big, dtype=torch.int32), None),
                 lambda: layer_ops._table_sizes(big, 1), lambda: layer_ops._table_sizes(1 << 31, 8),
                 lambda: layer_ops._table_sizes(4, big), lambda: layer_ops._step_number(big),
                 lambda: layer_ops._step_number(-big)):
        with pytest.raises(prism.PrismError, match="UNSUPPORTED"):
            call()
    assert layer_ops._stream_rows(meta((1 << 31) - 1, 1)) == ((1 << 31) - 1, 1, 1)
    assert layer_ops._id_sizes(meta(2, 3, dtype=torch.int32), None) == (2, 3, 32)
    assert layer_ops._table_sizes(100, 8) == (100, 8) and layer_ops._step_number(7) == 7


@pytest.mark.parametrize("bwd", [False, True])
def test_block_norm_refuses_more_wide_rows_than_32_bits_number(bwd):
    far = {n: 0x1000_0000_0000 * (i + 1) for i, n in enumerate(("x", "y", "post", "scale", "weight", "x_out", "h", "dh",
                                                                "dx_out", "dw", "dpost", "dscale", "ws"))}
    assert _block(bwd, B=1 << 16, T=1 << 15, D=257, **far) == UNSUPPORTED
    assert prism.lib().prism_block_norm_bwd_workspace_size(1 << 16, 1 << 15, 257) == 0
    assert prism.lib().prism_block_norm_bwd_workspace_size(1 << 16, 1 << 15, 256) > 0
