"""Refusals of the layer operators that need no GPU: the C entry points return
the documented status before any HIP call, and the binding raises for host
tensors."""
import ctypes
import os

import pytest
import torch

from gated_delta_rule_40_amd import libkda as K

P = ctypes.c_void_p(0x10000)       # aligned, never dereferenced
ODD = ctypes.c_void_p(0x10001)
WS = ctypes.c_void_p(0x100000)
Q, Q2 = ctypes.c_void_p(0x200000), ctypes.c_void_p(0x200010)
B, F = K.KDA_BF16, K.KDA_F32
INVALID, UNSUPPORTED = K.KDA_ERR_INVALID_ARG, K.KDA_ERR_UNSUPPORTED

CALLS = {
    "kda_scan_prefill": dict(x=P, g=P, init=None, cu=P, N=1, T=300, D=8, dt=B, out=P, fin=None, chk=None, ws=WS,
                             wsb=1 << 40, stream=None),
    "kda_scan_decode_step": dict(x=P, g=P, state=P, N=1, D=8, dt=B, out=P, stream=None),
    "kda_scan_backward": dict(x=P, g=P, init=None, cu=P, N=1, T=300, D=8, dt=B, dout=P, dfin=None, chk=None, dx=P,
                              dg=P, dinit=None, ws=WS, wsb=1 << 40, stream=None),
    "kda_conv_prefill": dict(x=P, w=P, b=None, init=None, cu=P, N=1, T=300, D=8, W=4, silu=1, dt=B, out=Q, fin=None,
                             stream=None),
    "kda_conv_decode_step": dict(x=P, w=P, b=None, state=P, N=1, D=8, W=4, silu=1, dt=B, out=P, stream=None),
    "kda_conv_backward": dict(x=P, w=P, b=None, init=None, cu=P, N=1, T=300, D=8, W=4, silu=1, dt=B, dout=P,
                              dfin=None, dx=Q, dw=P, db=None, dinit=None, ws=WS, wsb=1 << 40, stream=None),
    "kda_rmsnorm": dict(x=P, res=None, w=P, rows=4, D=64, eps=1e-6, dt=B, sum=None, out=P, mx=None, sc=None,
                        stream=None),
    "kda_rmsnorm_backward": dict(x=P, w=P, dout=P, dres=None, rows=4, D=64, eps=1e-6, dt=B, dx=P, dw=P, ws=WS,
                                 wsb=1 << 40, stream=None),
}


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(K.LIB_PATH):
        from gated_delta_rule_40_amd import build
        build.build()
    return K.load()


def call(lib, name, **kw):
    a = dict(CALLS[name])
    assert set(kw) <= set(a)
    a.update(kw)
    return getattr(lib, name)(*a.values())


BAD = [(name, {field: None}) for name, fields in (
    ("kda_scan_prefill", "x g cu out"), ("kda_scan_decode_step", "x g state out"),
    ("kda_scan_backward", "x g cu dout dx dg"), ("kda_conv_prefill", "x w cu out"),
    ("kda_conv_decode_step", "x w state out"), ("kda_conv_backward", "x w cu dout dx dw"), ("kda_rmsnorm", "x out"),
    ("kda_rmsnorm_backward", "x dout dx")) for field in fields.split()]
BAD += [(name, {field: ODD}) for name, a in CALLS.items() for field, v in a.items()
        if v in (P, Q) or v is None and field in ("init", "fin", "dfin", "chk", "dinit", "b", "db", "res", "dres", "sum")
        if not (name == "kda_rmsnorm" and field == "sum")]
BAD += [(name, {"dt": 7}) for name in CALLS]
BAD += [(name, {"D": d}) for name in CALLS for d in (0, -3)]
BAD += [(name, {"N": -1}) for name, a in CALLS.items() if "N" in a]
BAD += [(name, {"T": -1}) for name, a in CALLS.items() if "T" in a]
BAD += [(name, {"rows": -1}) for name, a in CALLS.items() if "rows" in a]
BAD += [(name, {"W": w}) for name, a in CALLS.items() if "W" in a for w in (0, -2)]
BAD += [(name, {"eps": e}) for name, a in CALLS.items() if "eps" in a for e in (-1e-6, float("nan"), float("inf"))]
BAD += [(name, {"N": 2 ** 31 - 65536}) for name in ("kda_scan_prefill", "kda_scan_backward", "kda_conv_prefill",
                                                    "kda_conv_backward")]
# arrays that overlap: token arrays moved by 16 bytes or, where that is not allowed, in place; states likewise
BAD += [("kda_scan_prefill", {"x": Q, "out": Q2}), ("kda_scan_prefill", {"init": Q, "fin": Q2}),
        ("kda_scan_backward", {"x": Q, "dx": Q2}), ("kda_scan_backward", {"dout": Q2, "dx": Q}),
        ("kda_scan_backward", {"g": Q2, "dg": Q}), ("kda_scan_backward", {"init": Q, "dinit": Q}),
        ("kda_scan_backward", {"dfin": Q, "dinit": Q}), ("kda_conv_prefill", {"x": Q}),
        ("kda_conv_prefill", {"x": Q2}), ("kda_conv_prefill", {"init": P, "fin": ctypes.c_void_p(0x10010)}),
        ("kda_conv_backward", {"x": Q}), ("kda_conv_backward", {"dout": Q2}),
        ("kda_conv_backward", {"init": P, "dinit": P}), ("kda_conv_backward", {"dfin": P, "dinit": P}),
        ("kda_scan_decode_step", {"N": 8, "x": Q, "out": Q2}), ("kda_conv_decode_step", {"N": 8, "x": Q2, "out": Q}),
        ("kda_rmsnorm", {"x": Q, "out": Q2}), ("kda_rmsnorm", {"res": Q, "out": Q2}),
        ("kda_rmsnorm", {"x": P, "res": Q, "sum": Q2}), ("kda_rmsnorm", {"res": Q, "sum": Q, "out": Q}),
        ("kda_rmsnorm_backward", {"x": Q, "dx": Q2}), ("kda_rmsnorm_backward", {"dout": Q, "dx": Q2}),
        ("kda_rmsnorm_backward", {"dres": Q2, "dx": Q})]
BAD += [("kda_rmsnorm", {"sum": P}),                    # a sum without a residual
        ("kda_rmsnorm", {"mx": P}), ("kda_rmsnorm", {"sc": P}), ("kda_rmsnorm", {"res": P, "sum": ODD})]


@pytest.mark.parametrize("name,kw", BAD, ids=["%s-%s" % (n, "-".join("%s=%s" % (k, getattr(v, "value", v))
                                                                     for k, v in kw.items())) for n, kw in BAD])
def test_rejects(lib, name, kw):
    assert call(lib, name, **kw) == INVALID


@pytest.mark.parametrize("name,kw", [
    ("kda_conv_prefill", dict(W=5)), ("kda_conv_prefill", dict(W=1)), ("kda_conv_decode_step", dict(W=5)),
    ("kda_conv_backward", dict(W=1)), ("kda_conv_backward", dict(W=8)), ("kda_rmsnorm", dict(D=16385)),
    ("kda_rmsnorm_backward", dict(D=16385)),
    # launches of 2^32 threads and more
    ("kda_scan_prefill", dict(T=2 ** 30 + 1, D=1, N=4)), ("kda_scan_backward", dict(T=2 ** 30 + 1, D=1, N=4)),
    ("kda_scan_prefill", dict(N=2 ** 27)), ("kda_conv_decode_step", dict(N=2 ** 31 - 1, D=1)),
    ("kda_conv_prefill", dict(N=2 ** 30, init=None, fin=ctypes.c_void_p(1 << 40))),
    ("kda_conv_backward", dict(D=2 ** 28, T=1, x=ctypes.c_void_p(1 << 40), dout=ctypes.c_void_p(1 << 41))),
    ("kda_rmsnorm", dict(rows=2 ** 31 - 1, D=1)),
])
def test_does_not_support(lib, name, kw):
    assert call(lib, name, **kw) == UNSUPPORTED


@pytest.mark.parametrize("name,kw", [
    ("kda_scan_prefill", dict(N=0, T=0, x=None, g=None, out=None, ws=None, wsb=0)), ("kda_scan_prefill", dict(N=0)),
    ("kda_scan_decode_step", dict(N=0, x=None, g=None, state=None, out=None)),
    ("kda_scan_backward", dict(N=0, T=0, x=None, g=None, dout=None, dx=None, dg=None, ws=None, wsb=0)),
    ("kda_conv_prefill", dict(N=0, T=0, x=None, out=None)), ("kda_conv_prefill", dict(N=0)),
    ("kda_conv_decode_step", dict(N=0, x=None, state=None, out=None)),
    ("kda_rmsnorm", dict(rows=0, x=None, out=None)),
    ("kda_rmsnorm_backward", dict(rows=0, x=None, dout=None, dx=None, dw=None, ws=None, wsb=0)),
])
def test_nothing_to_do_is_a_no_op(lib, name, kw):
    assert call(lib, name, **kw) == K.KDA_OK


def _sizes(lib):
    return {"kda_scan_backward": lib.kda_scan_backward_workspace_size(1, 300, 8, B, 0),
            "kda_scan_prefill": lib.kda_scan_workspace_size(1, 300, 8, B),
            "kda_conv_backward": lib.kda_conv_backward_workspace_size(1, 300, 8, 4, B),
            "kda_rmsnorm_backward": lib.kda_rmsnorm_backward_workspace_size(4, 64, B)}


@pytest.mark.parametrize("name", ["kda_scan_prefill", "kda_scan_backward", "kda_conv_backward", "kda_rmsnorm_backward"])
def test_workspace_is_checked(lib, name):
    need = _sizes(lib)[name]
    if need == 0:
        pytest.skip("needs no workspace at this size")
    assert call(lib, name, ws=None) == INVALID
    assert call(lib, name, ws=ODD) == INVALID
    assert call(lib, name, wsb=need - 1) == INVALID


def test_workspace_sizes_of_bad_sizes_are_zero(lib):
    assert lib.kda_scan_workspace_size(-1, 300, 8, B) == lib.kda_scan_workspace_size(1, 300, 0, B) == 0
    assert lib.kda_scan_backward_workspace_size(1, -1, 8, B, 0) == lib.kda_scan_backward_workspace_size(1, 300, 8, 9, 0) == 0
    assert lib.kda_conv_backward_workspace_size(1, 300, 8, 5, B) == lib.kda_conv_backward_workspace_size(1, 300, -8, 4, B) == 0
    assert lib.kda_rmsnorm_backward_workspace_size(-4, 64, B) == lib.kda_rmsnorm_backward_workspace_size(4, 20000, B) == 0


def test_binding_rejects_host_tensors():
    x, g, cu = torch.zeros(4, 8), torch.zeros(4, 8), torch.tensor([0, 4], dtype=torch.int32)
    w = torch.zeros(8, 4)
    for fn, args in ((K.kda_scan_prefill, (x, g, None, cu, x, None)), (K.kda_scan_decode_step, (x, g, g, x)),
                     (K.kda_scan_backward, (x, g, None, cu, x)), (K.kda_conv_prefill, (x, w, None, None, cu, x, None)),
                     (K.kda_conv_decode_step, (x, w, None, torch.zeros(4, 3, 8), x)),
                     (K.kda_conv_backward, (x, w, None, None, cu, x)), (K.kda_rmsnorm, (x, None, x)),
                     (K.kda_rmsnorm_backward, (x, None, x))):
        with pytest.raises(ValueError, match="device tensor"):
            fn(*args)


def test_binding_workspace_sizes_reject_unknown_types():
    for fn, args in ((K.kda_scan_workspace_size, (1, 16, 8)), (K.kda_scan_backward_workspace_size, (1, 16, 8)),
                     (K.kda_conv_backward_workspace_size, (1, 16, 8, 4)), (K.kda_rmsnorm_backward_workspace_size, (4, 8))):
        with pytest.raises(TypeError):
            fn(*args, torch.float16)


# ------------------------------------------------------------------ overlaps, every output against every other argument
# Sizes in bytes for 300 tokens of 40 channels in 3 sequences (decode: 3 tokens), bf16, width 4; norm: 300 rows of 40.
def _arrays(lib):
    tok, f32, st, row, cu = 300 * 40 * 2, 300 * 40 * 4, 3 * 40 * 4, 40 * 4, 4 * 4
    conv, chk, w = 3 * 3 * 40 * 2, 3 * 40 * 4, 40 * 4 * 4
    return {   # name: (arguments as in CALLS, their sizes, outputs: inputs each may equal)
        "kda_scan_prefill": (dict(N=3, D=40), dict(x=tok, g=f32, init=st, cu=cu, out=tok, fin=st, chk=chk,
                                                   ws=lib.kda_scan_workspace_size(3, 300, 40, B)),
                             dict(out="x", fin="init", chk="", ws="")),
        "kda_scan_decode_step": (dict(N=3, D=40), dict(x=240, g=480, state=480, out=240), dict(out="x", state="")),
        "kda_scan_backward": (dict(N=3, D=40), dict(x=tok, g=f32, init=st, cu=cu, dout=tok, dfin=st, chk=chk, dx=tok,
                                                    dg=f32, dinit=st,
                                                    ws=lib.kda_scan_backward_workspace_size(3, 300, 40, B, 1)),
                              dict(dx="x dout", dg="g", dinit="", ws="")),
        "kda_conv_prefill": (dict(N=3, D=40), dict(x=tok, w=w, b=row, init=conv, cu=cu, out=tok, fin=conv),
                             dict(out="", fin="init")),
        "kda_conv_decode_step": (dict(N=3, D=40), dict(x=240, w=w, b=row, state=conv, out=240), dict(out="x", state="")),
        "kda_conv_backward": (dict(N=3, D=40), dict(x=tok, w=w, b=row, init=conv, cu=cu, dout=tok, dfin=conv, dx=tok, dw=w,
                                                    db=row, dinit=conv,
                                                    ws=lib.kda_conv_backward_workspace_size(3, 300, 40, 4, B)),
                              dict(dx="", dw="", db="", dinit="", ws="")),
        "kda_rmsnorm": (dict(rows=300, D=40), dict(x=tok, res=tok, w=row, sum=tok, out=tok, mx=300 * 40, sc=300 * 2),
                        dict(sum="x res", out="x res", mx="", sc="")),
        "kda_rmsnorm_backward": (dict(rows=300, D=40), dict(x=tok, w=row, dout=tok, dres=tok, dx=tok, dw=row,
                                                            ws=lib.kda_rmsnorm_backward_workspace_size(300, 40, B)),
                                 dict(dx="x dout dres", dw="", ws="")),
    }


def _places(lib):
    """Every output moved onto every other argument: (call, its arguments, whether the output may lie there)."""
    for name, (sizes, arrays, outs) in _arrays(lib).items():
        at = {a: (i + 1) << 24 for i, a in enumerate(arrays)}
        assert all(0 < n < 1 << 24 for n in arrays.values())
        for o, may in outs.items():
            for a in set(arrays) - {o}:
                # on its first byte, on its last bytes, and so that it ends on its first (offsets of 8 bytes)
                for p in {at[a], at[a] + (arrays[a] - 1) // 8 * 8, at[a] - (arrays[o] - 1) // 8 * 8}:
                    kw = {k: ctypes.c_void_p(v) for k, v in {**at, o: p}.items()}
                    yield name, {**sizes, **kw}, p == at[a] and a in may.split()
                for p in (at[a] + (arrays[a] + 7) // 8 * 8, at[a] - (arrays[o] + 7) // 8 * 8):     # beside it
                    yield name, {**sizes, **{k: ctypes.c_void_p(v) for k, v in {**at, o: p}.items()}}, True


def test_overlaps_are_refused(lib):
    refused = taken = 0
    for name, kw, may in _places(lib):
        if not may:
            assert call(lib, name, **kw) == INVALID, (name, kw)
            refused += 1
        elif not torch.cuda.is_available():   # these addresses would reach a kernel: only where there is none
            assert call(lib, name, **kw) == K.KDA_ERR_LAUNCH, (name, kw)
            taken += 1
    assert refused > 500 and (taken > 300 or torch.cuda.is_available())
