"""Refusals of the norm and rotation of queries and keys, the cache of states, the
decoding on it and the verification of drafts that need no GPU: the C entry
points return the documented status before any HIP call, and the binding raises
for host tensors."""
import ctypes
import os

import pytest
import torch

from gated_delta_rule_40_amd import libkda as K

ptr = ctypes.c_void_p
ODD = ptr(0x10001)
B, F = K.KDA_BF16, K.KDA_F32
INVALID, UNSUPPORTED = K.KDA_ERR_INVALID_ARG, K.KDA_ERR_UNSUPPORTED
L2 = K.KDA_NORMS["l2"]


def at(i):
    """Array number i: aligned addresses 256 MiB apart, never dereferenced."""
    return ptr((i + 1) << 28)


# 300 tokens, 4 query and 2 key heads of 64 with 32 rotated; 3 sequences of 4 heads; 5 entries of 100 values; 70 tokens
CALLS = {
    "kda_qknorm": dict(q=at(0), k=at(1), qs=256, ks=128, qw=at(2), kw=at(3), pos=at(4), freq=at(5), axis=at(6), T=300, Hq=4,
                       Hk=2, d=64, rot=32, axes=2, inter=0, norm=L2, eps=1e-6, scale=1.0, dt=B, q_out=at(7), k_out=at(8),
                       stream=None),
    "kda_qknorm_backward": dict(q=at(0), k=at(1), qs=256, ks=128, qw=at(2), kw=at(3), pos=at(4), freq=at(5), axis=at(6),
                                T=300, Hq=4, Hk=2, d=64, rot=32, axes=2, inter=0, norm=L2, eps=1e-6, scale=1.0, dt=B, gdt=F,
                                dq_out=at(7), dk_out=at(8), dqs=256, dks=128, dq=at(9), dk=at(10), dqw=at(11), dkw=at(12),
                                ws=at(13), wsb=1 << 24, stream=None),
    "kda_cache_store": dict(src=at(0), slots=at(1), n=5, elems=100, dt=B, fmt=0, S=7, cache=at(2), scales=at(3), stream=None),
    "kda_cache_load": dict(cache=at(2), scales=at(3), slots=at(1), n=5, elems=100, dt=B, fmt=0, S=7, dst=at(0), stream=None),
    "kda_decode_tokens_cached": dict(q=at(0), k=at(1), v=at(2), g=at(3), beta=at(4), cu=at(5), num=at(6), cache=at(7),
                                     scales=at(8), slots=at(9), write=1, S=7, N=3, T=70, H=4, dk=128, dv=128, dt=B, fmt=0,
                                     out=at(10), stream=None),
    "kda_verify_drafts": dict(target=at(0), draft=at(1), tokens=at(2), cu=at(3), accept=at(4), sample=at(5), N=3, T=70,
                              V=1000, dt=B, num=at(6), next=at(7), ws=at(8), wsb=1 << 24, stream=None),
}
# sizes in bytes of the arrays above, and which outputs may lie whole in the place of which input
HEADS, KHEADS = 300 * 256 * 2, 300 * 128 * 2
TOK = 70 * 4 * 128
ARRAYS = {
    "kda_qknorm": (dict(q=HEADS, k=KHEADS, qw=256, kw=256, pos=2400, freq=64, axis=64, q_out=HEADS, k_out=KHEADS),
                   dict(q_out="q", k_out="k")),
    "kda_qknorm_backward": (dict(q=HEADS, k=KHEADS, qw=256, kw=256, pos=2400, freq=64, axis=64, dq_out=2 * HEADS,
                                 dk_out=2 * KHEADS, dq=HEADS, dk=KHEADS, dqw=256, dkw=256, ws=2 * 512 * 64 * 4),
                            dict(dq="q", dk="k", dqw="", dkw="", ws="")),
    "kda_cache_store": (dict(src=1000, slots=20, cache=700, scales=28), dict(cache="", scales="")),
    "kda_cache_load": (dict(cache=700, scales=28, slots=20, dst=1000), dict(dst="")),
    "kda_decode_tokens_cached": (dict(q=2 * TOK, k=2 * TOK, v=2 * TOK, g=4 * TOK, beta=70 * 16, cu=16, num=12,
                                      cache=7 * 4 * 128 * 128, scales=7 * 4 * 128 * 4, slots=12, out=2 * TOK),
                                 dict(cache="", scales="", out="")),
    "kda_verify_drafts": (dict(target=140000, draft=140000, tokens=280, cu=16, accept=280, sample=12, num=12, next=12, ws=36),
                          dict(num="", next="", ws="")),
}


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(K.LIB_PATH):
        from gated_delta_rule_40_amd import build
        build.build()
    return K.load()


def call(lib, name, **kw):
    a = dict(CALLS[name])
    assert set(kw) <= set(a), set(kw) - set(a)
    a.update(kw)
    return getattr(lib, name)(*a.values())


BAD = [(name, {f: None}) for name, fields in (
    ("kda_qknorm", "q k pos freq q_out k_out"), ("kda_qknorm_backward", "q k pos freq dq_out dk_out dq dk ws"),
    ("kda_cache_store", "src slots cache scales"), ("kda_cache_load", "dst slots cache scales"),
    ("kda_decode_tokens_cached", "q k v g beta cu cache scales slots"),
    ("kda_verify_drafts", "target tokens cu accept sample num next ws")) for f in fields.split()]
BAD += [(name, {f: ODD}) for name, a in CALLS.items() for f, v in a.items()
        if isinstance(v, ptr) and f not in ("cache", "scales")]
BAD += [(name, {"dt": 7}) for name in CALLS] + [("kda_qknorm_backward", {"gdt": 7}),
                                                 ("kda_qknorm_backward", {"dt": F, "gdt": B, "qs": 256})]
BAD += [(name, {f: v}) for name, a in CALLS.items() for f, vs in (
    ("T", (-1,)), ("N", (-1, 2 ** 31 - 65536)), ("S", (-1,)), ("n", (-1,)), ("elems", (0, -5)), ("H", (0, -1)), ("dk", (0,)),
    ("dv", (-1,)), ("V", (0, -1)), ("Hq", (-1, 2 ** 25)), ("Hk", (-1, 2 ** 25)), ("d", (0, -64)), ("rot", (-2, 31, 66)),
    ("axes", (0, -1)), ("norm", (-1, 3)), ("fmt", (-1, 3)), ("eps", (-1e-6, float("nan"), float("inf"))),
    ("scale", (float("nan"), float("inf"))), ("qs", (255, 2 ** 29 + 1)), ("ks", (127, -128)), ("dqs", (0, 2 ** 29 + 1)),
    ("dks", (127,)), ("wsb", (0,))) if f in a for v in vs]
BAD += [("kda_qknorm_backward", {"qw": None}), ("kda_qknorm_backward", {"kw": None}),   # a gradient of no weight
        ("kda_decode_tokens_cached", {"out": None, "write": 0})]                         # nothing to give


@pytest.mark.parametrize("name,kw", BAD, ids=["%s-%s" % (n, "-".join("%s=%s" % (k, getattr(v, "value", v))
                                                                     for k, v in kw.items())) for n, kw in BAD])
def test_rejects(lib, name, kw):
    assert call(lib, name, **kw) == INVALID


@pytest.mark.parametrize("name,kw", [
    ("kda_qknorm", dict(d=513, qs=4096, ks=4096)), ("kda_qknorm_backward", dict(d=514, qs=4096, ks=4096, dqs=4096, dks=4096)),
    ("kda_decode_tokens_cached", dict(dk=64)), ("kda_decode_tokens_cached", dict(dv=256)),
    ("kda_verify_drafts", dict(V=2 ** 30 + 1, draft=None, target=ptr(1 << 45))),
    # launches of 2^32 threads and more
    ("kda_qknorm", dict(T=2 ** 31 - 1, rot=0, q=ptr(1 << 44), k=ptr(2 << 44), q_out=ptr(3 << 44), k_out=ptr(4 << 44))),
    ("kda_cache_store", dict(n=2 ** 25, elems=2 ** 12, src=ptr(1 << 44))),
    ("kda_cache_load", dict(n=2 ** 25, elems=2 ** 12, dst=ptr(1 << 44))),
    ("kda_decode_tokens_cached", dict(N=2 ** 23, slots=ptr(1 << 44), num=None)),
    ("kda_verify_drafts", dict(N=2 ** 25, num=ptr(1 << 44), next=ptr(2 << 44), sample=ptr(3 << 44), cu=ptr(4 << 44),
                               ws=ptr(5 << 44), wsb=2 ** 40)),
])
def test_does_not_support(lib, name, kw):
    assert call(lib, name, **kw) == UNSUPPORTED


@pytest.mark.parametrize("name,kw", [
    ("kda_qknorm", dict(T=0, q=None, k=None, q_out=None, k_out=None, pos=None)),
    ("kda_qknorm", dict(Hq=0, Hk=0, q=None, k=None, q_out=None, k_out=None, freq=None)),
    ("kda_qknorm_backward", dict(T=0, q=None, k=None, dq_out=None, dk_out=None, dq=None, dk=None, dqw=None, dkw=None, ws=None,
                                 wsb=0)),
    ("kda_cache_store", dict(n=0, src=None, slots=None)), ("kda_cache_store", dict(S=0, cache=None, scales=None)),
    ("kda_cache_load", dict(n=0, dst=None, slots=None)),
    ("kda_decode_tokens_cached", dict(N=0, slots=None)),
    ("kda_decode_tokens_cached", dict(T=0, q=None, k=None, v=None, g=None, beta=None, out=None, write=0)),
    ("kda_verify_drafts", dict(N=0, sample=None, num=None, next=None, ws=None, wsb=0)),
])
def test_nothing_to_do_is_a_no_op(lib, name, kw):
    assert call(lib, name, **kw) == K.KDA_OK


def _places():
    """Every output moved onto every other argument: (call, its addresses, whether the output may lie there)."""
    for name, (sizes, outs) in ARRAYS.items():
        base = {a: v.value for a, v in CALLS[name].items() if isinstance(v, ptr)}
        assert set(base) == set(sizes), (name, set(base) ^ set(sizes))
        for o, may in outs.items():
            for a in set(sizes) - {o}:
                # on its first byte, on its last bytes, and so that it ends on its first (offsets of 8 bytes)
                for p in {base[a], base[a] + (sizes[a] - 1) // 8 * 8, base[a] - (sizes[o] - 1) // 8 * 8}:
                    yield name, {k: ptr(v) for k, v in {**base, o: p}.items()}, p == base[a] and a in may.split()
                for p in (base[a] + (sizes[a] + 7) // 8 * 8, base[a] - (sizes[o] + 7) // 8 * 8):     # beside it
                    yield name, {k: ptr(v) for k, v in {**base, o: p}.items()}, True


def test_overlaps_are_refused(lib):
    refused = taken = 0
    for name, kw, may in _places():
        if not may:
            assert call(lib, name, **kw) == INVALID, (name, kw)
            refused += 1
        elif not torch.cuda.is_available():   # these addresses would reach a kernel: only where there is none
            assert call(lib, name, **kw) == K.KDA_ERR_LAUNCH, (name, kw)
            taken += 1
    assert refused > 250 and (taken > 150 or torch.cuda.is_available())


def test_a_cache_that_is_only_read_may_not_be_written_over(lib):
    for a in ("cache", "scales"):
        assert call(lib, "kda_decode_tokens_cached", write=0, out=CALLS["kda_decode_tokens_cached"][a]) == INVALID


def test_columns_of_one_projection(lib):
    """q, k and their gradients as columns of the same rows: apart where the columns are, refused where they meet."""
    if torch.cuda.is_available():
        pytest.skip("these addresses would reach a kernel")
    x, y = 1 << 28, 2 << 28
    rows = dict(q=ptr(x), k=ptr(x + 512), qs=400, ks=400)
    grads = dict(dq=ptr(y), dk=ptr(y + 512), dqs=400, dks=400)
    assert call(lib, "kda_qknorm", **rows) == K.KDA_ERR_LAUNCH
    assert call(lib, "kda_qknorm_backward", **rows, **grads) == K.KDA_ERR_LAUNCH
    assert call(lib, "kda_qknorm_backward", **rows, **{**grads, "dk": ptr(y + 510)}) == INVALID
    assert call(lib, "kda_qknorm_backward", **rows, **{**grads, "dk": ptr(y + 512 + 34)}) == INVALID   # into the next row
    assert call(lib, "kda_qknorm_backward", **rows, **{**grads, "dk": ptr(y + 512 + 32)}) == K.KDA_ERR_LAUNCH
    assert call(lib, "kda_qknorm_backward", **rows, **{**grads, "dks": 401}) == INVALID                # columns that wander
    # gradients in the place of the rows
    assert call(lib, "kda_qknorm_backward", **rows, dq=rows["q"], dk=rows["k"], dqs=400, dks=400) == K.KDA_ERR_LAUNCH
    assert call(lib, "kda_qknorm_backward", **rows, dq=rows["q"], dk=rows["k"], dqs=400, dks=500) == INVALID
    assert call(lib, "kda_qknorm", **rows, q_out=ptr(x)) == INVALID                                    # not dense


def test_sizes(lib):
    assert [K.kda_cache_entry_bytes(n, f) for f in ("fp8", "int8", "fp4") for n in (0, 1, 32, 101)] == \
        [0, 1, 32, 101, 0, 1, 32, 101, 0, 1, 16, 51]
    assert lib.kda_cache_entry_bytes(-1, 0) == lib.kda_cache_entry_bytes(8, 3) == 0
    assert lib.kda_qknorm_backward_workspace_size(300, 4, 2, 64, B) > 0
    assert lib.kda_qknorm_backward_workspace_size(-1, 4, 2, 64, B) == lib.kda_qknorm_backward_workspace_size(1, 4, 2, 513, B) == 0
    assert lib.kda_verify_drafts_workspace_size(3, 1000, F) > 0
    assert lib.kda_verify_drafts_workspace_size(-1, 1000, F) == lib.kda_verify_drafts_workspace_size(3, 0, F) == 0
    need = lib.kda_verify_drafts_workspace_size(3, 1000, B)
    assert call(lib, "kda_verify_drafts", wsb=need - 1) == INVALID
    need = lib.kda_qknorm_backward_workspace_size(300, 4, 2, 64, B)
    assert call(lib, "kda_qknorm_backward", wsb=need - 1) == INVALID


def test_binding_rejects_host_tensors_and_names():
    x, cu, n = torch.zeros(4, 2, 128), torch.tensor([0, 4], dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    by = torch.zeros(2, 256, dtype=torch.uint8)
    for fn, args in ((K.kda_qknorm, (x, x, x, x)), (K.kda_qknorm_backward, (x, x, x, x)),
                     (K.kda_cache_store, (x, n, by, by)), (K.kda_cache_load, (by, by, n, x)),
                     (K.kda_decode_tokens_cached, (x, x, x, x, x, cu, by, by, n)),
                     (K.kda_verify_drafts, (x, x, n, cu, x, x, n, n))):
        with pytest.raises(ValueError, match="device tensor"):
            fn(*args)
    with pytest.raises(ValueError, match="format"):
        K.kda_cache_entry_bytes(8, "fp6")
    for fn, args in ((K.kda_qknorm_backward_workspace_size, (1, 1, 1, 8)), (K.kda_verify_drafts_workspace_size, (1, 8))):
        with pytest.raises(TypeError):
            fn(*args, torch.float16)
