"""The layer operators in a row, as a KDA layer uses them: norm with the
residual, convolution of the q, k and v channels, the recurrence, a norm for
each head; and the gated linear recurrence in the recurrence's place, forward,
backward and token by token."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import layer_ref as R
from gated_delta_rule_40_amd import libkda as K

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    K.load()


def host(t):
    return t.detach().double().cpu().numpy()


LENS = [70, 0, 1, 200, 33]
CU = [0] + list(np.cumsum(LENS))


def block(D=96, W=4, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    T, N = sum(LENS), len(LENS)
    return dict(x=rnd(T, D), res=rnd(T, D), nw=1 + 0.1 * rnd(D), cw=0.5 * rnd(D, W), cb=0.1 * rnd(D),
                cinit=rnd(N, W - 1, D), g=-0.3 * torch.rand(T, D, generator=gen), hinit=rnd(N, D),
                dout=rnd(T, D), dsum=rnd(T, D), cu=torch.tensor(CU, dtype=torch.int32))


def forward(d, chk=None):
    e = torch.empty_like
    total, y, u, cfin, h, hfin = e(d["x"]), e(d["x"]), e(d["x"]), e(d["cinit"]), e(d["x"]), e(d["hinit"])
    K.kda_rmsnorm(d["x"], d["nw"], y, residual=d["res"], residual_out=total)
    K.kda_conv_prefill(y, d["cw"], d["cb"], d["cinit"], d["cu"], u, cfin)
    K.kda_scan_prefill(u, d["g"], d["hinit"], d["cu"], h, hfin, checkpoints=chk)
    return total, y, u, cfin, h, hfin


def plain_block(d):
    """The same in torch, fp64, with a graph for autograd."""
    r = d["x"] + d["res"]
    y = r / torch.sqrt((r * r).mean(1, keepdim=True) + 1e-6) * d["nw"]
    outs, W = [], d["cw"].shape[1]
    for n in range(len(LENS)):
        rows = torch.cat((d["cinit"][n], y[CU[n]:CU[n + 1]]))
        h = d["hinit"][n]
        for p in range(LENS[n]):
            pre = (rows[p:p + W] * d["cw"].t()).sum(0) + d["cb"]
            h = torch.exp(d["g"][CU[n] + p]) * h + pre * torch.sigmoid(pre)
            outs.append(h)
    return r, torch.stack(outs)


def test_forward_and_backward_through_the_block():
    hd = block()
    leaves = {k: hd[k].double().requires_grad_() for k in ("x", "res", "nw", "cw", "cb", "cinit", "g", "hinit")}
    r, h = plain_block(leaves)
    ((h * hd["dout"].double()).sum() + (r * hd["dsum"].double()).sum()).backward()
    d = {k: v.cuda() for k, v in hd.items()}
    chk = torch.empty(-(-sum(LENS) // 128), 96, device="cuda")
    total, y, u, _, out, _ = forward(d, chk)
    gs = K.kda_scan_backward(u, d["g"], d["hinit"], d["cu"], d["dout"], checkpoints=chk)
    gc = K.kda_conv_backward(y, d["cw"], d["cb"], d["cinit"], d["cu"], gs["dx"])
    gn = K.kda_rmsnorm_backward(total, d["nw"], gc["dx"], dresidual=d["dsum"])
    got = dict(x=gn["dx"], res=gn["dx"], nw=gn["dweight"], cw=gc["dweight"], cb=gc["dbias"], cinit=gc["dinit"],
               g=gs["dg"], hinit=gs["dinit"])
    # fp32 throughout: three operators of at most a few hundred roundings of 2^-24 each, relative to the largest value
    near = lambda a, b: float((a.double().cpu() - b).abs().max() / b.abs().max())   # noqa: E731
    assert near(out, h.detach()) < 1000 * 2.0 ** -24
    for k, v in got.items():
        assert near(v, leaves[k].grad) < 3000 * 2.0 ** -24, k


def test_gradient_against_differences():
    # the kernels' own forward, stepped: a central difference of the loss along a direction against the gradient
    d = {k: v.cuda() for k, v in block(seed=1).items()}

    def loss(dd):
        return float((forward(dd)[4].double() * d["dout"].double()).sum())

    _, y, u, _, _, _ = forward(d)
    gs = K.kda_scan_backward(u, d["g"], d["hinit"], d["cu"], d["dout"])
    gc = K.kda_conv_backward(y, d["cw"], d["cb"], d["cinit"], d["cu"], gs["dx"])
    gen = torch.Generator(device="cuda").manual_seed(5)
    for name, grad in (("g", gs["dg"]), ("hinit", gs["dinit"]), ("cw", gc["dweight"]), ("cb", gc["dbias"]),
                       ("cinit", gc["dinit"])):
        v = torch.randn(grad.shape, device="cuda", generator=gen) * (0.05 if name == "g" else 1.0)
        eps = 2.0 ** -7
        diff = (loss({**d, name: d[name] + eps * v}) - loss({**d, name: d[name] - eps * v})) / (2 * eps)
        slope = float((grad.double() * v.double()).sum())
        # third-order term: eps^2 / 6 of a third derivative; the sum's scale stands for it (measured in fp64: < 1e-3)
        scale = float((grad.double().abs() * v.double().abs()).sum())
        assert abs(diff - slope) < 2e-3 * scale, (name, diff, slope, scale)


def test_tokens_one_by_one_equal_the_prompt():
    d = {k: v.cuda() for k, v in block(seed=2).items()}
    N, L, D = 3, 33, 96
    x, res, g = (d[k][:N * L].view(N, L, D) for k in ("x", "res", "g"))
    d2 = dict(d, x=d["x"][:N * L].contiguous(), res=d["res"][:N * L].contiguous(), g=d["g"][:N * L].contiguous(),
              cinit=d["cinit"][:N].contiguous(), hinit=d["hinit"][:N].contiguous(),
              cu=torch.arange(N + 1, dtype=torch.int32, device="cuda") * L)
    _, _, _, cfin, h, hfin = forward(d2)
    conv, state = d2["cinit"].clone(), d2["hinit"].clone()
    y, total, u, o = (torch.empty(N, D, device="cuda") for _ in range(4))
    for p in range(L):
        K.kda_rmsnorm(x[:, p].contiguous(), d["nw"], y, residual=res[:, p].contiguous(), residual_out=total)
        K.kda_conv_decode_step(y, d["cw"], d["cb"], conv, u)
        K.kda_scan_decode_step(u, g[:, p].contiguous(), state, o)
        assert float((o - h.view(N, L, D)[:, p]).abs().max()) < 1000 * 2.0 ** -24 * float(h.abs().max())
    assert torch.allclose(conv, cfin, rtol=0, atol=100 * 2.0 ** -24 * float(cfin.abs().max()))
    assert torch.allclose(state, hfin, rtol=0, atol=1000 * 2.0 ** -24 * float(hfin.abs().max()))


def test_around_the_delta_rule():
    # q, k and v through one convolution, the KDA recurrence, a norm for each head: shapes meet without copies
    T, H, D, N = sum(LENS), 2, 128, len(LENS)
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    qkv = [(rnd(T, H, D) * 0.3).bfloat16().cuda() for _ in range(3)]
    w = (0.4 * rnd(H, D, 4)).cuda()
    g, beta = (-0.3 * torch.rand(T, H, D, generator=gen)).cuda(), torch.rand(T, H, generator=gen).cuda()
    cu = torch.tensor(CU, dtype=torch.int32, device="cuda")
    conv = [torch.empty_like(t) for t in qkv]
    for a, b in zip(qkv, conv):
        K.kda_conv_prefill(a, w, None, None, cu, b, None)
    out, fin = torch.empty_like(conv[2]), torch.empty(N, H, D, D, device="cuda")
    K.kda_prefill(*conv, g, beta, None, cu, out, fin)
    y = torch.empty_like(out)
    mx = torch.empty(T, H, D, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(T, H, 4, dtype=torch.float8_e8m0fnu, device="cuda")
    K.kda_rmsnorm(out, None, y, out_mx=mx, scales=sc)
    f = R.conv(host(qkv[0]).reshape(T, H * D), host(w).reshape(H * D, 4), None, None, CU, True)
    R.close(host(conv[0]).reshape(T, H * D), f["out"], f["e_out"], "bf16", "conv of q")
    n = R.rmsnorm(host(out).reshape(T * H, D), None, None, 1e-6)
    R.close(host(y).reshape(T * H, D), n["y"], n["e_y"], "bf16", "norm of a head")
    back = mx.float() * sc.float().repeat_interleave(32, 2)
    assert float((back - y.float()).abs().max()) <= (2.0 ** -4 + 2.0 ** -8) * float(y.float().abs().max())


CHILD = r'''
import sys, torch
sys.path.insert(0, %(root)r)
from gated_delta_rule_40_amd import libkda as K
T, D = 70, 16
x, g, w = torch.randn(T, D, device="cuda"), -torch.rand(T, D, device="cuda"), torch.randn(D, 4, device="cuda")
o = torch.empty_like(x)
calls = {"kda_scan_prefill": lambda cu: K.kda_scan_prefill(x, g, None, cu, o, None),
         "kda_scan_backward": lambda cu: K.kda_scan_backward(x, g, None, cu, x),
         "kda_conv_prefill": lambda cu: K.kda_conv_prefill(x, w, None, None, cu, o, None),
         "kda_conv_backward": lambda cu: K.kda_conv_backward(x, w, None, None, cu, x)}
for name, fn in calls.items():
    fn(torch.tensor([0, 40, 70], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    for cu in ([0, 50, 40], [0, 40, T + 1], [1, 40, 70]):
        try:
            fn(torch.tensor(cu, dtype=torch.int32, device="cuda"))
            print("%%s %%s: accepted" %% (name, cu))
        except K.KdaError as e:
            print("%%s %%s: %%d" %% (name, cu, e.status))
'''


def test_validate_rejects_bad_cu_seqlens():
    # in a child: KDA_VALIDATE is read at the first call.  Rejected on the host: no kernel sees them.
    res = subprocess.run([sys.executable, "-c", CHILD % {"root": ROOT}], env=dict(os.environ, KDA_VALIDATE="1"),
                         capture_output=True, text=True, timeout=300)
    print(res.stdout, res.stderr[-2000:], flush=True)
    lines = [line for line in res.stdout.splitlines() if ": " in line]
    assert res.returncode == 0 and len(lines) == 12 and all(line.endswith(": 1") for line in lines)


def test_offsets_beyond_32_bits():
    # more than 2^31 elements before the last sequence's rows: they come out as in a call of their own
    L, D = 300, 2056
    T = (1 << 20) + L
    assert (T - L) * D > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = torch.empty(T, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    small = x[-L:].clone()
    cu = torch.tensor([0, T - L, T], dtype=torch.int32, device="cuda")
    own = torch.tensor([0, L], dtype=torch.int32, device="cuda")
    out, ref = torch.empty_like(x), torch.empty_like(small)
    g = torch.full((T, D), -0.05, device="cuda")
    chk = torch.empty(-(-T // 128), D, device="cuda")
    K.kda_scan_prefill(x, g, None, cu, out, None, checkpoints=chk)
    K.kda_scan_prefill(small, g[-L:].contiguous(), None, own, ref, None)
    # the tiles fall elsewhere in the sequence: fp32 rounding, then a rounding to bf16
    near = lambda a, b, rel: float((a.float() - b.float()).abs().max()) <= rel * float(b.float().abs().max())   # noqa: E731
    assert near(out[-L:], ref, 2.0 ** -8)
    gb = K.kda_scan_backward(x, g, None, cu, x, checkpoints=chk, want_dinit=False)
    gs = K.kda_scan_backward(small, g[-L:].contiguous(), None, own, small, want_dinit=False)
    assert near(gb["dx"][-L:], gs["dx"], 2.0 ** -8) and near(gb["dg"][-L:], gs["dg"], 1000 * 2.0 ** -24)
    del g, gb, chk
    w, b = torch.randn(D, 4, device="cuda"), torch.randn(D, device="cuda")
    K.kda_conv_prefill(x, w, b, None, cu, out, None)
    K.kda_conv_prefill(small, w, b, None, own, ref, None)
    assert torch.equal(out[-L:], ref)
    gc = K.kda_conv_backward(x, w, b, None, cu, x, want_dinit=False)
    assert torch.equal(gc["dx"][-L:], K.kda_conv_backward(small, w, b, None, own, small, want_dinit=False)["dx"])
    del gc
    mx = torch.empty(T, D, dtype=torch.uint8, device="cuda")
    sc = torch.empty(T, -(-D // 32), dtype=torch.uint8, device="cuda")
    mx2, sc2 = torch.empty(L, D, dtype=torch.uint8, device="cuda"), torch.empty(L, -(-D // 32), dtype=torch.uint8, device="cuda")
    K.kda_rmsnorm(x, b, out, residual=x, out_mx=mx, scales=sc)
    K.kda_rmsnorm(small, b, ref, residual=small, out_mx=mx2, scales=sc2)
    assert near(out[-L:], ref, 2.0 ** -8)
    back = lambda m, s: m.view(torch.float8_e4m3fn).float() * torch.exp2(s.float() - 127).repeat_interleave(32, 1)[:, :D]   # noqa: E731
    assert near(back(mx[-L:], sc[-L:]), back(mx2, sc2), 2.0 ** -3)
    K.kda_rmsnorm_backward(x, b, x, grads=dict(dx=out, dweight=torch.empty(D, device="cuda")))
    K.kda_rmsnorm_backward(small, b, small, grads=dict(dx=ref, dweight=torch.empty(D, device="cuda")))
    assert near(out[-L:], ref, 2.0 ** -8)


@pytest.mark.parametrize("D", [40, 257])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=str)
def test_arrays_side_by_side(D, dt):
    # all arrays of a call cut from one buffer without gaps: taken, and the same bits as from arrays of their own
    T, N, W, f32 = 300, 3, 4, torch.float32
    gen = torch.Generator(device="cuda").manual_seed(D)
    pool, at = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda"), [0]
    cu = torch.tensor([0, 100, 130, T], dtype=torch.int32, device="cuda")

    def cut(shape, dtype, like=None):
        e = torch.empty(0, dtype=dtype).element_size()
        start = (at[0] + e - 1) // e * e
        n = int(np.prod(shape))
        at[0] = start + n * e
        t = pool[start:at[0]].view(dtype).view(shape)
        if like is not None:
            t.copy_(like)
        return t

    r = lambda *s, dtype=f32: torch.randn(*s, device="cuda", generator=gen).to(dtype)   # noqa: E731
    x, dout, res, dres = (r(T, D, dtype=dt) for _ in range(4))
    g, st, w, b, nw = -r(T, D).abs(), r(N, D), r(D, W), r(D), r(D)
    cst = r(N, W - 1, D, dtype=dt)

    def ws(size):   # (the scan's are 8-byte aligned)
        return (-(-size // 8),), torch.int64

    calls = [   # call(inputs, outputs), inputs, the outputs' shapes and types
        (lambda i, o: K.kda_scan_prefill(i[0], i[1], i[2], i[3], o[0], o[1], checkpoints=o[2], workspace=o[3]),
         [x, g, st, cu], [((T, D), dt), ((N, D), f32), ((3, D), f32), ws(K.kda_scan_workspace_size(N, T, D, dt))]),
        (lambda i, o: K.kda_scan_backward(i[0], i[1], i[2], i[3], i[4], i[5], workspace=o[3],
                                          grads=dict(dx=o[0], dg=o[1], dinit=o[2])),
         [x, g, st, cu, dout, st], [((T, D), dt), ((T, D), f32), ((N, D), f32),
                                    ws(K.kda_scan_backward_workspace_size(N, T, D, dt))]),
        (lambda i, o: K.kda_conv_prefill(i[0], i[1], i[2], i[3], i[4], o[0], o[1]),
         [x, w, b, cst, cu], [((T, D), dt), ((N, W - 1, D), dt)]),
        (lambda i, o: K.kda_conv_backward(i[0], i[1], i[2], i[3], i[4], i[5], i[6], workspace=o[4],
                                          grads=dict(dx=o[0], dweight=o[1], dbias=o[2], dinit=o[3])),
         [x, w, b, cst, cu, dout, cst], [((T, D), dt), ((D, W), f32), ((D,), f32), ((N, W - 1, D), dt),
                                         ws(K.kda_conv_backward_workspace_size(N, T, D, W, dt))]),
        (lambda i, o: K.kda_rmsnorm(i[0], i[1], o[0], residual=i[2], residual_out=o[1], out_mx=o[2], scales=o[3]),
         [x, nw, res], [((T, D), dt), ((T, D), dt), ((T, D), torch.uint8), ((T, -(-D // 32)), torch.uint8)]),
        (lambda i, o: K.kda_rmsnorm_backward(i[0], i[1], i[2], i[3], workspace=o[2], grads=dict(dx=o[0], dweight=o[1])),
         [x, nw, dout, dres], [((T, D), dt), ((D,), f32), ws(K.kda_rmsnorm_backward_workspace_size(T, D, dt))]),
    ]
    for fn, ins, outs in calls:
        own = [torch.zeros(s, dtype=t, device="cuda") for s, t in outs]
        fn(ins, own)
        at[0] = 0
        side_in = [cut(t.shape, t.dtype, t) for t in ins]
        side = [cut(s, t) for s, t in outs]
        fn(side_in, side)
        assert all(torch.equal(a, c) for a, c in zip(own, side) if a.dtype is not torch.int64)
        assert all(torch.equal(a, c) for a, c in zip(ins, side_in))


def test_overlaps_raise():
    x, g = torch.randn(64, 64, device="cuda"), -torch.rand(64, 64, device="cuda")
    cu, before = torch.tensor([0, 64], dtype=torch.int32, device="cuda"), x.clone()
    x3, g3, o3 = torch.cat((x, x, x)), torch.cat((g, g, g)), torch.empty(192, 64, device="cuda")
    bad = [lambda: K.kda_rmsnorm(x, None, out_mx=x.view(torch.uint8)[:16].view(64, 64),
                                 scales=torch.empty(64, 2, dtype=torch.uint8, device="cuda")),
           lambda: K.kda_scan_prefill(x, g, None, cu, g, None),
           lambda: K.kda_scan_prefill(x, g, None, cu, torch.empty_like(x), x[:1]),
           lambda: K.kda_scan_decode_step(x, g, x, torch.empty_like(x)),
           lambda: K.kda_scan_backward(x, g, None, cu, x, grads=dict(dx=torch.empty_like(x), dg=x)),
           lambda: K.kda_scan_prefill(x3, g3, None, cu, o3, None, workspace=o3)]
    for fn in bad:
        with pytest.raises(K.KdaError) as e:
            fn()
        assert e.value.status == K.KDA_ERR_INVALID_ARG
    assert torch.equal(x, before)


def test_new_tensors_belong_to_the_call_s_stream():
    """Gradients that a call allocates lie in the memory of the stream it runs on, however that is given: as a stream,
    as its number (0: the null stream), or not at all."""
    x, g = torch.randn(600, 512, device="cuda"), -torch.rand(600, 512, device="cuda")
    w, cu = torch.randn(512, 4, device="cuda"), torch.tensor([0, 600], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def owner(t):
        p = t.data_ptr()
        return [s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= p < s["address"] + s["total_size"]][0]

    class Other:   # another library's stream object
        cuda_stream = side.cuda_stream

    want = K.kda_scan_backward(x, g, None, cu, x)
    for stream, raw in ((None, 0), (0, 0), (torch.cuda.default_stream(), 0), (side, side.cuda_stream),
                        (side.cuda_stream, side.cuda_stream), (Other(), side.cuda_stream)):
        for call in (lambda: K.kda_scan_backward(x, g, None, cu, x, stream=stream),
                     lambda: K.kda_conv_backward(x, w, None, None, cu, x, stream=stream),
                     lambda: K.kda_rmsnorm_backward(x, w[:, 0].contiguous(), x, stream=stream)):
            torch.cuda.synchronize()
            got = call()
            torch.cuda.synchronize()
            assert all(owner(t) == raw for t in got.values() if t is not None), stream
            if "dg" in got:
                assert all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.parametrize("D", [64, 130])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=str)
def test_any_alignment_gives_the_same_bits(D, dt):
    # every token array and state one element off a 16-byte boundary, against the same values on one
    T, N, W = 190, 2, 4
    gen = torch.Generator(device="cuda").manual_seed(D)
    r = lambda *s, dtype=torch.float32: torch.randn(*s, device="cuda", generator=gen).to(dtype)   # noqa: E731

    def off(t):
        base = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        v = base[1:].view(t.shape)
        assert v.data_ptr() % 16
        return v.copy_(t)

    cu = torch.tensor([0, 150, T], dtype=torch.int32, device="cuda")
    x, dout, res, g = r(T, D, dtype=dt), r(T, D, dtype=dt), r(T, D, dtype=dt), -r(T, D).abs()
    st, cst, w, b = r(N, D), r(N, W - 1, D, dtype=dt), r(D, W), r(D)
    e = torch.zeros_like
    u8 = torch.zeros(T, D, dtype=torch.uint8, device="cuda")

    def all_calls(v):   # v: how a tensor is laid out
        out, fin, o2, cf, o3, total, m8 = v(e(x)), v(e(st)), v(e(x)), v(e(cst)), v(e(x)), v(e(x)), v(u8)
        sc = torch.zeros(T, -(-D // 32), dtype=torch.uint8, device="cuda")
        K.kda_scan_prefill(v(x), v(g), v(st), cu, out, fin)
        gs = K.kda_scan_backward(v(x), v(g), v(st), cu, v(dout), v(st),
                                 grads=dict(dx=v(e(x)), dg=v(e(g)), dinit=v(e(st))))
        K.kda_conv_prefill(v(x), v(w), v(b), v(cst), cu, o2, cf)
        gc = K.kda_conv_backward(v(x), v(w), v(b), v(cst), cu, v(dout), v(cst),
                                 grads=dict(dx=v(e(x)), dweight=v(e(w)), dbias=v(e(b)), dinit=v(e(cst))))
        K.kda_rmsnorm(v(x), v(b), o3, residual=v(res), residual_out=total, out_mx=m8, scales=sc)
        gn = K.kda_rmsnorm_backward(v(x), v(b), v(dout), v(res), grads=dict(dx=v(e(x)), dweight=v(e(b))))
        s1, s2, d1, d2 = v(st), v(cst), v(x[:N].clone()), v(x[:N].clone())
        K.kda_scan_decode_step(d1, v(g[:N]), s1, d1)
        K.kda_conv_decode_step(d2, v(w), v(b), s2, d2)
        return [out, fin, *gs.values(), o2, cf, *gc.values(), o3, total, m8, sc, *gn.values(), s1, s2, d1, d2]

    for a, c in zip(all_calls(lambda t: t.clone()), all_calls(off)):
        assert torch.equal(a, c)


def test_token_calls_and_new_tensors_in_a_graph():
    # a decoding step captured (states move with every replay), and training calls that make their own tensors there
    N, D, W = 5, 200, 4
    gen = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen)   # noqa: E731
    x, res, g, nw, cw, cb = r(N, D), r(N, D), -r(N, D).abs(), r(D), r(D, W), r(D)
    y, total, u, h = (torch.empty(N, D, device="cuda") for _ in range(4))
    conv0, state0 = r(N, W - 1, D), r(N, D)
    conv, state = conv0.clone(), state0.clone()
    T = 700
    cu = torch.tensor([0, 300, 300, T], dtype=torch.int32, device="cuda")
    px, pg, dout, pout = r(T, D), -r(T, D).abs(), r(T, D), torch.empty(T, D, device="cuda")

    def step():
        K.kda_rmsnorm(x, nw, y, residual=res, residual_out=total)
        K.kda_conv_decode_step(y, cw, cb, conv, u)
        K.kda_scan_decode_step(u, g, state, h)
        K.kda_scan_prefill(px, pg, None, cu, pout, None)
        return [K.kda_scan_backward(px, pg, None, cu, dout), K.kda_conv_backward(px, cw, cb, None, cu, dout),
                K.kda_rmsnorm_backward(px, nw, dout)]

    results = lambda grads: [t.clone() for t in (y, total, u, h, conv, state, pout,   # noqa: E731
                                                 *(v for d in grads for v in d.values() if v is not None))]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = step()
    conv.copy_(conv0), state.copy_(state0)
    replayed, eager, px0 = [], [], px.clone()
    for i in range(4):
        x.copy_(res * (i + 1))
        px.copy_(px0 * (2 - i))
        graph.replay()
        torch.cuda.synchronize()
        replayed.append(results(made))
    conv.copy_(conv0), state.copy_(state0)
    for i in range(4):
        x.copy_(res * (i + 1))
        px.copy_(px0 * (2 - i))
        eager.append(results(step()))
    assert all(torch.equal(p, q) for a, b in zip(replayed, eager) for p, q in zip(a, b))
