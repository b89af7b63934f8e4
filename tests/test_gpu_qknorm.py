"""kda_qknorm and kda_qknorm_backward against the norm and rotation in fp64
(tests/cache_ref.py)."""
import numpy as np
import pytest
import torch

import cache_ref as C
from layer_ref import HALF_STEP, close
from gated_delta_rule_40_amd import libkda as K

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    K.load()


def host(t):
    return t.detach().double().cpu().numpy()


def make(T, Hq, Hk, d, rot=0, axes=1, dtype="bf16", grad=None, seed=0, far=0, fused=False, shuffled=False):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)                       # noqa: E731
    size = torch.exp(2 * rnd(T, 1, 1))                                    # heads of very different sizes
    dt, gt = DT[dtype], DT[grad or dtype]
    if fused:                                                             # columns of one array, with others behind
        rows = torch.cat(((rnd(T, Hq, d) * size).flatten(1), (rnd(T, Hk, d) * size).flatten(1), rnd(T, 5)), 1).to(dt).cuda()
        q, k = rows[:, :Hq * d].unflatten(1, (Hq, d)), rows[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d))
    else:
        q, k = (rnd(T, Hq, d) * size).to(dt).cuda(), (rnd(T, Hk, d) * size).to(dt).cuda()
    p = dict(q=q, k=k, qw=(1 + 0.2 * rnd(d)).cuda(), kw=(1 + 0.2 * rnd(d)).cuda(), dq=rnd(T, Hq, d).to(gt).cuda(),
             dk=rnd(T, Hk, d).to(gt).cuda(), turn={}, angle=None, rot=rot)
    if rot:
        freq = (0.5 ** torch.arange(rot // 2).div(max(1, rot // 16))).float()
        pos = torch.randint(-5, 200, (axes, T), generator=gen, dtype=torch.int32) + far
        axis = torch.randint(-1, axes + 1, (rot // 2,), generator=gen, dtype=torch.int32) if shuffled else None
        p["turn"] = dict(positions=pos.cuda() if axes > 1 or shuffled else pos[0].cuda(), inv_freq=freq.cuda(),
                         pair_axis=None if axis is None else axis.cuda())
        p["angle"] = C.angles(pos.numpy(), freq.double().numpy(), None if axis is None else axis.numpy())
    return p


def check(p, norm="l2", weight=True, interleaved=False, scale=0.25, eps=EPS, what=""):
    dt = p["q"].dtype
    name = {v: k for k, v in DT.items()}[dt]
    qw, kw = (p["qw"], p["kw"]) if weight else (None, None)
    form = dict(q_weight=qw, k_weight=kw, norm=norm, eps=eps, q_scale=scale, interleaved=interleaved, **p["turn"])
    qo, ko = (torch.empty(p[n].shape, dtype=dt, device="cuda") for n in "qk")
    K.kda_qknorm(p["q"], p["k"], qo, ko, **form)
    g = K.kda_qknorm_backward(p["q"], p["k"], p["dq"], p["dk"], **form)
    scale = float(np.float32(scale))
    for n, out, w, s in (("q", qo, qw, scale), ("k", ko, kw, 1.0)):
        w = None if w is None else host(w)
        y, e = C.qknorm(host(p[n]), w, norm, float(np.float32(eps)), s, p["angle"], p["rot"], interleaved)
        close(host(out), y, e, name, what + n)
        dx, ex, dw, ew = C.qknorm_backward(host(p[n]), w, norm, float(np.float32(eps)), s, p["angle"], p["rot"], interleaved,
                                           host(p["d" + n]))
        close(host(g["d" + n]), dx, ex, name, what + "d" + n)
        if w is not None:
            close(host(g["d%s_weight" % n]), dw, ew, "fp32", what + "d%s_weight" % n)
        else:
            assert g["d%s_weight" % n] is None
    return qo, ko, g


# every width of a piece, one lane to 64 a head, odd parts, one token
DIMS = [(1, 0), (2, 2), (3, 2), (5, 0), (8, 8), (16, 16), (17, 4), (36, 12), (64, 0), (64, 32), (72, 24), (80, 40), (96, 96),
        (100, 50), (127, 64), (128, 0), (128, 128), (129, 2), (192, 64), (255, 254), (256, 256), (500, 120), (511, 0),
        (512, 512)]


@pytest.mark.parametrize("d,rot", DIMS, ids=str)
@pytest.mark.parametrize("dtype,interleaved", [("bf16", False), ("fp32", True), ("bf16", True), ("fp32", False)])
def test_head_sizes(d, rot, dtype, interleaved):
    check(make(7, 3, 2, d, rot, dtype=dtype), interleaved=interleaved)


@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (1, 32, 8), (2, 1, 0), (3, 0, 1), (5, 7, 3), (40, 64, 1), (1000, 1, 1),
                                     (2500, 3, 3), (700, 16, 16)], ids=str)
@pytest.mark.parametrize("norm", ["l2", "rms", "none"])
def test_tokens_and_heads(T, Hq, Hk, norm):
    check(make(T, Hq, Hk, 64, 64, axes=3, grad="fp32", shuffled=True), norm=norm)


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("grad", ["bf16", "fp32"])
def test_without_weights_and_of_one_projection(fused, grad):
    check(make(130, 4, 4, 128, 0, grad=grad, fused=fused), weight=False, scale=128 ** -0.5)
    check(make(131, 4, 2, 128, 64, grad=grad, fused=fused), norm="rms")


@pytest.mark.parametrize("far", [2 ** 20, 2 ** 31 - 300, -2 ** 31 + 10])
def test_far_positions_keep_their_angles(far):
    check(make(50, 2, 2, 64, 64, dtype="fp32", far=far))


def test_gradients_into_the_projections_columns():
    p = make(90, 4, 2, 64, 16, fused=True, grad="fp32")
    _, _, want = check(p)
    form = dict(q_weight=p["qw"], k_weight=p["kw"], eps=EPS, q_scale=0.25, **p["turn"])
    rows = torch.full((90, 6 * 64 + 5), 7.0, dtype=torch.bfloat16, device="cuda")
    grads = dict(dq=rows[:, :256].unflatten(1, (4, 64)), dk=rows[:, 256:384].unflatten(1, (2, 64)),
                 dq_weight=torch.empty(64, device="cuda"), dk_weight=torch.empty(64, device="cuda"))
    got = K.kda_qknorm_backward(p["q"], p["k"], p["dq"], p["dk"], grads=grads, **form)
    for n in want:
        assert torch.equal(got[n], want[n]), n
    assert torch.all(rows[:, 384:] == 7.0)                       # what lies between the rows stays
    # in the place of q and k themselves
    K.kda_qknorm_backward(p["q"], p["k"], p["dq"], p["dk"], grads=dict(grads, dq=p["q"], dk=p["k"]), **form)
    assert torch.equal(p["q"], want["dq"]) and torch.equal(p["k"], want["dk"])


def test_in_place():
    p = make(33, 3, 5, 96, 32)
    qo, ko, _ = check(p)
    K.kda_qknorm(p["q"], p["k"], p["q"], p["k"], q_weight=p["qw"], k_weight=p["kw"], eps=EPS, q_scale=0.25, **p["turn"])
    assert torch.equal(p["q"], qo) and torch.equal(p["k"], ko)


def test_queries_alone_and_nothing_at_all():
    p = make(20, 3, 1, 64)
    want, _, g = check(p, weight=False)
    out = torch.empty_like(p["q"])
    K.kda_qknorm(p["q"], None, out, None, eps=EPS, q_scale=0.25)
    got = K.kda_qknorm_backward(p["q"], None, p["dq"], None, eps=EPS, q_scale=0.25)
    assert torch.equal(out, want) and torch.equal(got["dq"], g["dq"]) and got["dk"] is None
    z = torch.empty(0, 3, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    K.kda_qknorm(z, z, z.clone(), z.clone(), q_weight=w)
    g = K.kda_qknorm_backward(z, z, z, z, q_weight=w, k_weight=w)
    assert not g["dq_weight"].any() and not g["dk_weight"].any()          # written: zeros


def test_off_16_byte_boundaries_the_bits_are_the_same():
    p = make(60, 4, 4, 128, 128, grad="fp32")
    form = dict(q_weight=p["qw"], k_weight=p["kw"], eps=EPS, **p["turn"])
    want_q, want_k, want = check(p, scale=1.0)

    def off(t):
        u = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        return u.copy_(t)
    q, k, dq, dk = (off(p[n]) for n in ("q", "k", "dq", "dk"))
    qo, ko = off(want_q * 0), off(want_k * 0)
    form["q_weight"], form["k_weight"] = off(p["qw"]), off(p["kw"])
    K.kda_qknorm(q, k, qo, ko, **form)
    g = K.kda_qknorm_backward(q, k, dq, dk, **form)
    assert torch.equal(qo, want_q) and torch.equal(ko, want_k) and all(torch.equal(g[n], want[n]) for n in want)


def test_heads_of_zeros_infinities_and_nan_stay_their_own():
    p = make(6, 4, 4, 128, 64, dtype="fp32")
    clean = p["q"].clone()
    out, ref, ko = torch.empty_like(clean), torch.empty_like(clean), torch.empty_like(p["k"])
    K.kda_qknorm(clean, p["k"], ref, ko, **p["turn"])
    p["q"][0, 1], p["q"][2, 3, 5], p["q"][3, 0, 7] = 0.0, float("inf"), float("nan")
    K.kda_qknorm(p["q"], p["k"], out, ko, **p["turn"])
    assert torch.all(out[0, 1] == 0) and torch.isnan(out[2, 3, 5:]).any() and torch.all(torch.isnan(out[3, 0]))
    touched = torch.zeros(6, 4, dtype=torch.bool)
    touched[0, 1] = touched[2, 3] = touched[3, 0] = True
    assert torch.equal(out[~touched], ref[~touched])
    K.kda_qknorm(p["q"], p["k"], out, ko, eps=0.0, **p["turn"])
    assert torch.all(torch.isnan(out[0, 1]))                              # 0 / 0
    g = K.kda_qknorm_backward(p["q"], p["k"], p["dq"], p["dk"], **p["turn"])["dq"]
    assert torch.all(torch.isfinite(g[~touched])) and torch.all(torch.isfinite(g[0, 1]))


def test_without_a_norm_an_infinite_value_has_no_part_in_its_gradient():
    p = make(5, 3, 2, 77, 20)
    for x in (p["q"], p["k"]):
        x[1, 0, 3], x[2, 1, 76], x[4, 1, 0] = float("inf"), float("nan"), float("-inf")
    form = dict(norm="none", q_scale=0.5, **p["turn"])
    g = K.kda_qknorm_backward(p["q"], p["k"], p["dq"], p["dk"], **form)
    clean = [torch.nan_to_num(x, 0., 0., 0.) for x in (p["q"], p["k"])]
    want = K.kda_qknorm_backward(*clean, p["dq"], p["dk"], **form)
    for name in ("dq", "dk"):
        assert bool(torch.isfinite(g[name]).all()) and torch.equal(g[name], want[name])


def test_offsets_beyond_32_bits():
    """Tokens whose rows begin beyond 2^31 elements, in an array of which few rows are touched."""
    T, stride = 40, 1 << 26
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 6 GB")
    rows = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda").view(T, stride)
    p = make(T, 2, 2, 128, 128)
    q, k = rows[:, -512:-256].unflatten(1, (2, 128)), rows[:, -256:].unflatten(1, (2, 128))
    q.copy_(p["q"])
    k.copy_(p["k"])
    want_q, want_k, want = check(p, weight=False)
    qo, ko = torch.empty_like(want_q), torch.empty_like(want_k)
    form = dict(eps=EPS, q_scale=0.25, **p["turn"])
    K.kda_qknorm(q, k, qo, ko, **form)
    assert torch.equal(qo, want_q) and torch.equal(ko, want_k)
    K.kda_qknorm_backward(q, k, p["dq"], p["dk"], grads=dict(dq=q, dk=k), **form)
    assert torch.equal(q, want["dq"]) and torch.equal(k, want["dk"])


def test_against_autograd():
    """The gradients are those of the formula, by torch in fp64."""
    p = make(30, 3, 2, 40, 24, axes=2, shuffled=True, dtype="fp32")
    g = K.kda_qknorm_backward(p["q"], p["k"], p["dq"], p["dk"], q_weight=p["qw"], k_weight=p["kw"], norm="rms", eps=EPS,
                              q_scale=0.25, **p["turn"])
    angle = torch.tensor(p["angle"])[:, None]
    for n, s in (("q", 0.25), ("k", 1.0)):
        x = p[n].double().cpu().requires_grad_()
        w = p[n + "w"].double().cpu().requires_grad_()
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + float(np.float32(EPS))) * s * w
        a, b = y[..., :12], y[..., 12:24]
        y = torch.cat((a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin(), y[..., 24:]), -1)
        (y * p["d" + n].double().cpu()).sum().backward()
        _, ex, _, ew = C.qknorm_backward(x.detach().numpy(), w.detach().numpy(), "rms", EPS, s, p["angle"], 24, False,
                                         host(p["d" + n]))
        close(host(g["d" + n]), x.grad.numpy(), ex, "fp32", "d" + n)
        close(host(g["d%s_weight" % n]), w.grad.numpy(), ew, "fp32", "d%s_weight" % n)


def test_binding_refusals():
    p = make(8, 2, 2, 64, 32)
    q, k, o = p["q"], p["k"], torch.empty_like(p["q"])
    o2 = torch.empty_like(o)
    ok = dict(**p["turn"])
    pos, freq = p["turn"]["positions"], p["turn"]["inv_freq"]
    for kw, args in ((dict(norm="l1"), ()), (dict(inv_freq=freq), ()), (dict(positions=pos), ()),
                     (dict(positions=pos.long(), inv_freq=freq), ()), (dict(positions=pos[:5], inv_freq=freq), ()),
                     (dict(positions=pos, inv_freq=torch.ones(33, device="cuda")), ()),
                     (dict(pair_axis=pos), ()), (dict(q_weight=torch.ones(32, device="cuda"), **ok), ()),
                     ({}, (q.transpose(0, 1), k, o, o2)), ({}, (q, k[:4], o, o2)), ({}, (q, k, o[:4], o2)),
                     ({}, (q, k.float(), o, o2)), ({}, (q[:1].expand(8, 2, 64), k, o, o2)), ({}, (q, k, o.cpu(), o2)),
                     ({}, (q, k, torch.empty(8, 2, 128, dtype=q.dtype, device="cuda")[..., :64], o2))):
        with pytest.raises(ValueError):
            K.kda_qknorm(*(args or (q, k, o, o2)), **kw)
    with pytest.raises(K.KdaError) as e:
        K.kda_qknorm(q, k, o, o)
    assert e.value.status == K.KDA_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        K.kda_qknorm_backward(q, k, o.half(), o2)
    with pytest.raises(ValueError):
        K.kda_qknorm_backward(q, k, o, o2, grads=dict(dq=o))
    assert HALF_STEP["bf16"] == 2.0 ** -8
