"""kda_rmsnorm and kda_rmsnorm_backward against the norm in fp64
(tests/layer_ref.py), and the 8-bit output against the rule of its scale and
rounding."""
import numpy as np
import pytest
import torch

import layer_ref as R
from gated_delta_rule_40_amd import libkda as K

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    K.load()


def make(rows, D, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    size = torch.exp(2 * rnd(rows, 1))                # rows of very different sizes
    d = dict(x=(rnd(rows, D) * size).to(DT[dtype]), res=(rnd(rows, D) * size).to(DT[dtype]), w=1 + 0.2 * rnd(D),
             dout=rnd(rows, D).to(DT[dtype]), dres=rnd(rows, D).to(DT[dtype]))
    return {k: v.double().numpy() for k, v in d.items()}, {k: v.cuda() for k, v in d.items()}


def host(t):
    return t.detach().double().cpu().numpy()


def check_mx(q, scales, f, what):
    """Scales by their rule; every value within half an e4m3 step of the scaled y, and y within its own bound."""
    q = host(q.view(torch.float8_e4m3fn).float())
    y, e = f["y"], 1.01 * f["e_y"]
    rows, D = y.shape
    nb = -(-D // 32)
    assert scales.shape == (rows, nb)
    pad = lambda a: np.pad(a, ((0, 0), (0, nb * 32 - D))).reshape(rows, nb, 32)   # noqa: E731
    top, slack = np.abs(pad(y)).max(2), pad(e).max(2)
    # e8m0 begins at 2^-127 (byte 0)
    rule = lambda t: np.where(t > 0, np.maximum(np.ceil(np.log2(np.where(t > 0, t, 1) / 448)) + 127, 0), 127)   # noqa: E731
    sc = scales.cpu().numpy().astype(np.int64)
    assert np.all((sc == rule(top)) | (sc == rule(top - slack)) | (sc == rule(top + slack))), what
    s = np.repeat(2.0 ** (sc - 127.0), 32, 1)[:, :D]
    half = np.maximum(2.0 ** -4 * np.abs(y) / s, 2.0 ** -10)     # half a step; subnormal steps are 2^-9
    assert np.all(np.isfinite(q)) and np.all(np.abs(q) <= 448)
    assert np.all(np.abs(q - y / s) <= half * 1.0001 + 1.0625 * e / s), what


SHAPES = [(1, 1), (3, 7), (5, 31), (2, 32), (300, 33), (7, 64), (9, 100), (1000, 128), (4, 130), (3, 512), (2, 1000),
          (5, 2048), (3, 4100), (2, 7168), (3, 8191), (2, 16384)]


@pytest.mark.parametrize("rows,D", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("res,weight", [(True, True), (False, True), (True, False)])
def test_forward(rows, D, dtype, res, weight):
    h, d = make(rows, D, dtype)
    dres, w = d["res"] if res else None, d["w"] if weight else None
    f = R.rmsnorm(h["x"], h["res"] if res else None, h["w"] if weight else None, EPS)
    out, total = torch.empty_like(d["x"]), torch.empty_like(d["x"]) if res else None
    mx = torch.empty(rows, D, dtype=torch.uint8, device="cuda")
    sc = torch.empty(rows, -(-D // 32), dtype=torch.uint8, device="cuda")
    K.kda_rmsnorm(d["x"], w, out, residual=dres, residual_out=total, out_mx=mx, scales=sc, eps=EPS)
    R.close(host(out), f["y"], f["e_y"], dtype, "out")
    check_mx(mx, sc, f, "mx")
    if res:
        R.close(host(total), f["r"], f["e_r"], dtype, "sum")
    # each output by itself, and in place
    o2 = d["x"].clone()
    K.kda_rmsnorm(o2, w, o2, residual=dres, eps=EPS)
    assert torch.equal(o2, out)
    m2, s2 = torch.empty_like(mx), torch.empty_like(sc)
    stream = d["res"].clone() if res else None
    K.kda_rmsnorm(d["x"], w, residual=stream, residual_out=stream, out_mx=m2, scales=s2, eps=EPS)
    assert torch.equal(m2, mx) and torch.equal(s2, sc) and (not res or torch.equal(stream, total))


@pytest.mark.parametrize("rows,D", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("res,weight", [(True, True), (False, True), (True, False)])
def test_backward(rows, D, dtype, res, weight):
    h, d = make(rows, D, dtype, seed=1)
    dres, w = d["dres"] if res else None, d["w"] if weight else None
    g = K.kda_rmsnorm_backward(d["x"], w, d["dout"], dresidual=dres, eps=EPS)
    r = R.rmsnorm_backward(h["x"], h["w"] if weight else None, h["dout"], h["dres"] if res else None, EPS)
    R.close(host(g["dx"]), r["dx"], r["e_dx"], dtype, "dx")
    if weight:
        R.close(host(g["dweight"]), r["dweight"], r["e_dweight"], "fp32", "dweight")
    else:
        assert g["dweight"] is None
    # dx in the place of each of its inputs
    for name in ("x", "dout") + (("dres",) if res else ()):
        t = {k: d[k].clone() for k in ("x", "dout", "dres")}
        got = K.kda_rmsnorm_backward(t["x"], w, t["dout"], dresidual=t["dres"] if res else None, eps=EPS,
                                     grads=dict(dx=t[name], dweight=torch.empty_like(d["w"]) if weight else None))
        assert torch.equal(got["dx"], g["dx"])
        if weight:
            assert torch.equal(got["dweight"], g["dweight"])


def test_many_rows():
    # more rows than the weight gradient's partial sums
    for rows, D in ((5000, 96), (70000, 8)):
        h, d = make(rows, D, "bf16", seed=2)
        g = K.kda_rmsnorm_backward(d["x"], d["w"], d["dout"], eps=EPS)
        r = R.rmsnorm_backward(h["x"], h["w"], h["dout"], None, EPS)
        R.close(host(g["dweight"]), r["dweight"], r["e_dweight"], "fp32", "dweight")
        R.close(host(g["dx"]), r["dx"], r["e_dx"], "bf16", "dx")
        out = torch.empty_like(d["x"])
        K.kda_rmsnorm(d["x"], d["w"], out, eps=EPS)
        f = R.rmsnorm(h["x"], None, h["w"], EPS)
        R.close(host(out), f["y"], f["e_y"], "bf16", "out")


@pytest.mark.parametrize("D", [128, 200, 4096])
def test_mx_scale_edges(D):
    # rows whose blocks' largest values lie at, just below and just above a scale's end; tiny, huge and zero blocks
    x = torch.zeros(9, D)
    x[0] = 0.0
    for i, v in enumerate((448.0, np.nextafter(np.float32(448), np.float32(1000)), 447.9, 1.75 * 2.0 ** -20,
                           np.nextafter(np.float32(1.75 * 2.0 ** -20), np.float32(1)), 1e-30, 1e30, 3e-39)):
        x[i + 1, ::5] = float(v) * (-1) ** i
        x[i + 1, 1] = float(v) / 3
    x = x.cuda()
    # a weight and an eps that make y = x, or a known multiple, in fp32: mean(0) + eps with eps = 1 needs x tiny; so y
    # is taken from the fp32 output itself, which the 8-bit output has to follow
    y = torch.empty_like(x)
    mx = torch.empty(9, D, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(9, -(-D // 32), dtype=torch.float8_e8m0fnu, device="cuda")
    for eps in (1e-6, 1.0, 1e30):
        K.kda_rmsnorm(x, None, y, out_mx=mx, scales=sc, eps=eps)
        f = dict(y=host(y), e_y=np.zeros((9, D)))
        check_mx(mx.view(torch.uint8), sc.view(torch.uint8), f, "eps %g" % eps)
        assert bool((sc.view(torch.uint8)[0] == 127).all()) and bool((mx.view(torch.uint8)[0] == 0).all())


@pytest.mark.parametrize("D", [128, 4096])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_mx_rounds_once(D, dtype):
    """Rows of one magnitude c and eps = 0 have y = w or -w, exactly; the weights lie on ties of e4m3, on scales' ends,
    and a step or two of fp32 beside them.  The squares of eight bits and their sums are exact in fp32, so the only
    rounding there has to be is the last one."""
    gen = np.random.default_rng(D)
    c = np.array([1.0, 3.0, 129 / 128, 141 / 128, 182 / 256, 249.0, 193 * 2.0 ** -12, 255 * 2.0 ** 7])
    x = torch.tensor(c[:, None] * gen.choice([-1.0, 1.0], (len(c), D))).to(DT[dtype])
    assert np.array_equal(np.abs(host(x)), np.repeat(c[:, None], D, 1))
    w = 2.0 ** gen.integers(-6, 7, D) * (1 + (2 * gen.integers(0, 8, D) + 1) / 16)
    w[::32] = 448.0
    w = w * np.repeat(2.0 ** gen.integers(-30, 30, D // 32), 32)
    w = (w.astype(np.float32).view(np.int32) + gen.integers(-2, 3, D).astype(np.int32)).view(np.float32)
    mx = torch.empty(len(c), D, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(len(c), D // 32, dtype=torch.uint8, device="cuda")
    K.kda_rmsnorm(x.cuda(), torch.tensor(w).cuda(), out_mx=mx, scales=sc, eps=0.0)
    y = np.sign(host(x)) * w.astype(np.float64)
    m, e = np.frexp(np.abs(y).reshape(len(c), -1, 32).max(2))
    e = e - 9 + (m > 0.875)
    assert np.array_equal(sc.cpu().numpy(), e + 127)
    v = y / np.repeat(2.0 ** e, 32, 1)
    step = 2.0 ** (np.maximum(np.frexp(v)[1] - 1, -6) - 3)
    assert np.array_equal(host(mx.float()), np.rint(v / step) * step)      # ties to even


def test_mx_of_a_block_with_nan_or_infinity():
    x = torch.randn(4, 256, device="cuda")
    w = torch.ones(256, device="cuda")
    w[40], w[100] = float("nan"), float("inf")
    mx = torch.empty(4, 256, dtype=torch.uint8, device="cuda")
    sc = torch.empty(4, 8, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(x)
    K.kda_rmsnorm(x, w, out, out_mx=mx, scales=sc)
    assert bool((sc[:, [1, 3]] == 255).all()) and bool((sc[:, [0, 2, 4, 5, 6, 7]] < 255).all())
    assert bool(torch.isnan(out[:, 40]).all()) and bool(torch.isinf(out[:, 100]).all())


def test_rows_do_not_touch_each_other():
    x, res = torch.randn(6, 320, device="cuda"), torch.randn(6, 320, device="cuda")
    out, bad = torch.empty_like(x), torch.empty_like(x)
    K.kda_rmsnorm(x, None, out, residual=res)
    x[2, 5], x[4, 7] = float("nan"), float("inf")
    K.kda_rmsnorm(x, None, bad, residual=res)
    assert torch.equal(out[[0, 1, 3, 5]], bad[[0, 1, 3, 5]]) and bool(torch.isnan(bad[2]).all())


def test_leading_dimensions_and_unaligned_views():
    h, d = make(12, 128, "bf16", seed=3)
    f = R.rmsnorm(h["x"], None, h["w"], EPS)
    x3 = d["x"].view(3, 4, 128)                      # [T, H, d]: a norm for each head
    out = torch.empty_like(x3)
    K.kda_rmsnorm(x3, d["w"], out, eps=EPS)
    R.close(host(out.view(12, 128)), f["y"], f["e_y"], "bf16", "heads")
    base = torch.empty(12 * 128 + 1, dtype=torch.bfloat16, device="cuda")
    x = base[1:].view(12, 128)
    x.copy_(d["x"])
    mx = torch.empty(12 * 128 + 3, dtype=torch.uint8, device="cuda")[3:].view(12, 128)
    sc = torch.empty(12, 4, dtype=torch.uint8, device="cuda")
    o2 = torch.empty_like(d["x"])
    K.kda_rmsnorm(x, d["w"], o2, out_mx=mx, scales=sc, eps=EPS)
    R.close(host(o2), f["y"], f["e_y"], "bf16", "unaligned")
    check_mx(mx, sc, f, "unaligned")
    g = K.kda_rmsnorm_backward(x, d["w"], d["dout"], eps=EPS)
    r = R.rmsnorm_backward(h["x"], h["w"], h["dout"], None, EPS)
    R.close(host(g["dx"]), r["dx"], r["e_dx"], "bf16", "dx")
    R.close(host(g["dweight"]), r["dweight"], r["e_dweight"], "fp32", "dweight")


def test_same_bits_streams_and_graph_replays():
    h, d = make(3000, 1024, "bf16", seed=4)
    x = d["x"].clone()
    out, total = torch.empty_like(x), torch.empty_like(x)
    mx = torch.empty(3000, 1024, dtype=torch.uint8, device="cuda")
    sc = torch.empty(3000, 32, dtype=torch.uint8, device="cuda")
    ws = torch.empty(K.kda_rmsnorm_backward_workspace_size(3000, 1024), dtype=torch.uint8, device="cuda")
    grads = dict(dx=torch.empty_like(x), dweight=torch.empty(1024, device="cuda"))

    def step(stream=None):
        K.kda_rmsnorm(x, d["w"], out, residual=d["res"], residual_out=total, out_mx=mx, scales=sc, stream=stream)
        K.kda_rmsnorm_backward(total, d["w"], d["dout"], dresidual=d["dres"], grads=grads, workspace=ws, stream=stream)

    results = lambda: [t.clone() for t in (out, total, mx, sc, *grads.values())]   # noqa: E731
    step()
    first = results()
    torch.cuda.synchronize()
    step(torch.cuda.Stream())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, results()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(d["x"] * (i - 1.5))
        graph.replay()
        torch.cuda.synchronize()
        got = results()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, results()))


def test_no_rows():
    x = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    K.kda_rmsnorm(x, w, x)
    g = K.kda_rmsnorm_backward(x, w, x, grads=dict(dx=x, dweight=torch.full_like(w, 7.0)))
    assert bool((g["dweight"] == 0).all())


def test_rejects_mismatched_tensors():
    h, d = make(4, 64, "bf16")
    out = torch.empty_like(d["x"])
    with pytest.raises(ValueError, match="weight must be torch.float32"):
        K.kda_rmsnorm(d["x"], d["w"].bfloat16(), out)
    with pytest.raises(ValueError, match="go together"):
        K.kda_rmsnorm(d["x"], d["w"], out, scales=torch.empty(4, 2, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        K.kda_rmsnorm(d["x"], d["w"], out, residual=d["res"][:2].contiguous())
    with pytest.raises(ValueError, match="float8_e4m3fn"):
        K.kda_rmsnorm(d["x"], d["w"], out_mx=out, scales=torch.empty(4, 2, dtype=torch.uint8, device="cuda"))
    for kw in (dict(), dict(out=out, residual_out=out)):     # no output; a sum without a residual
        with pytest.raises(K.KdaError) as e:
            K.kda_rmsnorm(d["x"], d["w"], **kw)
        assert e.value.status == K.KDA_ERR_INVALID_ARG


def on_borders(x, eps, gen):
    """A weight for the row x that puts y = x / sqrt(mean(x^2) + eps) * weight as near as fp32 weights come: in every
    block 16 values below a scale's end (448 times a power of two) and 16 on either side of a tie of e4m3.  With it, y
    in extended precision."""
    D = len(x)
    wide = x.astype(np.longdouble)
    rms = np.sqrt((wide * wide).sum() / D + np.longdouble(np.float32(eps)))
    ties = 2.0 ** gen.integers(0, 8, D) * (1 + (2 * gen.integers(0, 8, D) + 1) / 16)
    end = np.arange(D) % 32 < 16
    goal = np.where(end, 448.0, ties) * np.repeat(2.0 ** gen.integers(-6, 6, D // 32), 32)
    w = (goal * rms / np.abs(wide)).astype(np.float32)
    w = np.where(end & (np.abs(wide / rms * w) >= goal), np.nextafter(w, np.float32(0)), w)
    return w, wide / rms * w


@pytest.mark.parametrize("D", [128, 512, 4096, 7168])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("size", [1.0, 300.0])
def test_mx_scales_and_values_beside_their_borders(D, dtype, size):
    """fp64 sums of exact squares are off by D 2^-53 at most, the root and the products by 2^-46: what lies further from
    a border than that is rounded as y itself."""
    gen = np.random.default_rng(int(D + size))
    slack = D * 2.0 ** -53 + 2.0 ** -46
    seen = 0
    for _ in range(4):
        x = torch.tensor(gen.standard_normal(D) * size).to(DT[dtype])
        x[x == 0] = 1.0
        w, y = on_borders(host(x), EPS, gen)
        mx = torch.empty(1, D, dtype=torch.float8_e4m3fn, device="cuda")
        sc = torch.empty(1, D // 32, dtype=torch.uint8, device="cuda")
        K.kda_rmsnorm(x.view(1, D).cuda(), torch.tensor(w).cuda(), out_mx=mx, scales=sc, eps=EPS)
        top = np.abs(y).reshape(-1, 32).max(1)
        m, e = np.frexp(top)
        e = e - 9 + (m > 0.875)
        sure = np.abs(m / np.longdouble(0.875) - 1) > slack
        assert np.array_equal(sc.cpu().numpy()[0][sure], (e + 127)[sure])
        v = y / np.repeat(2.0 ** e, 32)
        step = 2.0 ** (np.maximum(np.frexp(v)[1] - 1, -6) - 3)
        frac = np.abs(v / step) % 1
        sure = np.repeat(sure, 32) & (np.abs(frac - 0.5) * step > slack * np.abs(v))
        assert np.array_equal(host(mx.float())[0][sure], (np.rint(v / step) * step).astype(np.float64)[sure])
        seen += int(sure.sum())
    assert seen > 0.99 * 4 * D


def test_squares_beyond_fp32():
    # the sum of the squares passes fp32's largest number, their mean does not
    gen = torch.Generator().manual_seed(8)
    x = (1e18 * torch.randn(3, 4096, generator=gen)).cuda()
    out = torch.empty_like(x)
    K.kda_rmsnorm(x, None, out, eps=EPS)
    f = R.rmsnorm(host(x), None, None, EPS)
    R.close(host(out), f["y"], f["e_y"], "fp32", "out")


@pytest.mark.parametrize("D", [128, 512, 4096])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("same_row", [True, False])
def test_mx_of_values_below_fp32_beside_ties(D, dtype, same_row):
    """y that vanishes in fp32, of either sign, in a wave that also holds a tie of e4m3: in the same row (whose rms is
    exactly 1) or in the rows beside it."""
    gen = np.random.default_rng(D)
    x = gen.choice([-1.0, 1.0], (4, D))
    x[:, ::D // 8] = 2.0                                           # 8 squares of 4 and 24 of nothing: rms 1
    tiny = np.setdiff1d(np.arange(3, D, D // 32), np.arange(0, D, D // 8))[:24]
    x[:, tiny] = 2.0 ** -126 * gen.choice([-1.0, 1.0], (4, len(tiny)))
    x[:, tiny[0]] = -2.0 ** -126
    tie = np.array([5, D // 2 + 6])
    assert not set(tie) & (set(tiny) | set(range(0, D, D // 8)))
    if not same_row:
        x[[0, 2, 3]] *= 1.25                                       # a rms of 1.25 again gives ties: leave those rows none
        x[np.ix_([0, 2, 3], tie)] = 0.75
    w = np.full(D, 1.25)
    w[tiny] = 2.0 ** gen.integers(-30, -20, len(tiny))             # y from 2^-156 to 2^-146
    w[tiny[0]] = 2.0 ** -27                                        # -2^-153: nearer to zero than to fp32's smallest
    w[tie] = 1.0625, 1.9375
    xt = torch.tensor(x).to(DT[dtype])
    assert np.array_equal(host(xt), x)
    mx = torch.empty(4, D, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(4, D // 32, dtype=torch.uint8, device="cuda")
    K.kda_rmsnorm(xt.cuda(), torch.tensor(w, dtype=torch.float32).cuda(), out_mx=mx, scales=sc, eps=0.0)
    y = x / np.sqrt((x * x).sum(1, keepdims=True) / D) * w
    m, e = np.frexp(np.abs(y).reshape(4, -1, 32).max(2))
    e = e - 9 + (m > 0.875)
    assert np.array_equal(sc.cpu().numpy(), e + 127)
    v = y / np.repeat(2.0 ** e, 32, 1)
    step = 2.0 ** (np.maximum(np.frexp(v)[1] - 1, -6) - 3)
    assert np.array_equal(host(mx.float()), np.rint(v / step) * step)


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_mx_of_a_row_alone_and_among_others(D, dtype):
    """Values below 2^-6 of their scale, beside the ties that e4m3 has there: they may be rounded from fp32's y, and a
    row gets the same bytes whatever lies beside it, with ties of its own or without."""
    gen = np.random.default_rng(D)
    rows, x = [], torch.tensor(gen.standard_normal((6, D))).to(DT[dtype])
    x[x == 0] = 1.0
    x[1, D // 2:] = x[0, D // 2:]
    wide = np.abs(host(x))
    rms = np.sqrt((wide * wide).sum(1) / D + np.float64(np.float32(EPS)))
    goal = (2 * gen.integers(0, 8, D) + 1) * 2.0 ** -10              # ties below 2^-6
    goal[::32] = 300.0                                               # the largest of a block: scale 1
    w = (goal * rms[0] / wide[0]).astype(np.float32)
    w[1] = 1.0625 * 8 * rms[1] / wide[1, 1]                          # a tie for row 1, and one for row 5
    w[3] = 1.0625 * 4 * rms[5] / wide[5, 3]
    wd = torch.tensor(w).cuda()

    def call(t):
        mx = torch.empty(len(t), D, dtype=torch.uint8, device="cuda")
        sc = torch.empty(len(t), D // 32, dtype=torch.uint8, device="cuda")
        K.kda_rmsnorm(t.cuda().contiguous(), wd, out_mx=mx, scales=sc, eps=EPS)
        return mx, sc

    rows = [call(x[i:i + 1]) for i in range(6)]
    for order in ([0, 1, 2, 3, 4, 5], [5, 0, 4, 0, 0, 3], [2, 0, 3], [0, 1], [1, 0], [4, 5, 0, 0]):
        mx, sc = call(x[order])
        for i, n in enumerate(order):
            assert torch.equal(mx[i:i + 1], rows[n][0]) and torch.equal(sc[i:i + 1], rows[n][1]), (order, i)
