"""kda_scan_prefill, kda_scan_decode_step and kda_scan_backward against the
recurrence in fp64 (tests/layer_ref.py), over packed batches whose sequences
end inside, at and beyond the kernels' tiles of 128 tokens."""
import numpy as np
import pytest
import torch

import layer_ref as R
from gated_delta_rule_40_amd import libkda as K

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    K.load()


def make(lens, D, dtype, init=True, tail=0, rate=0.3, seed=0):
    """Host arrays (what the device holds, in fp64) and device tensors."""
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens) + tail, len(lens)
    rnd = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    d = dict(x=rnd(T, D).to(DT[dtype]), g=-rate * torch.rand(T, D, generator=gen) * torch.rand(D, generator=gen),
             init=rnd(N, D) if init else None, dout=rnd(T, D).to(DT[dtype]), dfinal=rnd(N, D) if init else None,
             cu=torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32))
    h = {k: None if v is None else v.double().numpy() for k, v in d.items()}
    h["cu"] = d["cu"].tolist()
    return h, {k: None if v is None else v.cuda() for k, v in d.items()}


def host(t):
    return t.detach().double().cpu().numpy()


def owned(lens, T):
    m = np.zeros(T, bool)
    m[:sum(lens)] = True
    return m


CASES = [
    ([1], 1), ([1], 64), ([1, 1, 1], 130), ([127], 8), ([128], 64), ([129], 256), ([5, 0, 3, 0, 0, 120], 33),
    ([0, 0], 16), ([300], 1), ([127, 1, 0, 130, 128], 96), ([0, 1, 3, 0, 255, 257, 64, 0], 520), ([1000, 24, 2049], 260),
    ([64] * 20 + [0] * 3 + [7] * 9, 1000), ([2 ** i for i in range(11)], 65), ([3000, 5000], 12),
    # channel counts at a workgroup's edge, and enough tiles for the widest rows
    ([300, 33], 129), ([200, 90, 0, 1], 257), ([64, 200], 259), ([129, 128], 383), ([5000, 11, 1000], 2562),
    ([6000, 90], 2561), ([9000, 0, 333, 7, 8001], 259), ([4100, 1, 8192], 385),
]


@pytest.mark.parametrize("lens,D", CASES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("init", [True, False])
def test_prefill(lens, D, dtype, init):
    tail = 3 if D % 2 else 0
    h, d = make(lens, D, dtype, init, tail)
    T, N = d["x"].shape[0], len(lens)
    out = torch.full((T, D), 77.0, dtype=DT[dtype], device="cuda")
    fin = torch.full((N, D), 77.0, device="cuda")
    chk = torch.full((-(-T // 128), D), 77.0, device="cuda")
    K.kda_scan_prefill(d["x"], d["g"], d["init"], d["cu"], out, fin, checkpoints=chk)
    f = R.scan(h["x"], h["g"], h["init"], h["cu"])
    own = owned(lens, T)
    R.close(host(out)[own], f["h"][own], f["e_h"][own], dtype, "out")
    R.close(host(fin), f["final"], f["e_final"], "fp32", "final")
    assert np.all(host(out)[~own] == 77.0)
    inside = ~np.isnan(f["chk"])
    R.close(host(chk)[inside], f["chk"][inside], f["e_chk"][inside], "fp32", "checkpoints")
    # without the optional outputs, and with the state updated in place
    again, state = torch.empty_like(out), None if d["init"] is None else d["init"].clone()
    K.kda_scan_prefill(d["x"], d["g"], state, d["cu"], again, state)
    assert torch.equal(again[:sum(lens)], out[:sum(lens)])
    if state is not None:
        assert torch.equal(state, fin)


@pytest.mark.parametrize("lens,D", CASES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("init", [True, False])
@pytest.mark.parametrize("checkpoints", [True, False])
def test_backward(lens, D, dtype, init, checkpoints):
    tail = 3 if D % 2 else 0
    h, d = make(lens, D, dtype, init, tail, seed=1)
    T, N = d["x"].shape[0], len(lens)
    chk = None
    if checkpoints:
        chk = torch.full((-(-T // 128), D), float("nan"), device="cuda")
        K.kda_scan_prefill(d["x"], d["g"], d["init"], d["cu"], torch.empty_like(d["x"]), None, checkpoints=chk)
    grads = dict(dx=torch.full((T, D), 77.0, dtype=DT[dtype], device="cuda"),
                 dg=torch.full((T, D), 77.0, device="cuda"),
                 dinit=torch.full((N, D), 77.0, device="cuda") if init else None)
    K.kda_scan_backward(d["x"], d["g"], d["init"], d["cu"], d["dout"], d["dfinal"], checkpoints=chk, grads=grads)
    b = R.scan_backward(h["x"], h["g"], h["init"], h["cu"], h["dout"], h["dfinal"])
    own = owned(lens, T)
    R.close(host(grads["dx"])[own], b["dx"][own], b["e_dx"][own], dtype, "dx")
    R.close(host(grads["dg"])[own], b["dg"][own], b["e_dg"][own], "fp32", "dg")
    assert np.all(host(grads["dx"])[~own] == 77.0) and np.all(host(grads["dg"])[~own] == 77.0)
    if init:
        R.close(host(grads["dinit"]), b["dinit"], b["e_dinit"], "fp32", "dinit")


@pytest.mark.parametrize("N,most", [(63, 9), (64, 9), (65, 400), (700, 20), (4100, 3), (9000, 2)])
def test_many_sequences(N, most):
    # more entries of cu_seqlens than a wave holds at once, empty sequences among them
    lens = np.random.default_rng(N).integers(0, most, N).tolist() + [0] * 70 + [3]
    h, d = make(lens, 6, "fp32", tail=1, seed=11)
    T = sum(lens)
    out, fin = torch.full_like(d["x"], 77.0), torch.full_like(d["init"], 77.0)
    K.kda_scan_prefill(d["x"], d["g"], d["init"], d["cu"], out, fin)
    b = R.scan_backward(h["x"], h["g"], h["init"], h["cu"], h["dout"], h["dfinal"])
    R.close(host(out)[:T], b["fwd"]["h"][:T], b["fwd"]["e_h"][:T], "fp32", "out")
    R.close(host(fin), b["fwd"]["final"], b["fwd"]["e_final"], "fp32", "final")
    g = K.kda_scan_backward(d["x"], d["g"], d["init"], d["cu"], d["dout"], d["dfinal"])
    R.close(host(g["dx"])[:T], b["dx"][:T], b["e_dx"][:T], "fp32", "dx")
    R.close(host(g["dg"])[:T], b["dg"][:T], b["e_dg"][:T], "fp32", "dg")
    R.close(host(g["dinit"]), b["dinit"], b["e_dinit"], "fp32", "dinit")
    assert float(out[T:].min()) == 77.0


SLOTS = [[40] + [0] * 200, [0] * 130 + [300], [150] + [0] * 90 + [1, 2] + [0] * 70 + [200, 0, 0, 9], [0] * 300]


@pytest.mark.parametrize("lens", SLOTS, ids=lambda v: "%dof%d" % (sum(map(bool, v)), len(v)))
@pytest.mark.parametrize("init", [True, False])
def test_slots_left_empty(lens, init):
    # more sequences begin at one token than a wave holds entries
    h, d = make(lens, 130, "bf16", init, tail=2, seed=13)
    T, N = sum(lens), len(lens)
    out, fin = torch.full_like(d["x"], 77.0), torch.full((N, 130), 77.0, device="cuda")
    K.kda_scan_prefill(d["x"], d["g"], d["init"], d["cu"], out, fin)
    b = R.scan_backward(h["x"], h["g"], h["init"], h["cu"], h["dout"], h["dfinal"])
    R.close(host(out)[:T], b["fwd"]["h"][:T], b["fwd"]["e_h"][:T], "bf16", "out")
    R.close(host(fin), b["fwd"]["final"], b["fwd"]["e_final"], "fp32", "final")
    assert float(out[T:].min()) == 77.0
    g = K.kda_scan_backward(d["x"], d["g"], d["init"], d["cu"], d["dout"], d["dfinal"])
    R.close(host(g["dx"])[:T], b["dx"][:T], b["e_dx"][:T], "bf16", "dx")
    R.close(host(g["dinit"]), b["dinit"], b["e_dinit"], "fp32", "dinit")
    if init:
        K.kda_scan_prefill(d["x"], d["g"], d["init"], d["cu"], out, d["init"])
        assert torch.equal(d["init"], fin)


@pytest.mark.parametrize("N,D", [(1, 1), (1, 64), (3, 5), (8, 2048), (513, 999)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decode(N, D, dtype):
    h, d = make([1] * N, D, dtype, seed=2)
    state, out = d["init"].clone(), torch.empty_like(d["x"])
    K.kda_scan_decode_step(d["x"], d["g"], state, out)
    f = R.scan(h["x"], h["g"], h["init"], h["cu"])
    R.close(host(state), f["final"], f["e_final"], "fp32", "state")
    R.close(host(out), f["h"], f["e_h"], dtype, "out")
    # the same token as a batch of one-token sequences
    o2, f2 = torch.empty_like(out), torch.empty_like(state)
    K.kda_scan_prefill(d["x"], d["g"], d["init"], d["cu"], o2, f2)
    R.close(host(f2), f["final"], f["e_final"], "fp32", "final")


def test_long_sequence_of_few_channels():
    # many tiles one after another; slow gates, so that the state crosses thousands of tokens
    h, d = make([70000, 11, 20000], 5, "fp32", rate=2e-3, seed=3)
    out, fin = torch.empty_like(d["x"]), torch.empty(3, 5, device="cuda")
    K.kda_scan_prefill(d["x"], d["g"], d["init"], d["cu"], out, fin)
    b = R.scan_backward(h["x"], h["g"], h["init"], h["cu"], h["dout"], h["dfinal"])
    R.close(host(out), b["fwd"]["h"], b["fwd"]["e_h"], "fp32", "out")
    R.close(host(fin), b["fwd"]["final"], b["fwd"]["e_final"], "fp32", "final")
    g = K.kda_scan_backward(d["x"], d["g"], d["init"], d["cu"], d["dout"], d["dfinal"])
    R.close(host(g["dx"]), b["dx"], b["e_dx"], "fp32", "dx")
    R.close(host(g["dg"]), b["dg"], b["e_dg"], "fp32", "dg")
    R.close(host(g["dinit"]), b["dinit"], b["e_dinit"], "fp32", "dinit")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gates_at_their_ends(dtype):
    # no decay, a dropped state (g = -infinity), decays that underflow, growth
    h, d = make([200, 150], 64, dtype, seed=4)
    g = d["g"].clone()
    g[::3] = 0.0
    g[5::40] = float("-inf")
    g[7::50] = -120.0
    g[9::60] = 0.5
    hg = host(g)
    out, fin = torch.empty_like(d["x"]), torch.empty(2, 64, device="cuda")
    K.kda_scan_prefill(d["x"], g, d["init"], d["cu"], out, fin)
    b = R.scan_backward(h["x"], hg, h["init"], h["cu"], h["dout"], h["dfinal"])
    R.close(host(out), b["fwd"]["h"], b["fwd"]["e_h"], dtype, "out")
    R.close(host(fin), b["fwd"]["final"], b["fwd"]["e_final"], "fp32", "final")
    grads = K.kda_scan_backward(d["x"], g, d["init"], d["cu"], d["dout"], d["dfinal"])
    R.close(host(grads["dx"]), b["dx"], b["e_dx"], dtype, "dx")
    R.close(host(grads["dg"]), b["dg"], b["e_dg"], "fp32", "dg")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("lens,hit", [([100, 30, 400, 50], 2), ([1000, 2000, 500], 1), ([128, 128, 128], 1)])
def test_nan_and_infinity_stay_in_their_sequence(lens, hit, bad):
    D = 70
    h, d = make(lens, D, "fp32", tail=2, seed=5)
    cu = h["cu"]
    clean = torch.empty_like(d["x"])
    K.kda_scan_prefill(d["x"], d["g"], d["init"], d["cu"], clean, None)
    gclean = K.kda_scan_backward(d["x"], d["g"], d["init"], d["cu"], d["dout"], d["dfinal"])
    x, dout, init = d["x"].clone(), d["dout"].clone(), d["init"].clone()
    x[cu[hit] + 3] = bad
    dout[cu[hit + 1] - 2] = bad
    init[hit] = bad
    x[cu[-1]:] = bad                                 # rows of no sequence
    dout[cu[-1]:] = bad
    out, fin = torch.zeros_like(x), torch.empty(len(lens), D, device="cuda")
    K.kda_scan_prefill(x, d["g"], init, d["cu"], out, fin)
    grads = K.kda_scan_backward(x, d["g"], init, d["cu"], dout, d["dfinal"])
    for n in range(len(lens)):
        s = slice(cu[n], cu[n + 1])
        if n != hit:
            assert torch.equal(out[s], clean[s]) and torch.equal(grads["dx"][s], gclean["dx"][s])
            assert torch.equal(grads["dg"][s], gclean["dg"][s]) and torch.equal(grads["dinit"][n], gclean["dinit"][n])
        else:
            assert not torch.isfinite(out[s]).any() and not torch.isfinite(fin[n]).any()


def test_same_bits_every_time_and_on_a_side_stream():
    h, d = make([5000, 0, 3000, 129, 9000], 200, "bf16", seed=6)
    call = lambda s=None: (K.kda_scan_prefill(d["x"], d["g"], d["init"], d["cu"], out, fin, stream=s),   # noqa: E731
                           K.kda_scan_backward(d["x"], d["g"], d["init"], d["cu"], d["dout"], d["dfinal"], stream=s))[1]
    out, fin = torch.empty_like(d["x"]), torch.empty(5, 200, device="cuda")
    g0 = call()
    o0, f0 = out.clone(), fin.clone()
    side = torch.cuda.Stream()
    for i in range(4):
        torch.cuda.synchronize()
        out.zero_()
        fin.zero_()
        torch.cuda.synchronize()
        g = call(side if i % 2 else None)
        torch.cuda.synchronize()
        assert torch.equal(out, o0) and torch.equal(fin, f0)
        assert all(torch.equal(g[k], g0[k]) for k in g0)


@pytest.mark.parametrize("lens,D", [([5, 0, 300], 33), ([700, 129, 2000], 1024), ([100], 64)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_in_place(lens, D, dtype):
    _, d = make(lens, D, dtype, seed=15)
    x, g, init, cu, dout, dfinal = (d[k] for k in ("x", "g", "init", "cu", "dout", "dfinal"))
    out, fin = torch.empty_like(x), torch.empty_like(init)
    K.kda_scan_prefill(x, g, init, cu, out, fin)
    a, s = x.clone(), init.clone()
    K.kda_scan_prefill(a, g, s, cu, a, s)
    assert torch.equal(a, out) and torch.equal(s, fin)
    want = K.kda_scan_backward(x, g, init, cu, dout, dfinal)
    for over in ("x", "dout"):
        c = {"x": x.clone(), "dout": dout.clone(), "g": g.clone()}
        got = dict(dx=c[over], dg=c["g"], dinit=torch.empty_like(init))
        K.kda_scan_backward(c["x"], c["g"], init, cu, c["dout"], dfinal, grads=got)
        assert all(torch.equal(got[k], want[k]) for k in want)
    n = len(lens)
    o, s1, s2, a = torch.empty_like(x[:n]), init.clone(), init.clone(), x[:n].clone()
    K.kda_scan_decode_step(x[:n], g[:n], s1, o)
    K.kda_scan_decode_step(a, g[:n], s2, a)
    assert torch.equal(a, o) and torch.equal(s1, s2)


def test_two_calls_at_once():
    # two streams, each call with a workspace of its own
    h, d = make([20000, 13000], 256, "bf16", seed=7)
    outs = [torch.empty_like(d["x"]) for _ in range(2)]
    ref = torch.empty_like(d["x"])
    K.kda_scan_prefill(d["x"], d["g"], d["init"], d["cu"], ref, None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for s, o in zip(streams, outs):
            K.kda_scan_prefill(d["x"], d["g"], d["init"], d["cu"], o, None, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


def test_graph_replays():
    h, d = make([3000, 1, 900], 96, "bf16", seed=8)
    x, dout = d["x"].clone(), d["dout"].clone()
    out, fin = torch.empty_like(x), torch.empty(3, 96, device="cuda")
    T = x.shape[0]
    chk = torch.empty(-(-T // 128), 96, device="cuda")
    ws = torch.empty(max(8, K.kda_scan_workspace_size(3, T, 96)), dtype=torch.uint8, device="cuda")
    wsb = torch.empty(max(8, K.kda_scan_backward_workspace_size(3, T, 96, has_checkpoints=True)), dtype=torch.uint8,
                      device="cuda")
    grads = dict(dx=torch.empty_like(x), dg=torch.empty(T, 96, device="cuda"), dinit=torch.empty(3, 96, device="cuda"))

    def step():
        K.kda_scan_prefill(x, d["g"], d["init"], d["cu"], out, fin, checkpoints=chk, workspace=ws)
        K.kda_scan_backward(x, d["g"], d["init"], d["cu"], dout, d["dfinal"], checkpoints=chk, grads=grads,
                            workspace=wsb)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(5):
        x.copy_(d["x"] * (i + 1))
        dout.copy_(d["dout"] * (2 - i))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, fin, grads["dx"], grads["dg"], grads["dinit"])]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (out, fin, grads["dx"], grads["dg"], grads["dinit"])):
            assert torch.equal(a, b)


def test_unaligned_views():
    # rows that start off the 16-byte boundary take the narrow path
    h, d = make([150, 40], 64, "bf16", seed=9)
    T = 190
    base = torch.empty(T * 64 + 1, dtype=torch.bfloat16, device="cuda")
    x = base[1:].view(T, 64)
    x.copy_(d["x"])
    out, ref = torch.empty_like(d["x"]), torch.empty_like(d["x"])
    K.kda_scan_prefill(x, d["g"], d["init"], d["cu"], out, None)
    K.kda_scan_prefill(d["x"], d["g"], d["init"], d["cu"], ref, None)
    f = R.scan(h["x"], h["g"], h["init"], h["cu"])
    R.close(host(out), f["h"], f["e_h"], "bf16", "out")
    grads = K.kda_scan_backward(x, d["g"], d["init"], d["cu"], d["dout"], None)
    b = R.scan_backward(h["x"], h["g"], h["init"], h["cu"], h["dout"], None)
    R.close(host(grads["dx"]), b["dx"], b["e_dx"], "bf16", "dx")
    R.close(host(grads["dg"]), b["dg"], b["e_dg"], "fp32", "dg")


def test_heads_as_channels():
    # [T, H, d] tensors as the recurrence's q, k, v: the same as [T, H * d]
    h, d = make([130, 70], 2 * 48, "bf16", seed=10)
    shaped = lambda t: t.view(t.shape[0], 2, 48)   # noqa: E731
    out, fin = torch.empty(200, 2, 48, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 2, 48, device="cuda")
    K.kda_scan_prefill(shaped(d["x"]), shaped(d["g"]), shaped(d["init"]), d["cu"], out, fin)
    o2, f2 = torch.empty_like(d["x"]), torch.empty(2, 96, device="cuda")
    K.kda_scan_prefill(d["x"], d["g"], d["init"], d["cu"], o2, f2)
    assert torch.equal(out.view(200, 96), o2) and torch.equal(fin.view(2, 96), f2)


def test_rejects_mismatched_tensors():
    h, d = make([8], 16, "bf16")
    out = torch.empty_like(d["x"])
    with pytest.raises(ValueError, match="g must be torch.float32"):
        K.kda_scan_prefill(d["x"], d["g"].bfloat16(), d["init"], d["cu"], out, None)
    with pytest.raises(ValueError, match="shape"):
        K.kda_scan_prefill(d["x"], d["g"], d["init"][:, :8].contiguous(), d["cu"], out, None)
    with pytest.raises(ValueError, match="contiguous"):
        K.kda_scan_prefill(d["x"], d["g"], d["init"], d["cu"], out.t().contiguous().t(), None)
    with pytest.raises(ValueError, match="int32"):
        K.kda_scan_prefill(d["x"], d["g"], d["init"], d["cu"].long(), out, None)
    with pytest.raises(TypeError):
        K.kda_scan_prefill(d["x"].half(), d["g"], d["init"], d["cu"], out, None)
    with pytest.raises(ValueError, match="tensor on"):
        K.kda_scan_decode_step(d["x"], d["g"], d["init"].cpu(), out)


@pytest.mark.parametrize("lens,D", [([200, 150], 64), ([300, 33], 130), ([6000, 90], 2561)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gates_of_the_lowest_values(lens, D, dtype):
    # finite gates so low that g log2(e) is not: the decay is 0, as for -infinity
    h, d = make(lens, D, dtype, seed=16)
    T, g = sum(lens), d["g"].clone()
    for i, v in enumerate((torch.finfo(torch.float32).min, -2.5e38, -2.3e38, -1e30, -151.0, -104.0)):
        g[3 + 7 * i::50, i::4] = v
    g[lens[0]:lens[0] + 9] = torch.finfo(torch.float32).min     # whole rows, a sequence's first among them
    hg = host(g)
    out, fin = torch.empty_like(d["x"]), torch.empty_like(d["init"])
    K.kda_scan_prefill(d["x"], g, d["init"], d["cu"], out, fin)
    b = R.scan_backward(h["x"], hg, h["init"], h["cu"], h["dout"], h["dfinal"])
    R.close(host(out), b["fwd"]["h"], b["fwd"]["e_h"], dtype, "out")
    R.close(host(fin), b["fwd"]["final"], b["fwd"]["e_final"], "fp32", "final")
    grads = K.kda_scan_backward(d["x"], g, d["init"], d["cu"], d["dout"], d["dfinal"])
    R.close(host(grads["dx"]), b["dx"], b["e_dx"], dtype, "dx")
    R.close(host(grads["dg"]), b["dg"], b["e_dg"], "fp32", "dg")
    R.close(host(grads["dinit"]), b["dinit"], b["e_dinit"], "fp32", "dinit")
    n = min(T, 40)
    state, o = torch.randn(n, D, device="cuda"), torch.empty_like(d["x"][:n])
    f = R.scan(h["x"][:n], hg[:n], host(state), list(range(n + 1)))
    K.kda_scan_decode_step(d["x"][:n], g[:n], state, o)
    R.close(host(state), f["final"], f["e_final"], "fp32", "state")
    R.close(host(o), f["h"], f["e_h"], dtype, "token")
