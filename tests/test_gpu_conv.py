"""kda_conv_prefill, kda_conv_decode_step and kda_conv_backward against the
convolution in fp64 (tests/layer_ref.py), over sequences shorter than the
kernel, empty ones, and ones that end at and beyond the kernels' strips."""
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


def make(lens, D, W, dtype, init=True, bias=True, tail=0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens) + tail, len(lens)
    rnd = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    d = dict(x=rnd(T, D).to(DT[dtype]), w=rnd(D, W) * 0.6, b=rnd(D) if bias else None,
             init=rnd(N, W - 1, D).to(DT[dtype]) if init else None, dout=rnd(T, D).to(DT[dtype]),
             dfinal=rnd(N, W - 1, D).to(DT[dtype]) if init else None,
             cu=torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32))
    h = {k: None if v is None else v.double().numpy() for k, v in d.items()}
    h["cu"] = d["cu"].tolist()
    return h, {k: None if v is None else v.cuda() for k, v in d.items()}


def host(t):
    return t.detach().double().cpu().numpy()


LENS = [[1], [2, 1, 3], [0, 0], [4, 0, 0, 1, 2, 0, 3], [31, 33, 64, 65, 1], [128, 128], [257, 0, 500], [3] * 50 + [700]]
SHAPES = [(1, 2), (3, 4), (64, 3), (130, 4), (512, 4), (520, 2), (1000, 3), (257, 4), (515, 3), (1023, 2)]
CASES = [(lens, *SHAPES[(i * 3 + j) % len(SHAPES)]) for i, lens in enumerate(LENS) for j in range(3)]


@pytest.mark.parametrize("lens,D,W", CASES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("silu,init,bias", [(True, True, True), (False, False, False), (True, False, True)])
def test_prefill(lens, D, W, dtype, silu, init, bias):
    tail = 5 if D % 2 == 0 else 0
    h, d = make(lens, D, W, dtype, init, bias, tail)
    T, N, own = d["x"].shape[0], len(lens), sum(lens)
    out = torch.full((T, D), 77.0, dtype=DT[dtype], device="cuda")
    fin = torch.full((N, W - 1, D), 77.0, dtype=DT[dtype], device="cuda")
    K.kda_conv_prefill(d["x"], d["w"], d["b"], d["init"], d["cu"], out, fin, silu=silu)
    f = R.conv(h["x"], h["w"], h["b"], h["init"], h["cu"], silu)
    R.close(host(out)[:own], f["out"][:own], f["e_out"][:own], dtype, "out")
    assert np.all(host(out)[own:] == 77.0)
    assert np.array_equal(host(fin), f["final"])
    again, state = torch.empty_like(out), None if d["init"] is None else d["init"].clone()
    K.kda_conv_prefill(d["x"], d["w"], d["b"], state, d["cu"], again, state, silu=silu)   # in place, or not wanted
    assert torch.equal(again[:own], out[:own])
    if state is not None:
        assert torch.equal(state, fin)


@pytest.mark.parametrize("lens,D,W", CASES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("silu,init,bias", [(True, True, True), (False, False, False), (False, True, True)])
def test_backward(lens, D, W, dtype, silu, init, bias):
    tail = 5 if D % 2 == 0 else 0
    h, d = make(lens, D, W, dtype, init, bias, tail, seed=1)
    T, N, own = d["x"].shape[0], len(lens), sum(lens)
    f32 = torch.float32
    full = lambda dt, *s: torch.full(s, 77.0, dtype=dt, device="cuda")   # noqa: E731
    grads = dict(dx=full(DT[dtype], T, D), dweight=full(f32, D, W), dbias=full(f32, D) if bias else None,
                 dinit=full(DT[dtype], N, W - 1, D) if init else None)
    K.kda_conv_backward(d["x"], d["w"], d["b"], d["init"], d["cu"], d["dout"], d["dfinal"], silu=silu, grads=grads)
    g = R.conv_backward(h["x"], h["w"], h["b"], h["init"], h["cu"], silu, h["dout"], h["dfinal"])
    if own < T:   # rows of no sequence count for nothing
        assert np.all(host(grads["dx"])[own:] == 77.0)
    R.close(host(grads["dx"])[:own], g["dx"][:own], g["e_dx"][:own], dtype, "dx")
    sub = {**h, "x": h["x"][:own], "dout": h["dout"][:own]}
    g = R.conv_backward(sub["x"], h["w"], h["b"], h["init"], h["cu"], silu, sub["dout"], h["dfinal"])
    R.close(host(grads["dweight"]), g["dweight"], g["e_dweight"], "fp32", "dweight")
    if bias:
        R.close(host(grads["dbias"]), g["dbias"], g["e_dbias"], "fp32", "dbias")
    if init:
        R.close(host(grads["dinit"]), g["dinit"], g["e_dinit"], dtype, "dinit")


@pytest.mark.parametrize("N,most", [(63, 9), (64, 9), (65, 90), (700, 8), (4100, 3)])
def test_many_sequences(N, most):
    # more entries of cu_seqlens than a wave holds at once, empty sequences among them
    lens = np.random.default_rng(N).integers(0, most, N).tolist() + [0] * 70 + [3]
    h, d = make(lens, 8, 4, "fp32", tail=1, seed=6)
    T = sum(lens)
    out, fin = torch.full_like(d["x"], 77.0), torch.full_like(d["init"], 77.0)
    K.kda_conv_prefill(d["x"], d["w"], d["b"], d["init"], d["cu"], out, fin)
    g = K.kda_conv_backward(d["x"], d["w"], d["b"], d["init"], d["cu"], d["dout"], d["dfinal"])
    r = R.conv_backward(h["x"][:T], h["w"], h["b"], h["init"], h["cu"], True, h["dout"][:T], h["dfinal"])
    R.close(host(out)[:T], r["fwd"]["out"], r["fwd"]["e_out"], "fp32", "out")
    assert np.array_equal(host(fin), r["fwd"]["final"]) and float(out[T:].min()) == 77.0
    R.close(host(g["dx"])[:T], r["dx"], r["e_dx"], "fp32", "dx")
    R.close(host(g["dweight"]), r["dweight"], r["e_dweight"], "fp32", "dweight")
    R.close(host(g["dbias"]), r["dbias"], r["e_dbias"], "fp32", "dbias")
    R.close(host(g["dinit"]), r["dinit"], r["e_dinit"], "fp32", "dinit")


SLOTS = [[40] + [0] * 200, [0] * 130 + [300], [150] + [0] * 90 + [1, 2] + [0] * 70 + [200, 0, 0, 9], [0] * 300]


@pytest.mark.parametrize("lens", SLOTS, ids=lambda v: "%dof%d" % (sum(map(bool, v)), len(v)))
@pytest.mark.parametrize("init", [True, False])
def test_slots_left_empty(lens, init):
    # more sequences begin at one token than a wave holds entries
    h, d = make(lens, 130, 4, "bf16", init, tail=2, seed=13)
    T, N = sum(lens), len(lens)
    out = torch.full_like(d["x"], 77.0)
    fin = torch.full((N, 3, 130), 77.0, dtype=torch.bfloat16, device="cuda")
    K.kda_conv_prefill(d["x"], d["w"], d["b"], d["init"], d["cu"], out, fin)
    g = K.kda_conv_backward(d["x"], d["w"], d["b"], d["init"], d["cu"], d["dout"], d["dfinal"])
    r = R.conv_backward(h["x"][:T], h["w"], h["b"], h["init"], h["cu"], True, h["dout"][:T], h["dfinal"])
    R.close(host(out)[:T], r["fwd"]["out"], r["fwd"]["e_out"], "bf16", "out")
    assert np.array_equal(host(fin), r["fwd"]["final"]) and float(out[T:].min()) == 77.0
    R.close(host(g["dx"])[:T], r["dx"], r["e_dx"], "bf16", "dx")
    R.close(host(g["dweight"]), r["dweight"], r["e_dweight"], "fp32", "dweight")
    R.close(host(g["dinit"]), r["dinit"], r["e_dinit"], "bf16", "dinit")
    if init:
        K.kda_conv_prefill(d["x"], d["w"], d["b"], d["init"], d["cu"], out, d["init"])
        assert torch.equal(d["init"], fin)


@pytest.mark.parametrize("N,D", [(1, 1), (3, 5), (8, 512), (65, 999)])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decode_steps_equal_prefill(N, D, W, dtype):
    # five tokens one by one against one prefill of five tokens, for a batch of N
    h, d = make([5] * N, D, W, dtype, seed=2)
    f = R.conv(h["x"], h["w"], h["b"], h["init"], h["cu"], True)
    state = d["init"].clone()
    x = d["x"].view(N, 5, D)
    for p in range(5):
        out = torch.empty(N, D, dtype=DT[dtype], device="cuda")
        K.kda_conv_decode_step(x[:, p].contiguous(), d["w"], d["b"], state, out)
        R.close(host(out), f["out"].reshape(N, 5, D)[:, p], f["e_out"].reshape(N, 5, D)[:, p], dtype, "out")
    assert np.array_equal(host(state), f["final"])
    # in place, without bias and activation
    y = x[:, 0].contiguous()
    K.kda_conv_decode_step(y, d["w"], None, d["init"].clone(), y, silu=False)
    f = R.conv(h["x"].reshape(N, 5, D)[:, 0], h["w"], None, h["init"], list(range(N + 1)), False)
    R.close(host(y), f["out"], f["e_out"], dtype, "in place")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nan_and_infinity_reach_only_their_tokens(bad):
    lens, D, W = [40, 2, 90, 30], 72, 4
    h, d = make(lens, D, W, "fp32", tail=2, seed=3)
    cu = h["cu"]
    clean, fin = torch.empty_like(d["x"]), torch.empty_like(d["init"])
    K.kda_conv_prefill(d["x"], d["w"], d["b"], d["init"], d["cu"], clean, fin, silu=False)
    gclean = K.kda_conv_backward(d["x"], d["w"], d["b"], d["init"], d["cu"], d["dout"], d["dfinal"], silu=False)
    x, dout = d["x"].clone(), d["dout"].clone()
    x[cu[2] - 1] = bad                     # the last token of sequence 1
    x[cu[-1]:] = bad
    dout[cu[-1]:] = bad
    dout[cu[2]] = bad                      # the first of sequence 2
    out, f2 = torch.zeros_like(x), torch.empty_like(fin)
    K.kda_conv_prefill(x, d["w"], d["b"], d["init"], d["cu"], out, f2, silu=False)
    g = K.kda_conv_backward(x, d["w"], d["b"], d["init"], d["cu"], dout, d["dfinal"], silu=False)
    keep = torch.ones(sum(lens), dtype=torch.bool)
    keep[cu[2] - 1] = False
    assert torch.equal(out[:sum(lens)][keep], clean[:sum(lens)][keep])
    assert not torch.isfinite(out[cu[2] - 1]).any()
    keep[:] = True
    keep[cu[2]] = False                    # its gradient goes to its own sequence's tokens and state only
    assert torch.equal(g["dx"][:sum(lens)][keep], gclean["dx"][:sum(lens)][keep])
    assert torch.equal(g["dinit"][[0, 1, 3]], gclean["dinit"][[0, 1, 3]])


def test_silu_at_large_inputs():
    # exp(-pre) overflows or vanishes: out is 0 or pre, and nothing is NaN
    x = torch.tensor([[-1e30, -200.0, -90.0, 0.0, 90.0, 200.0, 1e30]], device="cuda")
    w = torch.zeros(7, 2, device="cuda")
    w[:, 1] = 1.0
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)
    K.kda_conv_prefill(x, w, None, None, cu, out, None)
    assert torch.allclose(out, torch.tensor([[0.0, 0.0, 0.0, 0.0, 90.0, 200.0, 1e30]], device="cuda"), atol=1e-30)
    g = K.kda_conv_backward(x, w, None, None, cu, torch.ones_like(x))
    assert torch.allclose(g["dx"], torch.tensor([[0.0, 0.0, 0.0, 0.5, 1.0, 1.0, 1.0]], device="cuda"), atol=1e-30)


def test_token_in_place_and_prompt_refused():
    _, d = make([40, 3], 72, 4, "bf16", seed=15)
    a, o, s1, s2 = d["x"][:2].clone(), torch.empty_like(d["x"][:2]), d["init"].clone(), d["init"].clone()
    K.kda_conv_decode_step(d["x"][:2], d["w"], d["b"], s1, o)
    K.kda_conv_decode_step(a, d["w"], d["b"], s2, a)
    assert torch.equal(a, o) and torch.equal(s1, s2)
    before = d["x"].clone()
    with pytest.raises(RuntimeError):
        K.kda_conv_prefill(d["x"], d["w"], d["b"], d["init"], d["cu"], d["x"], None)
    with pytest.raises(RuntimeError):
        K.kda_conv_backward(d["x"], d["w"], d["b"], None, d["cu"], d["dout"],
                            grads=dict(dx=d["x"], dweight=torch.empty_like(d["w"])))
    assert torch.equal(d["x"], before)


def test_same_bits_streams_and_graph_replays():
    h, d = make([900, 1, 2000, 3], 264, 4, "bf16", seed=4)
    x, dout = d["x"].clone(), d["dout"].clone()
    T = x.shape[0]
    out, fin = torch.empty_like(x), torch.empty_like(d["init"])
    ws = torch.empty(max(4, K.kda_conv_backward_workspace_size(4, T, 264, 4)), dtype=torch.uint8, device="cuda")
    grads = dict(dx=torch.empty_like(x), dweight=torch.empty(264, 4, device="cuda"),
                 dbias=torch.empty(264, device="cuda"), dinit=torch.empty_like(d["init"]))

    def step(stream=None):
        K.kda_conv_prefill(x, d["w"], d["b"], d["init"], d["cu"], out, fin, stream=stream)
        K.kda_conv_backward(x, d["w"], d["b"], d["init"], d["cu"], dout, d["dfinal"], grads=grads, workspace=ws,
                            stream=stream)

    results = lambda: [t.clone() for t in (out, fin, *grads.values())]   # noqa: E731
    step()
    first = results()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, results()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(d["x"] * (i + 1))
        dout.copy_(d["dout"] * (2 - i))
        graph.replay()
        torch.cuda.synchronize()
        got = results()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, results()))


def test_no_sequences_and_no_tokens():
    x = torch.zeros(6, 16, device="cuda")
    w, b = torch.ones(16, 4, device="cuda"), torch.ones(16, device="cuda")
    g = K.kda_conv_backward(x, w, b, None, torch.zeros(1, dtype=torch.int32, device="cuda"), x, want_dinit=False,
                            grads=dict(dx=torch.full_like(x, 7.0), dweight=torch.full_like(w, 7.0),
                                       dbias=torch.full_like(b, 7.0)))
    assert bool((g["dweight"] == 0).all()) and bool((g["dbias"] == 0).all()) and bool((g["dx"] == 7.0).all())
    init = torch.randn(2, 3, 16, device="cuda")
    fin, x0 = torch.empty_like(init), torch.empty(0, 16, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    K.kda_conv_prefill(x0, w, b, init, cu, torch.empty_like(x0), fin)
    assert torch.equal(fin, init)
    g = K.kda_conv_backward(x0, w, b, init, cu, x0, init)
    assert torch.equal(g["dinit"], init) and bool((g["dweight"] == 0).all()) and bool((g["dbias"] == 0).all())


def test_unaligned_views():
    h, d = make([150, 40], 64, 4, "bf16", seed=5)
    base = torch.empty(190 * 64 + 1, dtype=torch.bfloat16, device="cuda")
    x = base[1:].view(190, 64)
    x.copy_(d["x"])
    out = torch.empty_like(d["x"])
    K.kda_conv_prefill(x, d["w"], d["b"], d["init"], d["cu"], out, None)
    f = R.conv(h["x"], h["w"], h["b"], h["init"], h["cu"], True)
    R.close(host(out), f["out"], f["e_out"], "bf16", "out")
    g = K.kda_conv_backward(x, d["w"], d["b"], d["init"], d["cu"], d["dout"], d["dfinal"])
    r = R.conv_backward(h["x"], h["w"], h["b"], h["init"], h["cu"], True, h["dout"], h["dfinal"])
    R.close(host(g["dx"]), r["dx"], r["e_dx"], "bf16", "dx")
    R.close(host(g["dweight"]), r["dweight"], r["e_dweight"], "fp32", "dweight")


def test_rejects_mismatched_tensors():
    h, d = make([8], 16, 4, "bf16")
    out = torch.empty_like(d["x"])
    with pytest.raises(ValueError, match="weight must be torch.float32"):
        K.kda_conv_prefill(d["x"], d["w"].bfloat16(), None, None, d["cu"], out, None)
    with pytest.raises(ValueError, match="initial_state must be torch.bfloat16"):
        K.kda_conv_prefill(d["x"], d["w"], None, d["init"].float(), d["cu"], out, None)
    with pytest.raises(ValueError, match="shape"):
        K.kda_conv_prefill(d["x"], d["w"], None, d["init"][:, :2].contiguous(), d["cu"], out, None)
    with pytest.raises(ValueError, match="out must be"):
        K.kda_conv_prefill(d["x"], d["w"], None, None, d["cu"], out.float(), None)
    with pytest.raises(K.KdaError) as e:
        K.kda_conv_prefill(d["x"], torch.zeros(16, 5, device="cuda"), None, None, d["cu"], out, None)
    assert e.value.status == K.KDA_ERR_UNSUPPORTED
