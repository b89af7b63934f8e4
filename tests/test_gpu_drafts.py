"""A KDA layer's queries, keys and states when tokens are drafted, as they would be
used together: norm and rotation, decoding on cached states without committing,
verification, and the accepted tokens committed; a prompt into the recurrence and
its gradients; streams, graphs and threads."""
import threading

import numpy as np
import pytest
import torch

import cache_ref as C
from layer_ref import close
from gated_delta_rule_40_amd import libkda as K

pytestmark = pytest.mark.gpu

D, H, V = 128, 3, 700
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    K.load()


def host(t):
    return t.detach().double().cpu().numpy()


def batch(lens, seed=0, fmt="int8", dtype=torch.float32):
    """A step's inputs: a token and its drafts for every sequence, states in a cache."""
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)                       # noqa: E731
    N, T = len(lens), sum(lens)
    d = dict(rows=rnd(T, 3 * H * D).to(dtype), g=-5 / 16 * torch.rand(T, H, D, generator=gen), beta=torch.sigmoid(rnd(T, H)),
             cu=torch.tensor(np.cumsum([0] + lens), dtype=torch.int32), tokens=torch.randint(0, V, (T,), generator=gen).int(),
             accept=torch.rand(T, generator=gen), sample=torch.rand(N, generator=gen))
    logits = 2 * rnd(T, V)
    logits[torch.arange(T - 1), d["tokens"][1:].long()] += 4.0          # drafts that are often right
    d["target"] = torch.softmax(logits, 1)
    d["draft"] = torch.softmax(logits + 2.0 * rnd(T, V), 1).roll(1, 0)
    d = {k: v.cuda() for k, v in d.items()}
    S = N + 2
    d["slots"] = torch.randperm(S, generator=gen)[:N].int().cuda()
    d["cache"] = torch.empty(S, H, D, D // 2 if fmt == "fp4" else D, dtype=torch.uint8, device="cuda")
    d["scales"] = torch.empty(S, H, D, 4, dtype=torch.uint8, device="cuda")
    K.kda_cache_store(0.2 * rnd(S, H, D, D).cuda(), torch.arange(S, dtype=torch.int32, device="cuda"), d["cache"], d["scales"], fmt)
    d["fmt"] = fmt
    for name in ("q", "k"):
        d[name + "_out"] = torch.empty(T, H, D, dtype=dtype, device="cuda")
    d["out"] = torch.empty(T, H, D, dtype=dtype, device="cuda")
    d["num"], d["next"] = (torch.empty(N, dtype=torch.int32, device="cuda") for _ in range(2))
    d["ws"] = torch.empty(K.kda_verify_drafts_workspace_size(N, V), dtype=torch.uint8, device="cuda")
    return d


def step(d, stream=None):
    """The calls of one step, as a server makes them."""
    q, k, v = d["rows"].unflatten(1, (3, H, D)).unbind(1)
    if "v" not in d:
        d["v"] = v.contiguous()
    K.kda_qknorm(q, k, d["q_out"], d["k_out"], norm="l2", eps=EPS, q_scale=D ** -0.5, stream=stream)
    args = (d["q_out"], d["k_out"], d["v"], d["g"], d["beta"], d["cu"], d["cache"], d["scales"], d["slots"], d["fmt"])
    K.kda_decode_tokens_cached(*args, out=d["out"], write=False, stream=stream)
    K.kda_verify_drafts(d["target"], d["draft"], d["tokens"], d["cu"], d["accept"], d["sample"], d["num"], d["next"],
                        workspace=d["ws"], stream=stream)
    K.kda_decode_tokens_cached(*args, num_tokens=d["num"], write=True, stream=stream)


RESULTS = ("q_out", "k_out", "out", "num", "next", "cache", "scales")


def results(d):
    return {n: d[n].clone() for n in RESULTS}


@pytest.mark.parametrize("fmt", ["fp8", "int8", "fp4"])
def test_a_step_of_drafts(fmt):
    lens = [5, 1, 4, 0, 6, 2, 5]
    d = batch(lens, fmt=fmt)
    before, bsc = d["cache"].cpu().numpy(), d["scales"].cpu().numpy()
    step(d)
    rows = host(d["rows"]).reshape(-1, 3, H, D)
    normed = {}
    for i, name, scale in ((0, "q", float(np.float32(D ** -0.5))), (1, "k", 1.0)):
        y, e = C.qknorm(rows[:, i], None, "l2", float(np.float32(EPS)), scale, None, 0, False)
        close(host(d[name + "_out"]), y, e, "fp32", name)
        normed[name] = host(d[name + "_out"])                            # the next call's inputs are the rounded ones
    num, nxt = C.verify(host(d["target"]), host(d["draft"]), d["tokens"].tolist(), d["cu"].tolist(), host(d["accept"]),
                        host(d["sample"]))
    assert d["num"].tolist() == num and d["next"].tolist() == nxt
    assert 1 < max(num) and num[3] == 0 and any(a < b for a, b in zip(num, lens))
    after, asc = d["cache"].cpu().numpy(), d["scales"].cpu().numpy()
    cu, g, beta = d["cu"].tolist(), host(d["g"]), host(d["beta"])
    for n, slot in enumerate(d["slots"].tolist()):
        for h in range(H):
            S0 = C.dequantise(before[slot, h], bsc[slot, h], fmt, D)
            at = slice(cu[n], cu[n + 1])
            o, _, eo, _ = C.decode(normed["q"][at, h], normed["k"][at, h], rows[at, 2, h], g[at, h], beta[at, h], S0)
            close(host(d["out"][at, h]), o, eo, "fp32", "out")
            at = slice(cu[n], cu[n] + num[n])
            _, S, _, E = C.decode(normed["q"][at, h], normed["k"][at, h], rows[at, 2, h], g[at, h], beta[at, h], S0)
            value = C.dequantise(after[slot, h], asc[slot, h], fmt, D)
            half = np.repeat(2.0 ** (asc[slot, h].astype(float) - 127), 32, 1) * {"fp8": 16, "int8": 1 / 128, "fp4": 1}[fmt]
            assert np.all(np.abs(value - S) <= half + 1.01 * E)           # half of the format's largest step
    untouched = [s for s in range(len(before)) if s not in [int(x) for x, c in zip(d["slots"], num) if c]]
    assert np.array_equal(before[untouched], after[untouched]) and np.array_equal(bsc[untouched], asc[untouched])


def test_a_committed_draft_is_the_tokens_one_by_one():
    """fp32 states: committing an accepted prefix from a cached state equals the uncached replay of the same prefix."""
    d = batch([4, 4, 4])
    state = torch.empty(3, H, D, D, device="cuda")
    K.kda_cache_load(d["cache"], d["scales"], d["slots"], state, "int8")
    step(d)
    K.kda_decode_tokens(d["q_out"], d["k_out"], d["v"], d["g"], d["beta"], d["cu"], state, state, num_tokens=d["num"])
    again = torch.empty_like(state)
    K.kda_cache_load(d["cache"], d["scales"], d["slots"], again, "int8")
    # a scale is below 128 / 127 of the block's largest, and half a step of int8 is 1 / 128 of it: less than 1 / 127 of the
    # largest, and 1 / 64 leaves room for what two fp32 evaluations differ by
    top = state.abs().unflatten(-1, (4, 32)).amax(-1, keepdim=True).expand(-1, -1, -1, -1, 32).flatten(-2)
    assert torch.all((again - state).abs() <= top / 64)


def test_steps_in_a_graph_are_the_eager_ones():
    d, e = batch([3, 5, 1, 2], seed=3), batch([3, 5, 1, 2], seed=3)
    step(d)                                                               # sizes are asked for before the capture
    torch.cuda.synchronize()
    for n in ("cache", "scales"):
        d[n].copy_(e[n])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(d)
    for n in ("cache", "scales"):
        d[n].copy_(e[n])
    for i in range(4):                                                    # each advances the cached states
        for x in (d, e):
            x["rows"].copy_(torch.randn(x["rows"].shape, generator=torch.Generator().manual_seed(i)))
            x.pop("v", None) if x is e else x["v"].copy_(x["rows"].unflatten(1, (3, H, D))[:, 2])
        graph.replay()
        step(e)
        torch.cuda.synchronize()
        a, b = results(d), results(e)
        assert all(torch.equal(a[n], b[n]) for n in RESULTS), (i, [n for n in RESULTS if not torch.equal(a[n], b[n])])


def test_other_streams_and_threads_at_once():
    want = []
    for i in range(4):
        d = batch([2 + i, 1, 5], seed=i)
        step(d)
        torch.cuda.synchronize()
        want.append(results(d))
    work = [batch([2 + i, 1, 5], seed=i) for i in range(4)]
    for d in work:
        d["v"] = d["rows"].unflatten(1, (3, H, D))[:, 2].contiguous()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    threads = [threading.Thread(target=step, args=(d, s)) for d, s in zip(work, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i, d in enumerate(work):
        assert all(torch.equal(d[n], want[i][n]) for n in RESULTS), i


def test_a_call_that_makes_its_tensors_on_another_stream():
    """Gradients and a workspace of a call on a stream of its own, used there."""
    x = torch.randn(50, 2, 64, device="cuda")
    w, dy = torch.ones(64, device="cuda"), torch.randn(50, 2, 64, device="cuda")
    want = K.kda_qknorm_backward(x, x, dy, dy, q_weight=w, k_weight=w)
    d = batch([3, 2])
    step(d)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = K.kda_qknorm_backward(x, x, dy, dy, q_weight=w, k_weight=w, stream=s)
    num, nxt = torch.empty_like(d["num"]), torch.empty_like(d["next"])
    K.kda_verify_drafts(d["target"], d["draft"], d["tokens"], d["cu"], d["accept"], d["sample"], num, nxt, stream=s)
    s.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want) and torch.equal(num, d["num"]) and torch.equal(nxt, d["next"])


def test_gradients_in_a_graph_beside_eager_ones():
    """Forward and backward captured, replayed with eager work between, against eager calls."""
    gen = torch.Generator().manual_seed(0)
    T = 300
    q, k = torch.randn(T, 4, D, generator=gen).cuda(), torch.randn(T, 2, D, generator=gen).cuda()
    w, dq, dk = torch.rand(D).cuda() + 0.5, torch.randn_like(q), torch.randn_like(k)
    form = dict(q_weight=w, k_weight=w, norm="rms", positions=torch.arange(T, dtype=torch.int32, device="cuda"),
                inv_freq=torch.rand(32).cuda())
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    grads = K.kda_qknorm_backward(q, k, dq, dk, **form)
    ws = torch.empty(K.kda_qknorm_backward_workspace_size(T, 4, 2, D, torch.float32), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        K.kda_qknorm(q, k, qo, ko, **form)
        K.kda_qknorm_backward(q, k, dq, dk, grads=grads, workspace=ws, **form)
    for i in range(3):
        q.normal_()
        dk.normal_()
        graph.replay()
        torch.cuda.synchronize()
        q2, k2 = torch.empty_like(q), torch.empty_like(k)
        K.kda_qknorm(q, k, q2, k2, **form)
        want = K.kda_qknorm_backward(q, k, dq, dk, **form)
        assert torch.equal(qo, q2) and torch.equal(ko, k2) and all(torch.equal(grads[n], want[n]) for n in want), i


def test_through_the_recurrence_and_back():
    """Norm of queries and keys, prefill, kda_backward, and the norm's gradients from its fp32 ones, against autograd in fp64."""
    T, lens = 70, [40, 0, 30]
    gen = torch.Generator().manual_seed(7)
    rows = torch.randn(T, 2 * H * D, generator=gen)
    v, g, beta = torch.randn(T, H, D, generator=gen), -0.3 * torch.rand(T, H, D, generator=gen), torch.rand(T, H, generator=gen)
    dout = torch.randn(T, H, D, generator=gen)
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32)
    x = rows.double().requires_grad_()
    q, k = x.unflatten(1, (2, H, D)).unbind(1)
    unit = lambda y: y / torch.sqrt((y * y).sum(-1, keepdim=True) + EPS)  # noqa: E731
    q, k, outs = unit(q) * D ** -0.5, unit(k), []
    for n in range(3):
        S = torch.zeros(H, D, D, dtype=torch.float64)
        for t in range(int(cu[n]), int(cu[n + 1])):
            S = S * torch.exp(g[t].double())[..., None]
            u = beta[t].double()[:, None] * (v[t].double() - (S * k[t][..., None]).sum(1))
            S = S + k[t][..., None] * u[:, None]
            outs.append((S * q[t][..., None]).sum(1))
    (torch.stack(outs) * dout.double()).sum().backward()

    dev = {n: t.cuda() for n, t in dict(rows=rows, v=v, g=g, beta=beta, dout=dout, cu=cu).items()}
    qd, kd = dev["rows"].unflatten(1, (2, H, D)).unbind(1)
    qn, kn = (torch.empty(T, H, D, device="cuda") for _ in range(2))
    form = dict(norm="l2", eps=EPS, q_scale=D ** -0.5)
    K.kda_qknorm(qd, kd, qn, kn, **form)
    out = torch.empty(T, H, D, device="cuda")
    K.kda_prefill(qn, kn, dev["v"], dev["g"], dev["beta"], None, dev["cu"], out, None)
    gr = K.kda_backward(qn, kn, dev["v"], dev["g"], dev["beta"], None, dev["cu"], dev["dout"], want_dinit=False)
    drows = torch.empty_like(dev["rows"])
    dq, dk = drows.unflatten(1, (2, H, D)).unbind(1)
    K.kda_qknorm_backward(qd, kd, gr["dq"], gr["dk"], grads=dict(dq=dq, dk=dk), **form)
    ref = torch.stack(outs).detach()
    rms = float(ref.pow(2).mean().sqrt())
    assert float((out.double().cpu() - ref).abs().max()) <= 1e-4 * rms    # the library's bound for fp32 inputs
    rms = float(x.grad.pow(2).mean().sqrt())
    assert float((drows.double().cpu() - x.grad).abs().max()) <= 1e-3 * rms


def test_snapshots_kept_in_a_cache_restore_a_prefix():
    """kda_prefill_snapshots' states written to slots (those that are not kept to none), read back, and the prompt continued."""
    T, gen = 128, torch.Generator().manual_seed(9)
    rnd = lambda *s: torch.randn(*s, generator=gen).cuda()                # noqa: E731
    q, k, v = rnd(T, H, D) * D ** -0.5, rnd(T, H, D), rnd(T, H, D)
    k = k / k.norm(dim=-1, keepdim=True)
    g, beta = -0.3 * torch.rand(T, H, D, generator=gen).cuda(), torch.rand(T, H, generator=gen).cuda()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")    # noqa: E731
    out, snaps = torch.empty(T, H, D, device="cuda"), torch.zeros(1, 4, H, D, D, device="cuda")
    K.kda_prefill_snapshots(q, k, v, g, beta, None, i32(0, T), out, None, snaps, 32)
    cache = torch.zeros(3, H, D, D, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(3, H, D, 4, dtype=torch.uint8, device="cuda")
    K.kda_cache_store(snaps[0], i32(-1, 2, -1, 0), cache, scales, "int8")  # after 64 and 128 tokens
    state = torch.empty(1, H, D, D, device="cuda")
    K.kda_cache_load(cache, scales, i32(2), state, "int8")
    top = snaps[0, 1].abs().unflatten(-1, (4, 32)).amax(-1, keepdim=True).expand(-1, -1, -1, 32).flatten(-2)
    assert torch.all((state[0] - snaps[0, 1]).abs() <= top / 127)         # half a step (as above)
    rest = torch.empty(64, H, D, device="cuda")
    K.kda_prefill(q[64:], k[64:], v[64:], g[64:], beta[64:], state, i32(0, 64), rest, None)
    # the state's rounding alone is between them: its share decays with the gates
    off = (rest - out[64:]).abs().amax((1, 2))
    assert float(off[-1]) < float(off[0]) < 0.05
