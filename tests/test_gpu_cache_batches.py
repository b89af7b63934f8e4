"""kda_decode_tokens_cached: what a sequence gives goes by its own token rows, to the
bit, whatever batch it stands in; and cached calls whose cu_seqlens or slots break
their rules, or whose codes come in a type of their own."""
import pytest
import torch

from gated_delta_rule_40_amd import libkda as K
from test_gpu_cache import DT, FORMATS, check_decode, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    K.load()


def batch_of(p, order, pad=0):
    """The sequences `order` of p (None: an empty one, whose slot nothing is in) as a batch of their own, over the same cache."""
    cu, at, lens = p["cu"].tolist(), [], []
    for n in order:
        rows = [] if n is None else list(range(cu[n], cu[n + 1]))
        at += rows
        lens.append(len(rows))
    pick = torch.tensor(at + [at[0]] * pad).cuda()             # (rows behind the last, of some token)
    s = {name: p[name][pick].contiguous() for name in ("q", "k", "v", "g", "beta")}
    s["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32).cuda()
    s["slots"] = torch.stack([p["slots"][0] * 0 - 1 if n is None else p["slots"][n] for n in order])
    return s, at


@pytest.mark.parametrize("write", [False, True])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_the_bits_are_those_of_the_sequence_alone(dtype, fmt, write):
    """One-row sequences and drafts: alone, side by side, among empty ones, in front of rows that are no sequence's."""
    lens = [1, 4, 1, 1, 9, 1, 2, 1]
    p = make(lens, 3, fmt, dtype, seed=11)
    want = {}

    def run(order, pad):
        s, at = batch_of(p, order, pad)
        cache, scales = p["cache"].clone(), p["scales"].clone()
        out = torch.full(s["v"].shape, 7.0, dtype=DT[dtype], device="cuda")
        K.kda_decode_tokens_cached(*(s[x] for x in ("q", "k", "v", "g", "beta", "cu")), cache, scales, s["slots"], fmt, out=out,
                                   write=write)
        assert torch.all(out[len(at):] == 7.0)
        for i, n in enumerate(order):
            if n is None:
                continue
            slot = int(p["slots"][n])
            got = (out[int(s["cu"][i]):int(s["cu"][i + 1])], cache[slot], scales[slot])
            for a, b in zip(got, want.setdefault(n, got)):
                assert torch.equal(a, b), (order, pad, n)

    for n in range(len(lens)):
        run([n], 0)
    singles = [n for n, length in enumerate(lens) if length == 1]
    drafts = [n for n, length in enumerate(lens) if length > 1]
    for order in (list(range(len(lens))), singles, drafts, drafts + [None] * 20, [None] + singles + [None], [4, 0] + [None] * 12):
        for pad in (0, 1, 40):
            run(order, pad)
    check_decode(dict(p, **batch_of(p, list(range(len(lens))))[0]), fmt, write)
    check_decode(dict(p, **batch_of(p, drafts + [None] * 20)[0]), fmt, write)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_the_bits_do_not_go_by_the_registers(dtype, fmt):
    """No more rows than sequences, and more than 768 of all heads: the kernel for four workgroups a CU.  One row less, or one
    sequence less: the one for three."""
    lens, H = [1, 7, 1, 1, 5, 1, 2, 1, 1, 3, 1, 1], 32                  # 25 rows, 800 with their heads
    p = make(lens, H, fmt, dtype, seed=5)
    whole = list(range(len(lens)))
    results = []
    for order, pad in ((whole + [None] * 13, 0), (whole + [None] * 12, 0), (whole, 30), (whole + [None] * 30, 2)):
        s, at = batch_of(p, order, pad)
        cache, scales = p["cache"].clone(), p["scales"].clone()
        out = torch.empty_like(s["v"])
        K.kda_decode_tokens_cached(*(s[x] for x in ("q", "k", "v", "g", "beta", "cu")), cache, scales, s["slots"], fmt, out=out)
        results.append((out[:25], cache, scales))
    few, _ = batch_of(p, whole[:11] + [None] * 13)                       # 24 rows: 768
    cache, scales = p["cache"].clone(), p["scales"].clone()
    out = torch.empty_like(few["v"])
    K.kda_decode_tokens_cached(*(few[x] for x in ("q", "k", "v", "g", "beta", "cu")), cache, scales, few["slots"], fmt, out=out)
    slots = p["slots"][:11].long()
    for o, c, sc in results:
        assert torch.equal(o, results[0][0]) and torch.equal(c, results[0][1]) and torch.equal(sc, results[0][2])
        assert torch.equal(o[:24], out) and torch.equal(c[slots], cache[slots]) and torch.equal(sc[slots], scales[slots])
    check_decode(dict(p, **batch_of(p, whole + [None] * 13)[0]), fmt, True)


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_sequence_goes_by_its_rows_and_not_by_those_processed(fmt):
    """The first token of a draft has one output, however many tokens are processed."""
    p = make([5, 5, 1], 2, fmt, "fp32")
    outs = []
    for counts in (None, [1, 1, 1], [2, 5, 1], [5, 1, 9]):
        out = torch.full_like(p["v"], 7.0)
        K.kda_decode_tokens_cached(*(p[x] for x in ("q", "k", "v", "g", "beta", "cu")), p["cache"], p["scales"], p["slots"], fmt,
                                   out=out, write=False,
                                   num_tokens=None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda())
        outs.append(out[[0, 5, 10]])
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_every_format_s_own_type_holds_the_same_codes():
    x = torch.randn(3, 77, device="cuda")
    slots = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    for fmt, own in (("fp8", torch.float8_e4m3fn), ("int8", torch.int8), ("fp4", torch.float4_e2m1fn_x2)):
        per = K.kda_cache_entry_bytes(77, fmt)
        cache, scales = torch.zeros(3, per, dtype=torch.uint8, device="cuda"), torch.zeros(3, 3, dtype=torch.uint8, device="cuda")
        again, again_scales = torch.zeros_like(cache).view(own), torch.zeros_like(scales).view(torch.float8_e8m0fnu)
        K.kda_cache_store(x, slots, cache, scales, fmt)
        K.kda_cache_store(x, slots, again, again_scales, fmt)
        assert torch.equal(cache, again.view(torch.uint8)) and torch.equal(scales, again_scales.view(torch.uint8))
        a, b = torch.empty_like(x), torch.empty_like(x)
        K.kda_cache_load(cache, scales, slots, a, fmt)
        K.kda_cache_load(again, again_scales, slots, b, fmt)
        assert torch.equal(a, b)
        p = make([2, 1], 2, fmt)
        o, o2 = torch.empty_like(p["v"]), torch.empty_like(p["v"])
        for out, cache, scales in ((o, p["cache"].clone(), p["scales"].clone()),
                                   (o2, p["cache"].clone().view(own), p["scales"].clone().view(torch.float8_e8m0fnu))):
            K.kda_decode_tokens_cached(*(p[n] for n in ("q", "k", "v", "g", "beta", "cu")), cache, scales, p["slots"], fmt, out=out)
        assert torch.equal(o, o2)


# ------------------------------------------------------------------ cu_seqlens and slots against the rules
GUARD = 4096


def guarded(t):
    """A copy of t inside a larger array, and a function that tells whether what lies around it is as it was."""
    n = t.numel() * t.element_size()
    rows = torch.full((n + 2 * GUARD,), 0x5C, dtype=torch.uint8, device="cuda")
    inner = rows[GUARD:GUARD + n].view(t.dtype).view(t.shape).copy_(t)
    return inner, lambda: bool((rows[:GUARD] == 0x5C).all()) and bool((rows[GUARD + n:] == 0x5C).all())


# entries, and what they come to for six token rows: an entry is held to [0, 6], and a sequence ends no earlier than it begins
BAD_CU = [([-5, 2, 99, 7], [(0, 2), (2, 6), (6, 6)]), ([4, 1, 3, -9], [(4, 4), (1, 3), (3, 3)]),
          ([2 ** 31 - 1, -2 ** 31, 5, 2 ** 31 - 1], [(6, 6), (0, 5), (5, 6)]), ([-1, -1, -1, -1], [(0, 0)] * 3)]


@pytest.mark.parametrize("cu,means", BAD_CU, ids=str)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("out", [True, False])
def test_bad_cu_seqlens_are_held_to_the_token_rows(cu, means, fmt, out):
    p = make([2, 2, 2], 2, fmt, extra=4)
    p["slots"] = torch.tensor([5, 2, 3], dtype=torch.int32, device="cuda")
    want = {}
    for n, (a, b) in enumerate(means):                        # the rows that they come to, as calls of their own
        s = {x: p[x][a:b].contiguous() for x in ("q", "k", "v", "g", "beta")}
        o, cache, scales = torch.empty_like(s["v"]), p["cache"].clone(), p["scales"].clone()
        if b > a:
            K.kda_decode_tokens_cached(*s.values(), torch.tensor([0, b - a], dtype=torch.int32, device="cuda"), cache, scales,
                                       p["slots"][n:n + 1].clone(), fmt, out=o if out else None)
        want[n] = o, cache[p["slots"][n]], scales[p["slots"][n]]
    arrays, intact = {}, []
    for name, t in (("out", torch.full_like(p["v"], 7.0)), ("cache", p["cache"]), ("scales", p["scales"])):
        arrays[name], ok = guarded(t)
        intact.append(ok)
    K.kda_decode_tokens_cached(*(p[x] for x in ("q", "k", "v", "g", "beta")), torch.tensor(cu, dtype=torch.int32, device="cuda"),
                               arrays["cache"], arrays["scales"], p["slots"], fmt, out=arrays["out"] if out else None)
    assert all(ok() for ok in intact)
    rows = torch.zeros(6, dtype=torch.bool)
    for n, (a, b) in enumerate(means):
        o, cache, scales = want[n]
        rows[a:b] = True
        assert not out or torch.equal(arrays["out"][a:b], o)
        slot = int(p["slots"][n])
        assert torch.equal(arrays["cache"][slot], cache) and torch.equal(arrays["scales"][slot], scales)
    others = [s for s in range(7) if s not in (5, 2, 3)]
    assert torch.equal(arrays["cache"][others], p["cache"][others]) and torch.equal(arrays["scales"][others], p["scales"][others])
    assert torch.all(arrays["out"][~rows.cuda() if out else slice(None)] == 7.0)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("elems", [77, 2048])
def test_slots_out_of_range_are_not_written(fmt, elems):
    x = torch.randn(5, elems, device="cuda")
    per = K.kda_cache_entry_bytes(elems, fmt)
    cache, c_ok = guarded(torch.full((3, per), 9, dtype=torch.uint8, device="cuda"))
    scales, s_ok = guarded(torch.full((3, -(-elems // 32)), 9, dtype=torch.uint8, device="cuda"))
    dst, d_ok = guarded(torch.full((5, elems), 7.0, device="cuda"))
    slots = torch.tensor([-1, 3, 1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    K.kda_cache_store(x, slots, cache, scales, fmt)
    K.kda_cache_load(cache, scales, slots, dst, fmt)
    assert c_ok() and s_ok() and d_ok()
    assert torch.all(cache[[0, 2]] == 9) and torch.all(scales[[0, 2]] == 9)
    assert not dst[[0, 1, 3, 4]].any() and dst[2].any()
