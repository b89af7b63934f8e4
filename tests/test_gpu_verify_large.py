"""kda_verify_drafts where a wave sums two parts of a row, on either side of that, and
where cu_seqlens breaks its rules, against the definition in fp64
(tests/cache_ref.py)."""
import pytest
import torch

from gated_delta_rule_40_amd import libkda as K
from test_gpu_cache_batches import guarded
from test_gpu_verify import check, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    K.load()


# 65 parts of 1,024 a row, the last of 464; 16,384 parts and more go by twos: 252 sequences have 16,380, 253 16,445
@pytest.mark.parametrize("greedy", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N", [252, 253])
def test_where_two_parts_a_wave_begin(N, dtype, greedy):
    lens = [(1, 3, 0, 2, 1, 4)[n % 6] for n in range(N)]
    a = list(make(lens, 66000, dtype, seed=N))
    if greedy:
        a[1] = None
    num, nxt = check(*a)
    assert 0 in num and any(0 < c < n for c, n in zip(num, lens)) and -1 in nxt
    t, d, tok, cu, acc, smp = a
    for n in (0, 1, 5, N - 2, N - 1):                         # the same sequences alone
        at = slice(int(cu[n]), int(cu[n + 1]))
        assert run(t[at], None if greedy else d[at], tok[at], [0, lens[n]], acc[at], smp[n:n + 1]) == ([num[n]], [nxt[n]])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_the_first_and_last_weights_of_rows_by_twos(dtype):
    """A single weight in the first, the last and the odd part; and thresholds at the ends of a row."""
    N, V = 256, 65536 + 500
    t = torch.zeros(N, V, dtype=torch.float32)
    at = torch.tensor([(0, 1023, 1024, 2047, 2048, 65535, 65536, V - 1)[n % 8] for n in range(N)])
    t[torch.arange(N), at] = 0.25
    t = t.to(torch.float32 if dtype == "fp32" else torch.bfloat16).cuda()
    zeros = [0.0] * N
    for u in (0.0, 0.5, 0.99999994):
        assert check(t, None, [0] * N, range(N + 1), zeros, [u] * N) == ([1] * N, at.tolist())
    t[:, 0] = t[:, V - 1] = 0.5                               # equal weights at both ends: the second from one half on
    t[:, 1:V - 1] = 0
    sample = [0.5 if n % 2 else 0.49999997 for n in range(N)]
    assert check(t, None, [0] * N, range(N + 1), zeros, sample)[1] == [V - 1 if n % 2 else 0 for n in range(N)]


# entries, and what they come to for nine token rows: an entry is held to [0, 9], and a sequence ends no earlier than it begins
@pytest.mark.parametrize("V", [200, 20000])                   # one launch and two
@pytest.mark.parametrize("cu,means", [([-4, 3, 100, 5], [(0, 3), (3, 9), (9, 9)]), ([7, 2, 2 ** 31 - 1, -2 ** 31],
                                      [(7, 7), (2, 9), (9, 9)]), ([-1, -2, -3, -4], [(0, 0)] * 3)], ids=str)
def test_bad_cu_seqlens_are_held_to_the_token_rows(cu, means, V):
    t, d, tok, _, acc, smp = make([3, 4, 2], V)
    dev = lambda x, dt: torch.as_tensor(x, dtype=dt).cuda()   # noqa: E731
    need = K.kda_verify_drafts_workspace_size(3, V)
    arrays, intact = {}, []
    for name, x in (("num", torch.zeros(3, dtype=torch.int32)), ("next", torch.zeros(3, dtype=torch.int32)),
                    ("ws", torch.zeros(need, dtype=torch.uint8))):
        arrays[name], ok = guarded(x)
        intact.append(ok)
    K.kda_verify_drafts(t, d, dev(tok, torch.int32), dev(cu, torch.int32), dev(acc, torch.float32), dev(smp, torch.float32),
                        arrays["num"], arrays["next"], workspace=arrays["ws"])
    assert all(ok() for ok in intact)
    for n, (a, b) in enumerate(means):
        want = ([0], [-1])
        if b > a:
            want = check(t[a:b], d[a:b], tok[a:b], [0, b - a], acc[a:b], smp[n:n + 1])
        assert ([int(arrays["num"][n])], [int(arrays["next"][n])]) == want


@pytest.mark.parametrize("V", [4000, 40000])                  # one launch and two
def test_differences_are_rounded_once(V):
    """fp32 probabilities more than 53 binary places apart: the sign of what is left is exact, and so is a tiny remainder alone."""
    t, d = torch.zeros(2, V, device="cuda"), torch.zeros(2, V, device="cuda")
    t[0, 5], d[1, 5] = 0.5, 2.0 ** -70                        # rounds to 0.5
    t[0, V - 1], d[1, V - 1] = 2.0 ** -70, 2.0 ** -71         # left over: 2^-71
    t[0, 9], d[1, 9] = 2.0 ** -71, 2.0 ** -70                 # nothing left
    for sample, want in ((0.0, 5), (0.9999, 5)):
        assert check(t, d, [0, 9], [0, 2], [0, 0.9], [sample]) == ([1], [want])
    d[1, 5] = 0.5                                             # the remainder alone
    for sample in (0.0, 0.5, 0.99999994):
        assert check(t, d, [0, 9], [0, 2], [0, 0.9], [sample]) == ([1], [V - 1])


def test_draws_beside_a_boundary():
    """Running sums that fp64 holds exactly in any order, and marks one step of fp32 beside them, in rows of one part to 65."""
    for V in (1024, 16384, 17000, 66000):
        n = 16
        t = torch.zeros(n, V, device="cuda")
        at = torch.linspace(0, V - 1, 8).long()
        t[:, at.cuda()] = 0.125
        marks = torch.arange(n) % 8 / 8.0
        sample = torch.where(torch.arange(n) < 8, marks, torch.nextafter(marks, torch.tensor(-1.0)).clamp(min=0)).tolist()
        want = [int(at[i]) for i in range(8)] + [int(at[max(i - 1, 0)]) for i in range(8)]
        assert check(t, None, [0] * n, range(n + 1), [0.0] * n, sample)[1] == want
