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
