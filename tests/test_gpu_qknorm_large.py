"""kda_qknorm and kda_qknorm_backward where a workgroup walks several tiles of tokens,
and several rounds of heads in one, against the norm and rotation in fp64
(tests/cache_ref.py)."""
import pytest
import torch

from gated_delta_rule_40_amd import libkda as K
from test_gpu_qknorm import check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    K.load()


# With weights 512 workgroups take a gradient's tiles.  bf16, 64 values a head, four lanes: tiles of two tokens of 64 heads
# (1,301, the last of one token) and of four of 33 (651; 132 heads in rounds of 128); fp32, eight lanes: of one token, and of
# two of 33 (66 heads in rounds of 64).
@pytest.mark.parametrize("dtype,interleaved", [("bf16", False), ("bf16", True), ("fp32", False)])
def test_more_tiles_than_workgroups(dtype, interleaved):
    check(make(2601, 64, 33, 64, 64, axes=3, dtype=dtype, grad="fp32", shuffled=True), norm="rms", interleaved=interleaved)


def test_more_tiles_than_workgroups_without_a_rotation():
    check(make(2601, 64, 33, 64, 0))


# heads of 16 and 64 lanes: 16 and 4 at a time, by twos or fours, of 70 and 69
@pytest.mark.parametrize("d,dtype,rot", [(256, "bf16", 256), (256, "bf16", 0), (512, "fp32", 64), (512, "fp32", 0),
                                         (512, "bf16", 512), (200, "fp32", 100)])
def test_more_heads_than_a_round(d, dtype, rot):
    check(make(37, 70, 69, d, rot, axes=2, dtype=dtype, grad="fp32", shuffled=True))


# tiles as long as leaves 256 workgroups, between one round of heads and the rounds read at once: 97 tokens of 64 to 256 for one
# head, 31 of 22 to 86 for three; and the longest, 128, in 547 tiles
@pytest.mark.parametrize("T,Hq,Hk", [(25001, 1, 1), (8003, 3, 1), (70001, 1, 0)], ids=str)
def test_tiles_by_the_number_of_tokens(T, Hq, Hk):
    check(make(T, Hq, Hk, 64, 64, axes=2, grad="fp32", shuffled=True))


def test_a_tile_s_turns_are_its_own():
    """Tokens far apart in position, in every tile and round: outputs and gradients of a call are those of its halves."""
    p = make(2601, 64, 33, 64, 64, axes=3, grad="fp32", shuffled=True)
    form = dict(eps=1e-5, q_scale=0.25, inv_freq=p["turn"]["inv_freq"], pair_axis=p["turn"]["pair_axis"])
    pos = p["turn"]["positions"]
    whole, parts = [], []
    for at, into in ((slice(0, 2601), whole), (slice(0, 1000), parts), (slice(1000, 2601), parts)):
        q, k, dq, dk = (p[n][at] for n in ("q", "k", "dq", "dk"))
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        K.kda_qknorm(q, k, qo, ko, positions=pos[:, at].contiguous(), **form)
        g = K.kda_qknorm_backward(q, k, dq, dk, positions=pos[:, at].contiguous(), **form)
        into.append((qo, ko, g["dq"], g["dk"]))
    for a, b in zip(whole[0], map(torch.cat, zip(*parts))):
        assert torch.equal(a, b)


# the last piece of a part lies over the one before, in the same wave
@pytest.mark.parametrize("d,rot,dtype", [(77, 0, "fp32"), (77, 20, "bf16"), (100, 50, "bf16"), (129, 2, "fp32"), (511, 0, "fp32"),
                                         (13, 6, "bf16")])
def test_in_place_where_pieces_overlap(d, rot, dtype):
    p = make(41, 9, 6, d, rot, dtype=dtype, grad="fp32")
    qo, ko, g = check(p)
    form = dict(q_weight=p["qw"], k_weight=p["kw"], eps=1e-5, q_scale=0.25, **p["turn"])
    q, k = p["q"].clone(), p["k"].clone()
    K.kda_qknorm(q, k, q, k, **form)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    q, k = p["q"].clone(), p["k"].clone()
    K.kda_qknorm_backward(q, k, p["dq"], p["dk"], grads=dict(g, dq=q, dk=k), **form)
    assert torch.equal(q, g["dq"]) and torch.equal(k, g["dk"])
