"""The policy loss where its epilogues, row kernels and roundings meet their
limits: ragged vocabularies behind many tiles, NaN in weighted tokens, and the
roundings of confident policies."""
import numpy as np
import pytest
import torch

from tests._parity import assert_device_ok, assert_frob, f64
from tests.test_gpu_policy import Problem

pytestmark = pytest.mark.gpu

C = pytest.importorskip("gemm_epilogue_transformer_tma_gb300")


@pytest.mark.parametrize("V", [1816, 1864], ids=["one_block", "three_blocks"])
def test_tiles_behind_a_ragged_vocabulary(V):
    """17 x 8 tiles on fewer SM pairs: the pairs that take the last, ragged
    vocabulary tile (24 or 72 columns of a block of 128: an odd number of 32
    wide stores) go on to tiles of the next rows.  Nearly all probability lies
    in those columns, so that a stored block which another one replaced shows
    in the 32 rows it belongs to.  Bar per 32 rows: three roundings to bf16
    (kept exponential, dL, result) of 2^-8 / sqrt(3) rms each, 3.9e-3."""
    pb = Problem(4128, 64, V, seed=V)
    pb.W[1792:] *= 8
    r = pb.run(old=False, ref=False)
    assert_device_ok()
    got = f64(pb.dH).reshape(-1, 32, 64)
    ref = r["dH"].reshape(-1, 32, 64)
    err = np.linalg.norm(got - ref, axis=(1, 2)) / np.linalg.norm(ref, axis=(1, 2))
    assert err.max() <= 5e-3, err.argmax()
    assert_frob(pb.dW, r["dWt"], "dWt")
    want = (pb.dH.clone(), pb.dW.clone())
    pb.run(old=False, ref=False)
    assert torch.equal(want[0], pb.dH) and torch.equal(want[1], pb.dW)


@pytest.mark.parametrize("M", [40, 700])
@pytest.mark.parametrize("least", [False, True], ids=["kept", "least"])
@pytest.mark.parametrize("what", ["old", "old_without_advantage", "advantage", "logits", "logits_without_old"])
def test_a_nan_of_a_weighted_token_is_not_clipped(M, what, least):
    """It reaches the loss, the token's row of dH and every row of dW (its row
    of dL meets them all); the other tokens' dH keep their bits, and the KL
    statistic is NaN only where the log-probability is."""
    pb = Problem(M, 64, 264, seed=3)
    pb.least = least
    old = what != "logits_without_old"
    pb.run(old=old)
    clean = pb.dH.clone()
    t = M // 2
    if what == "advantage":
        pb.adv[t] = np.nan
    elif what.startswith("logits"):
        pb.H[t] = float("nan")
    else:
        pb.old[t] = np.nan
        pb.adv[t] = 0.0 if what == "old_without_advantage" else -0.7
    pb.run(old=old)
    assert torch.isnan(pb.stats[:2]).all()
    assert torch.isnan(pb.logp[t]).item() == torch.isnan(pb.stats[2]).item() == what.startswith("logits")
    assert torch.isfinite(pb.stats[3]).item()
    assert torch.isnan(pb.dH[t]).all() and torch.isnan(pb.dW).all()
    rest = torch.arange(M, device="cuda") != t
    assert torch.equal(pb.dH[rest], clean[rest])
    assert_device_ok()


def test_the_open_clip_and_a_finite_ratio_are_as_before():
    """r A on the border of the clip and an infinite upper bound pass the
    gradient; a token outside does not."""
    pb = Problem(30, 64, 264, seed=4)
    for kw in (dict(lo=1.0, hi=float("inf")), dict(lo=0.0, hi=0.0), dict(lo=0.2, hi=0.28, old=False)):
        pb.grade(pb.run(**kw))


def _of_one_rounding(pb, r):
    """dH's and dW's errors over that of the fp64 results rounded to bf16."""
    out = []
    for got, ref in ((pb.dH, r["dH"]), (pb.dW, r["dWt"])):
        ref = torch.from_numpy(ref)
        out.append(((got.cpu().double() - ref).norm() / (ref.to(got.dtype).double() - ref).norm()).item())
    return out


# dL's entries beside the label's are rounded to bf16 and the label's is not.
# Rounding to nearest costs the same share of every value, so with `share` of
# dL's square beside the label the error is sqrt(1 + share) of that of rounding
# the results alone.  sum p_v = 1 - p_y over the others, hence sum p_v^2 <=
# (1 - p_y)^2, the label's square: share <= 1/2.  Kept exponentials round those
# that are not their block's largest once more, half of the share where two
# tokens lead: sqrt(1 + 1/2 + 1/4) = 1.32, and 2 % for fp32 sums and for W rows
# that are not orthogonal.  On a flat softmax the label is all of dL.
ONE_ROUNDING = {0.9: 1.02, 5.0: 1.35, 8.0: 1.35}


@pytest.mark.parametrize("spread", sorted(ONE_ROUNDING))
@pytest.mark.parametrize("least", [False, True], ids=["kept", "least"])
@pytest.mark.parametrize("M", [200, 2600])
def test_rounding_of_the_gradients_by_confidence(M, least, spread):
    """Labels drawn from the softmax of logits with this spread: a flat
    policy, and mean label probabilities of 0.4 and 0.6."""
    pb = Problem(M, 128, 1000, seed=int(spread))
    g = torch.Generator().manual_seed(M)
    pb.W.copy_((torch.randn(1000, 128, generator=g) * spread / 128 ** 0.5).to(pb.W.dtype))
    L = f64(pb.H) @ f64(pb.W).T
    p = np.exp(L - L.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    u = np.random.default_rng(M).random((M, 1))
    pb.y = np.minimum((p.cumsum(1) < u).sum(1), 999).astype(np.int32)
    pb.least = least
    r = pb.run(old=False, ref=False)
    assert_device_ok()
    assert max(_of_one_rounding(pb, r)) <= ONE_ROUNDING[spread]


@pytest.mark.parametrize("least", [False, True], ids=["kept", "least"])
def test_two_tokens_of_one_half(least):
    """The label and one other token share the probability: the largest share
    beside the label that there is."""
    pb = Problem(96, 64, 520, seed=8)
    rows = torch.randn(520, 64, generator=torch.Generator().manual_seed(1)).to(pb.W.dtype).cuda()
    pb.W.copy_(rows)
    a = torch.from_numpy(pb.y.astype(np.int64)).cuda()
    pb.H.copy_((rows[a].float() + rows[(a + 7) % 520].float()).to(pb.H.dtype) * 0.5)
    pb.least = least
    r = pb.run(old=False, ref=False)
    assert_device_ok()
    assert max(_of_one_rounding(pb, r)) <= 1.35
