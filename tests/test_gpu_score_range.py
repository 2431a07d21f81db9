"""Scoring at the ends of what it accepts.  Tolerances as tests/test_gpu_score.py."""
import pytest
import torch

from tests import _lmhead as R
from tests._parity import assert_device_ok
from tests.test_gpu_score import Call

pytestmark = pytest.mark.gpu

C = pytest.importorskip("gemm_epilogue_transformer_tma_gb300")


@pytest.mark.parametrize("T", [1e30, 3e36, 1e38, 3e38])
@pytest.mark.parametrize("M,V", [(1, 8), (3, 1000), (33, 32000), (64, 50280), (100, 264), (200, 1000), (300, 2056)])
@pytest.mark.parametrize("k", [0, 5])
def test_temperatures_that_flatten_every_row(M, V, T, k):
    """All V tokens are equally probable, and columns that do not exist, in the
    last block of a row or beside a narrow one, are not among them."""
    H, W, y = R.grid_inputs(M, 64, V, seed=M)
    c = Call(H, W, y, T, k).run()
    c.grade()
    assert ((c.entropy - torch.log(torch.tensor(float(V)))).abs() <= 2.0 ** -16 * 12).all()


@pytest.mark.parametrize("M,V,k", [(3, 1000, 5), (64, 4096, 0), (200, 1000, 5), (300, 5000, 0), (4100, 20000, 8)])
@pytest.mark.parametrize("sign", [-1.0, 1.0], ids=["minus", "plus"])
def test_an_infinite_logit(M, V, k, sign):
    """Of one token in every row: its log-probabilities and entropy are NaN, the
    others keep their ranks."""
    H, W, y = R.grid_inputs(M, 64, V, seed=5)
    H[:, 0], W[:, 0] = 1.0, 0.0
    a = Call(H, W, y, 1.0, k).run()
    W2, v = W.clone(), V // 2
    W2[v, 0] = sign * float("inf")
    c = Call(H, W2, y, 1.0, k).run()
    for t in (c.logp, c.entropy) + ((c.top,) if k else ()):
        assert torch.isnan(t).all()
    if k:
        for m in range(0, M, max(1, M // 7)):
            others = [i for i in a.ids[m].tolist() if i != v]
            want = [v] + others if sign > 0 else others
            n = min(k, len(want))
            assert c.ids[m, :n].tolist() == want[:n]
    assert_device_ok()


@pytest.mark.parametrize("M,V,k", [(1, 1000, 20), (40, 9000, 256), (200, 1000, 20), (300, 50280, 64), (4100, 20000, 8)])
def test_logits_within_2_to_the_minus_122(M, V, k):
    """Their range has no finite reciprocal; each token keeps its rank."""
    H, W, y = R.grid_inputs(M, 64, V, seed=6)
    H.zero_()
    W.zero_()
    H[:, 0] = 2.0 ** -60
    mix = torch.randint(0, 128, (V,), generator=torch.Generator().manual_seed(3)).cuda()
    W[:, 0] = ((1 + mix / 128.0) * 2.0 ** -62).to(W.dtype)
    H[1::3] = 0
    c = Call(H, W, y, 1.0, k).run()
    for rows in (slice(0, 50), slice(M - min(M, 50), M)):
        c.grade(rows)
