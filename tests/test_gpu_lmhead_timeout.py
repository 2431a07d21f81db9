"""Bounded waits of the scoring and distillation GEMMs, as
tests/test_gpu_step_timeout.py: a stage stays unfilled or one CTA of the first
pair stops, the wait expires, no copy is left in flight, and the same call right
after gives its usual bits."""
import pytest
import torch

from tests import _lmhead as R
from tests._parity import assert_device_ok
from tests.test_gpu_step_timeout import _expire

pytestmark = pytest.mark.gpu

C = pytest.importorskip("gemm_epilogue_transformer_tma_gb300")
from gemm_epilogue_transformer_tma_gb300.path import DistillHead, ScoringHead  # noqa: E402


def _same_after_a_timeout(call, mode):
    want = [t.clone() for t in call()]
    assert_device_ok()
    _expire(call, mode)
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
    assert_device_ok()


@pytest.mark.parametrize("M,mode", [(1, 1), (40, 1), (100, 1), (200, 1), (200, 2)])
@pytest.mark.parametrize("k", [0, 5])
def test_scoring(M, mode, k):
    H, W, y = R.grid_inputs(M, 192, 5000)
    head = ScoringHead(W, M, k)
    _same_after_a_timeout(lambda: [t for t in head.score(H, y) if t is not None], mode)


@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("M,d", [(200, 192), (1100, 2560)])
@pytest.mark.parametrize("grads", [False, True], ids=["loss", "gradients"])
def test_distillation(grads, M, d, mode):
    H, W, y = R.grid_inputs(M, d, 1048)
    ids = torch.stack([y, (y + 7) % 1048], 1).contiguous()
    val = torch.log(torch.tensor([0.6, 0.3], device="cuda")).expand(M, 2).contiguous()
    head = DistillHead(W, M, 2, backward=grads)
    _same_after_a_timeout(lambda: [t for t in head.step(H, ids, val) if t is not None], mode)
