"""Copies in flight when a bounded wait gives up: a kernel returns only after
they have landed.  As tests/test_gpu_step_timeout.py, at the sizes where the
producer itself never waits."""
import pytest
import torch

from tests._parity import assert_device_ok
from tests.test_gpu_step_timeout import _expire

pytestmark = pytest.mark.gpu

C = pytest.importorskip("gemm_epilogue_transformer_tma_gb300")
from gemm_epilogue_transformer_tma_gb300.path import BlockScaledLinear  # noqa: E402

BF = torch.bfloat16


@pytest.mark.parametrize("M,N,K", [(1, 128, 128), (1, 128, 512), (20, 256, 2048), (60, 6144, 2048), (100, 2048, 2048),
                                   (128, 136, 640)],
                         ids=["one_block", "one_range", "few32", "few64", "few128", "few128_ragged"])
def test_no_more_k_blocks_than_stages(M, N, K):
    """The ranges of K (1 to 4 blocks of 128) fit the ring: the producer of
    the first CTA ends well although its first stage was never filled."""
    g = torch.Generator(device="cuda").manual_seed(M + K)
    lin = BlockScaledLinear(torch.randn(N, K, device="cuda", generator=g).to(BF), M, backward=False)
    x = torch.randn(M, K, device="cuda", generator=g).to(BF)
    want = lin.forward(x).clone()
    assert_device_ok()
    for _ in range(2):
        _expire(lambda: lin.forward(x), 1)
        assert torch.equal(lin.forward(x), want)
        assert_device_ok()
