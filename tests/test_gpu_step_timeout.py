"""Bounded waits of the block-scaled GEMMs and of the policy loss's GEMMs, as
tests/test_gpu_timeout.py: the hook leaves a stage unfilled or stops one CTA
of the first pair, the wait expires, no copy is left in flight, and the same
call right after gives its usual bits."""
import pytest
import torch

from tests._parity import assert_device_ok

pytestmark = pytest.mark.gpu

C = pytest.importorskip("gemm_epilogue_transformer_tma_gb300")
from gemm_epilogue_transformer_tma_gb300.path import BlockScaledLinear, PolicyHead  # noqa: E402

BF = torch.bfloat16
TIMEOUT_BITS, DRAIN_BIT = 0x1 | 0x2 | 0x4, 0x8


def _expire(call, mode):
    C.coda_set_wait_timeout_ns(50_000_000)  # 50 ms
    C.coda_debug_skip_first_stage(mode)
    try:
        call()
        st, bits = C.coda_sync_status()
    finally:
        C.coda_debug_skip_first_stage(0)
        C.coda_set_wait_timeout_ns(0)
    assert st == 6, f"expected CODA_ERR_TIMEOUT, got {C.STATUS_NAMES.get(st)} bits={bits:#x}"
    assert bits & TIMEOUT_BITS, f"a bounded wait should have expired (bits={bits:#x})"
    assert not bits & DRAIN_BIT, f"in-flight copies did not drain (bits={bits:#x})"


@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("M,N,K", [(8, 512, 4096), (64, 256, 1024), (3000, 4608, 1664), (1536, 2816, 4608)],
                         ids=["few_split", "few", "pairs", "pairs_split"])
def test_block_scaled_gemm(M, N, K, mode):
    g = torch.Generator(device="cuda").manual_seed(M)
    lin = BlockScaledLinear(torch.randn(N, K, device="cuda", generator=g).to(BF), M, backward=False)
    x = torch.randn(M, K, device="cuda", generator=g).to(BF)
    want = lin.forward(x).clone()
    assert_device_ok()
    _expire(lambda: lin.forward(x), mode)
    assert torch.equal(lin.forward(x), want)
    assert_device_ok()


@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("grads", [False, True], ids=["logits", "gradients"])
def test_policy_head(grads, mode):
    g = torch.Generator(device="cuda").manual_seed(5)
    M, d, V = 200, 192, 4096
    head = PolicyHead((torch.randn(V, d, device="cuda", generator=g) * 0.05).to(BF), M, backward=grads)
    h = torch.randn(M, d, device="cuda", generator=g).to(BF)
    y = torch.randint(0, V, (M,), device="cuda", generator=g, dtype=torch.int64).to(torch.int32)
    adv = torch.randn(M, device="cuda", generator=g)

    def call():
        return [t for t in head.step(h, y, adv) if t is not None]

    want = [t.clone() for t in call()]
    assert_device_ok()
    _expire(call, mode)
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
    assert_device_ok()
