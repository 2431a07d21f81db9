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


@pytest.mark.parametrize("M,nq,nk,D", [(5000, 32, 8, 128), (777, 6, 3, 80), (3, 2, 1, 64)])
def test_head_norm_backward_with_the_least_wait_limit(M, nq, nk, D):
    """A limit of 1 ns: every wait either meets its copies or reports that it
    gave up, and the call after has its usual bits."""
    g = torch.Generator(device="cuda").manual_seed(M)
    width = (nq + 2 * nk) * D
    qkv, dout = (torch.randn(M, width, device="cuda", generator=g).to(BF) for _ in range(2))
    gain = torch.ones(D, dtype=BF, device="cuda")
    cos, sin = torch.empty(1000, D // 2, device="cuda"), torch.empty(1000, D // 2, device="cuda")
    C.coda_rope_table(cos, sin)
    ws = torch.empty(C.coda_qknorm_rope_bwd_workspace_bytes(M, D), dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(qkv), torch.empty(D, device="cuda"), torch.empty(D, device="cuda")]

    def call():
        C.coda_qknorm_rope_bwd(dout, qkv, gain, gain, cos, sin, *out, ws, nq, nk, D)
        return [t.clone() for t in out]

    want = call()
    assert_device_ok()
    C.coda_set_wait_timeout_ns(1)
    try:
        for _ in range(10):
            got = call()
            st, bits = C.coda_sync_status()
            assert st in (0, 6), bits
            assert st == 6 or all(torch.equal(a, b) for a, b in zip(got, want))
    finally:
        C.coda_set_wait_timeout_ns(0)
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
    assert_device_ok()


@pytest.mark.parametrize("M,N,K", [(128, 256, 64), (130, 264, 256), (700, 1032, 136)])
def test_one_sm_gemm_with_no_more_k_blocks_than_stages(M, N, K):
    """The one-SM form of the bf16 GEMMs (4 stages of 64 of K), as above."""
    g = torch.Generator(device="cuda").manual_seed(K)
    a, b = (torch.randn(r, K, device="cuda", generator=g).to(BF) for r in (M, N))
    out = torch.empty(M, N, dtype=BF, device="cuda")

    def call():
        C.coda_gemm(a, False, b, False, out, M, N, K)
        return out

    C.coda_set_sm_pairing(False)
    try:
        want = call().clone()
        assert_device_ok()
        for _ in range(2):
            _expire(call, 1)
            assert torch.equal(call(), want)
            assert_device_ok()
    finally:
        C.coda_set_sm_pairing(True)
