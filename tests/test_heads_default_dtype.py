"""The heads' buffers are what the entry points take, whatever torch's default dtype is."""
import pytest
import torch

C = pytest.importorskip("gemm_epilogue_transformer_tma_gb300")
from gemm_epilogue_transformer_tma_gb300.path import DistillHead, PolicyHead, QKVProjection, ScoringHead  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(params=[torch.float64, torch.bfloat16], ids=str)
def default_dtype(request):
    keep = torch.get_default_dtype()
    torch.set_default_dtype(request.param)
    yield
    torch.set_default_dtype(keep)


def test_lm_heads(default_dtype):
    W = torch.zeros(136, 64, dtype=BF)
    s, d, p = ScoringHead(W, 8, 3), DistillHead(W, 8, 3), PolicyHead(W, 8)
    for t in (s.logp, s.entropy, s.top_logp, d.stats, d.row_loss, p.stats, p.logp):
        assert t.dtype is F32
    assert s.top_ids.dtype is torch.int32 and d.dH.dtype is d.dWt.dtype is p.dH.dtype is BF


@pytest.mark.gpu
def test_calls(default_dtype):
    H, W = (torch.zeros(n, 64, dtype=BF, device="cuda") for n in (8, 136))
    y = torch.zeros(8, dtype=torch.int32, device="cuda")
    _, _, ids, top = ScoringHead(W, 8, 3).score(H, y)
    DistillHead(W, 8, 3).step(H, ids, top)
    PolicyHead(W, 8).step(H, y, torch.ones(8, dtype=F32, device="cuda"))
    g = torch.ones(64, dtype=BF, device="cuda")
    q = QKVProjection(torch.zeros(256, 128, dtype=BF, device="cuda"), g, g, 2, 1, 8, 16)
    q.backward(q.forward(torch.zeros(8, 128, dtype=BF, device="cuda")))
    assert torch.equal(q.cos_t[0], torch.ones(32, dtype=F32, device="cuda"))
    assert C.coda_sync_status()[0] == 0
