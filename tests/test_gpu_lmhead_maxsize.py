"""Scoring and distillation past the sizes at which their kernels change how
they go through a row: vocabularies of more blocks than a thread holds or a list
sort counts at a time, rows x vocabulary past 2^31 values."""
import pytest
import torch

from tests import _lmhead as R
from tests._parity import assert_device_ok, assert_frob
from tests.test_gpu_distill import Call as Distill
from tests.test_gpu_distill import teacher
from tests.test_gpu_score import Call as Score

pytestmark = pytest.mark.gpu

C = pytest.importorskip("gemm_epilogue_transformer_tma_gb300")


@pytest.mark.parametrize("M", [3, 70])
@pytest.mark.parametrize("V,k", [(147456, 7), (160000, 100), (1048576, 20)])
def test_scoring_over_wide_vocabularies(M, V, k):
    H, W, y = R.grid_inputs(M, 16, V, seed=V % 97)
    Score(H, W, y, 1.0, k).run().grade()
    H[0] = 0
    Score(H, W, y, 1.0, k).run().grade()


@pytest.mark.parametrize("M,V", [(40, 524416), (70, 1048584)])
def test_distillation_over_wide_vocabularies(M, V):
    H, W, y = R.grid_inputs(M, 16, V, seed=3)
    Distill(H, W, *teacher(H, W, y, 40, R.TAIL, 1.0, 3), R.TAIL).run().grade()


def test_a_list_in_one_block():
    """All entries of 32 rows in the same 128 columns, every token of them
    twice: the fullest bucket a list sort can have."""
    M, V, k = 64, 5000, 256
    H, W, _ = R.grid_inputs(M, 64, V, seed=8)
    ids = torch.arange(k, device="cuda").remainder(128).add(1280).to(torch.int32).expand(M, k).contiguous()
    val = torch.log_softmax(torch.randn(M, k, generator=torch.Generator().manual_seed(0)), 1).cuda() - 0.2
    w = torch.full((M,), 1 / M, device="cuda")
    for mode in (R.LISTED, R.NORMALIZED, R.TAIL):
        c = Distill(H, W, ids, val.contiguous(), w, mode).run()
        c.grade()
        first = [t.clone() for t in c.outputs()]
        c.run()
        assert all(torch.equal(a, b) for a, b in zip(first, c.outputs()))


def test_kept_values_past_2_31():
    M, d, V, k = 20000, 16, 131072, 4
    H, W, y = R.grid_inputs(M, d, V, seed=2)
    g = torch.Generator().manual_seed(1)
    ids = torch.randint(0, V, (M, k), generator=g).to(torch.int32)
    ids[:, 0] = y.cpu()
    val = torch.log(torch.tensor([0.5, 0.2, 0.1, 0.05])).expand(M, k)
    w = (torch.rand(M, generator=g) + 0.5) / M
    ids, val, w = ids.cuda(), val.contiguous().cuda(), w.cuda()
    assert M * V > 2 ** 31
    c = Distill(H, W, ids, val, w, R.TAIL).run()
    dW = torch.zeros(V, d, dtype=torch.float64, device="cuda")
    for m in range(0, M, 500):
        s = slice(m, m + 500)
        r = R.distill(H[s], W, ids[s], val[s], w[s], R.TAIL)
        dW += r["dW"]
        assert ((c.loss[s].double() - r["loss"]).abs() <= 2.0 ** -15 * (1 + r["loss"])).all()
        if m % 5000 == 0 or m + 500 == M:
            assert_frob(c.dH[s], r["dH"].cpu().numpy(), f"dH {m}")
    assert_frob(c.dW, dW.cpu().numpy(), "dWt")
    assert_device_ok()
    del c, dW
    torch.cuda.empty_cache()


def test_scored_rows_past_2_31():
    """More logits than a workspace holds at once, and more than 2^31: row
    chunks of 4096."""
    M, V = 20000, 131072
    H, W, y = R.grid_inputs(M, 16, V, seed=4)
    c = Score(H, W, y, 1.0, 2).run()
    for m in (0, 4090, 16380, 19990):
        c.grade(slice(m, m + 10))
