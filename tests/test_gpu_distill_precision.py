"""What is left of distillation's gradients when the formula cancels: against
fp64 on inputs whose logits are exact in fp32 (tests/_lmhead.py)."""
import pytest
import torch

from tests import _lmhead as R
from tests._parity import assert_device_ok
from tests.test_gpu_distill import MODES, Call, make, teacher

pytestmark = pytest.mark.gpu

C = pytest.importorskip("gemm_epilogue_transformer_tma_gb300")

BF, I32 = torch.bfloat16, torch.int32


@pytest.mark.parametrize("M,d,V", [(20, 64, 264), (64, 64, 9000), (200, 64, 3000), (700, 512, 1048), (1100, 2560, 1048)])
@pytest.mark.parametrize("mode", MODES)
def test_a_row_without_entries_has_no_loss_and_no_gradient(mode, M, d, V):
    c = make(M, d, V, 4, mode)
    c.ids.fill_(-1)
    c.run()
    assert (c.loss == 0).all() and (c.dH == 0).all() and (c.dW == 0).all()
    # beside rows that have some
    c = make(M, d, V, 4, mode)
    c.ids[::2] = -1
    c.run()
    c.grade()
    assert (c.loss[::2] == 0).all() and (c.dH[::2] == 0).all()
    assert_device_ok()


def _readable(M, d, V, k, noise, seed):
    """The same k tokens for all rows, with P = Q (1 + noise).  Column 1 of the
    head is 1 off the list and 0 on it and meets a 0 in Hs, so that dHs[:, 1] is
    the sum of dL off the list; column 2 of Hs is 1 and meets 0 in the head."""
    H, W, _ = R.grid_inputs(M, d, V, sure=0.5, seed=seed)
    H = (H.float() / 4).to(BF)
    H[:, 1], H[:, 2] = 0.0, 1.0
    W[:, 1] = (torch.arange(V, device="cuda") >= k).to(BF)
    W[:, 2] = 0.0
    ids = torch.arange(k, dtype=I32, device="cuda").expand(M, k).contiguous()
    lq = torch.log_softmax(R.logits(H, W), 1)[:, :k]
    sign = torch.where(torch.arange(M, device="cuda") % 2 == 0, 1.0, -1.0)[:, None]
    val = (lq + torch.log1p(sign * noise).double()).float()
    return Call(H, W, ids, val.contiguous(), torch.full((M,), 1 / M, device="cuda"), R.TAIL)


@pytest.mark.parametrize("M,d,V", [(40, 64, 2000), (300, 64, 2000), (1100, 2560, 1048)])
@pytest.mark.parametrize("noise", [2.0 ** -13, 2.0 ** -16])
def test_the_gradient_off_the_list_of_a_student_near_its_teacher(M, d, V, noise):
    """Off the list dL = weight q (1 - r / R), and 1 - r / R = (P - Q) / R.  The
    list's exponentials and targets are good to 2^-33, and those off the list may be
    off by 2^-21 together: Q is off by 2^-21 Q R, and so is the sum of dL.  The
    gradients carry three roundings to bf16 of terms of one sign, dWt four: 2^-8
    each."""
    c = _readable(M, d, V, 8, noise, M).run()
    r = R.distill(c.H, c.W, c.ids, c.val, c.w, R.TAIL)
    q = torch.softmax(R.logits(c.H, c.W), 1)
    Q, w = q[:, :8].sum(1), c.w.double()
    assert Q.max() < 0.1
    ref = r["dH"][:, 1]
    assert (ref.abs() <= 2 * w * noise * Q).all()   # the difference that is looked at
    bar = 2.0 ** -21 * w * Q * (1 - Q) + 3 * 2.0 ** -8 * ref.abs()
    assert ((c.dH[:, 1].double() - ref).abs() <= bar).all()
    ref = r["dW"][8:, 2]
    off = r["dL"][:, 8:].abs().sum(0)
    bar = 2.0 ** -21 * (w * Q)[:, None].mul(q[:, 8:]).sum(0) + 4 * 2.0 ** -8 * off
    assert ((c.dW[8:, 2].double() - ref).abs() <= bar).all()
    assert_device_ok()


@pytest.mark.parametrize("M,d,V,k", [(1, 256, 9000, 1), (40, 512, 4096, 1), (40, 1024, 1000, 20), (64, 512, 9000, 64),
                                     (65, 512, 9000, 20), (300, 256, 4096, 1), (700, 512, 4096, 33),
                                     (1100, 2560, 1048, 1), (1100, 2560, 1048, 33)])
@pytest.mark.parametrize("mean", [0.25, 1.0])
@pytest.mark.parametrize("mode", MODES)
def test_a_head_whose_rows_share_a_mean(M, d, V, k, mean, mode):
    """5 and 20 times their spread.  A row of dL sums to 0, so the
    mean leaves dHs; it stays out of it as far as the entries keep their digits: off
    the list each is rounded by itself (half a step, 2^-8 at most and of independent
    signs), twice at most, on the list those below 2^-9 of the row's largest.
    The fp32 sum over the vocabulary may be off by 2^-23 of its parts every 16
    columns."""
    H, W, y = R.grid_inputs(M, d, V, seed=M + k)
    W = (W.float() + mean).to(BF)
    H = (H.float() / 8).to(BF)
    c = Call(H, W, *teacher(H, W, y, k, mode, 1.0, M), mode).run()
    r = c.grade(grads=False)
    dL, Wd, ref = r["dL"], W.double(), r["dH"]
    used = (c.ids >= 0) & (c.ids < V)
    on = torch.zeros_like(dL).scatter_add_(1, torch.where(used, c.ids, 0).long(), used.double()) > 0
    steep = torch.where(on, dL.abs(), 0.0).amax(1, keepdim=True)
    rounded = torch.where(on & (dL.abs() > 2.0 ** -9 * steep), 0.0, dL)
    one = (ref.to(BF).double() - ref).norm()
    bar = ((1.02 * one) ** 2 + 4 * 2.0 ** -16 * (rounded ** 2 @ Wd ** 2).sum()).sqrt()
    bar += (2.0 ** -15 + 2.0 ** -23 * V / 16) * (dL.abs() @ Wd.abs()).norm()
    assert (c.dH.double() - ref).norm() <= bar
    assert_device_ok()


@pytest.mark.parametrize("M,d,V", [(40, 64, 1000), (300, 64, 1000), (1100, 2560, 1048)])
@pytest.mark.parametrize("mode", MODES)
def test_temperatures_that_flatten_every_row(mode, M, d, V):
    """All tokens are equally probable, and columns that do not exist are not among
    them.  The gradients, 1 / T of others, are fp32 numbers at 1e30."""
    for T, grads in ((1e30, True), (3e36, False), (3e38, False)):
        make(M, d, V, 7, mode, T=T, grads=grads).run().grade()


@pytest.mark.parametrize("M,d", [(64, 64), (300, 64), (1100, 2560)])
def test_the_mass_that_a_list_leaves(M, d):
    """r = 1 - P down to 2^-29, of lists whose probabilities lie between 1e-6 and 1:
    as good as the sum of their exponentials, 2^-34.5 of P.  The student has all on
    the list, so that dL off it sums to -weight r; it is read off column 1 of dHs
    (_readable), with four roundings to bf16 of terms of one sign."""
    V, k = 1048, 40
    g = torch.Generator().manual_seed(M)
    H, W = torch.zeros(M, d), torch.zeros(V, d)
    H[:, 0], W[:k, 0], W[k:, 1] = 1.0, 100.0, 1.0
    p = torch.rand(M, k - 1, generator=g, dtype=torch.float64) ** 3 + 1e-5
    left = 2.0 ** (-29 + 6 * torch.rand(M, 1, generator=g, dtype=torch.float64))
    val = torch.log(p / p.sum(1, keepdim=True) * (1 - 1e-6)).float()
    last = torch.log(1 - left - val.double().exp().sum(1, keepdim=True)).float()
    val = torch.cat([val, last], 1).cuda()
    ids = torch.arange(k, dtype=I32, device="cuda").expand(M, k).contiguous()
    w = torch.full((M,), 1 / M, device="cuda")
    c = Call(H.to(BF).cuda(), W.to(BF).cuda(), ids, val, w, R.TAIL).run()
    r = 1 - val.double().exp().sum(1)
    assert r.min() > 2.0 ** -30 and r.max() < 2.0 ** -22
    got = -c.dH[:, 1].double() / w.double()
    assert ((got - r).abs() <= 2.0 ** -34.5 + 4 * 2.0 ** -8 * r).all()
    assert_device_ok()


@pytest.mark.parametrize("M", [24, 200])
@pytest.mark.parametrize("mode", [R.LISTED, R.TAIL])
@pytest.mark.parametrize("ratio", [1.6, 0.4])
def test_small_targets_far_from_the_student(ratio, mode, M):
    """Targets of 1e-5, q / ratio.  u = q - t is good to 2^-32 of
    t.  log(t / q) from log1p(u / t) or the quotient is off by 4 2^-24 at most, and a
    term of the loss, t (log(t / q) - 1 + q / t) >= 0.13 t, by 5 2^-24 t; with LISTED
    t log(t / q) itself, the more so.  Off the list the powers of two are off by 2^-22
    together, which the loss meets times R - r (TAIL) or times the sum of t (LISTED);
    the fp32 sums by 2^-22."""
    V, k = 60000, 40
    H, W, _ = R.grid_inputs(M, 64, V, sure=0.5, seed=M)
    H = (H.float() / 4).to(BF)
    ids = torch.randint(0, V, (M, k), generator=torch.Generator().manual_seed(5)).cuda()
    lq = torch.log_softmax(R.logits(H, W), 1).gather(1, ids)
    val = (lq - torch.log(torch.tensor(ratio, dtype=torch.float64))).float()
    c = Call(H, W, ids.to(I32), val, None, mode, grads=False).run()
    r = R.distill(H, W, c.ids, val, None, mode)
    t, q = val.double().exp().sum(1), lq.exp().sum(1)
    off = (q - t).abs() if mode == R.TAIL else t
    bar = 5 * 2.0 ** -24 * t + 2.0 ** -22 * (off + r["loss"].abs())
    assert ((c.loss.double() - r["loss"]).abs() <= bar).all()
    assert_device_ok()
