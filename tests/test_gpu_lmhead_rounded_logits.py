"""Scoring and distillation on logits that round, against fp64.

The logits' error.  An MMA takes 16 of K: its products and the running sum are
aligned to the largest and cut no earlier than behind 24 bits, so that each of 17
terms loses 2^-23 of the largest at most.  The running sum starts at 0 every 512 of
K, and the pieces are added with 2^-24 of their sum each.  cut() adds that up for
every logit.  With e its result, a log-sum-exp is off by sum p e / T at most, the
entropy by sum p |log p + entropy| e / T, distillation's loss by sum |d loss / d z|
e / T (to first order: e is below 2^-9), beside what the other tests of the two
allow."""
import pytest
import torch

from tests import _lmhead as R
from tests._parity import assert_device_ok, assert_frob
from tests.test_gpu_distill import MODES, teacher
from tests.test_gpu_distill import Call as Distill
from tests.test_gpu_score import REL
from tests.test_gpu_score import Call as Score

pytestmark = pytest.mark.gpu

C = pytest.importorskip("gemm_epilogue_transformer_tma_gb300")

BF, F64, I32 = torch.bfloat16, torch.float64, torch.int32


def inputs(M, d, V, seed):
    g = torch.Generator().manual_seed(seed)
    W = torch.randn(V, d, generator=g) * 0.05
    y = torch.randint(0, V, (M,), generator=g)
    lean = torch.rand(M, 1, generator=g) * (10 / (0.0025 * d))
    H = torch.randn(M, d, generator=g) * 0.5 + lean * W[y]
    return H.to(BF).cuda(), W.to(BF).cuda(), y.to(I32).cuda()


def cut(H, W):
    H, W = H.to(F64), W.to(F64)
    e = torch.zeros(H.shape[0], W.shape[0], dtype=F64, device=H.device)
    run, total = torch.zeros_like(e), torch.zeros_like(e)
    for k in range(0, H.shape[1], 16):
        if k % 512 == 0:
            total += run
            e += 2.0 ** -24 * total.abs()
            run.zero_()
        h, w = H[:, k:k + 16], W[:, k:k + 16]
        step = h @ w.t()
        top = torch.maximum(run.abs(), (run + step).abs())
        top = torch.maximum(top, h.abs() @ w.abs().t())
        run += step
        e += 17 * 2.0 ** -23 * top
    return e + 2.0 ** -24 * (total + run).abs()


@pytest.mark.parametrize("M,d,V,k,T", [(3, 4096, 5000, 20, 1.0), (50, 1000, 9000, 64, 0.7), (200, 2048, 5000, 256, 1.0),
                                       (136, 520, 33000, 0, 2.0), (4100, 264, 20000, 8, 1.0)])
def test_scoring(M, d, V, k, T):
    H, W, y = inputs(M, d, V, M)
    c = Score(H, W, y, T, k).run()
    for rows in (slice(0, 64), slice(M - min(M, 64), M)):
        L, e = R.logits(H[rows], W), cut(H[rows], W)
        assert e.max() < 2.0 ** -9
        r = R.score(H[rows], W, y[rows], T, 0)
        lq = torch.log_softmax(L / T, 1)
        p = lq.exp()
        lse = (p * e).sum(1) / T
        at = y[rows].long()[:, None]
        assert ((c.logp[rows].double() - r["logp"]).abs() <= e.gather(1, at)[:, 0] / T + lse + REL * r["logp"].abs()).all()
        ent = r["entropy"]
        bar = (p * (lq + ent[:, None]).abs() * e).sum(1) / T
        assert ((c.entropy[rows].double() - ent).abs() <= 1.01 * bar + REL * ent).all()
        if k == 0:
            continue
        ids = c.ids[rows].long()
        assert ids.min() >= 0 and ids.max() < V and (torch.sort(ids, 1).values.diff(dim=1) > 0).all()
        top, top_e = L.gather(1, ids), e.gather(1, ids)
        want = lq.gather(1, ids)
        assert ((c.top[rows].double() - want).abs() <= top_e / T + lse[:, None] + REL * want.abs()).all()
        # ranks hold but for logits closer than their errors
        assert (top[:, 1:] - top[:, :-1] <= top_e[:, 1:] + top_e[:, :-1]).all()
        left = (L - e).scatter(1, ids, -torch.inf).amax(1)
        assert (left <= (top + top_e).amin(1)).all()
    assert_device_ok()


@pytest.mark.parametrize("M,d,V,k", [(7, 4096, 5000, 20), (64, 1000, 9000, 5), (200, 2048, 3000, 64),
                                     (1100, 2560, 1048, 33)])
@pytest.mark.parametrize("mode", MODES)
def test_distillation(mode, M, d, V, k):
    H, W, y = inputs(M, d, V, M)
    c = Distill(H, W, *teacher(H, W, y, k, mode, 1.0, M), mode).run()
    r, e = R.distill(H, W, c.ids, c.val, c.w, mode), cut(H, W)
    live = c.w != 0
    slope = torch.where(live[:, None], r["dL"] / c.w.double()[:, None], 0.0).abs()
    one = torch.ones_like(r["loss"])
    used = (c.ids >= 0) & (c.ids < V)
    mass = one * 2 if mode != R.LISTED else torch.where(used, c.val.double().exp(), 0.0).sum(1) + 1
    bar = 1.01 * (slope * e).sum(1) + 2.0 ** -17 * (mass + 1) + 2.0 ** -19 * r["loss"].abs()
    assert ((c.loss.double() - r["loss"]).abs() <= bar).all()
    assert_frob(c.dH, r["dH"].cpu().numpy(), "dH")
    assert_frob(c.dW, r["dW"].cpu().numpy(), "dWt")
    assert_device_ok()


@pytest.mark.parametrize("M", [40, 256])
def test_a_logit_summed_in_pieces(M):
    """A token whose logit, -20, grows evenly over K = 2048.  Each 16 of K cost the
    running sum half a unit of its last place on average, 2^-24.5 of it: of four
    pieces 16.5 2^-24.5 |z| in the mean, of one sum 64.5 times; the bar lies half
    way between the two (2^-19.5).  The rest of the row's log-sum-exp is near 0."""
    d, V = 2048, 1000
    g = torch.Generator().manual_seed(M)
    H = (1 + 0.1 * torch.randn(M, d, generator=g)).to(BF).cuda()
    W = (0.001 * torch.randn(V, d, generator=g))
    W[500] = -20 / d * (1 + 0.1 * torch.randn(d, generator=g))
    W = W.to(BF).cuda()
    y = torch.full((M,), 500, dtype=I32, device="cuda")
    c = Score(H, W, y).run()
    r = R.score(H, W, y)
    z = R.logits(H, W)[:, 500].abs().mean()
    bar = 2.0 ** -19.5 * z + 2.0 ** -22 * r["logp"].abs().mean()
    assert (c.logp.double() - r["logp"]).mean().abs() <= bar
    s = Distill(H, W, y[:, None].contiguous(), torch.zeros(M, 1, device="cuda"), None, R.LISTED, grads=False).run()
    assert (s.loss.double() + r["logp"]).mean().abs() <= bar
    assert_device_ok()
