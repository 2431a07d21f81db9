"""The fp64 forms of tests/_lmhead.py against brute force, closed forms and
differences."""
import math

import pytest
import torch

from tests import _lmhead as R

F64 = torch.float64


def test_grid_inputs_have_exact_logits():
    H, W, _ = R.grid_inputs(40, 256, 300, device="cpu")
    L = R.logits(H, W)
    assert torch.equal((H.float() @ W.float().t()).double(), L)
    assert torch.equal(L * 2 ** 11, torch.round(L * 2 ** 11)) and L.abs().max() < 2 ** 12


def test_score_by_hand():
    H = torch.tensor([[1.0], [0.0]], dtype=torch.bfloat16)
    W = torch.tensor([[0.0], [1.0], [1.0], [-2.0]], dtype=torch.bfloat16)
    r = R.score(H, W, torch.tensor([3, -1]), T=0.5, k=3)
    p = [math.exp(z / 0.5) for z in (0, 1, 1, -2)]
    p = [x / sum(p) for x in p]
    assert abs(r["logp"][0].item() - math.log(p[3])) < 1e-14 and r["logp"][1].item() == 0
    assert abs(r["entropy"][0].item() + sum(x * math.log(x) for x in p)) < 1e-14
    assert abs(r["entropy"][1].item() - math.log(4)) < 1e-14
    assert r["ids"].tolist() == [[1, 2, 0], [0, 1, 2]]


def _case(mode, seed=0, M=5, d=4, V=12, k=5):
    g = torch.Generator().manual_seed(seed)
    H, W = torch.randn(M, d, generator=g, dtype=F64), torch.randn(V, d, generator=g, dtype=F64)
    ids = torch.stack([torch.randperm(V, generator=g)[:k] for _ in range(M)])
    ids[1, 3] = ids[1, 0]           # two entries for one token
    ids[2, 2:] = -1                 # a short list
    val = torch.log_softmax(torch.randn(M, k, generator=g, dtype=F64), 1) - 0.4
    w = torch.rand(M, generator=g, dtype=F64)
    w[3] = 0.0
    return H, W, ids, val, w


@pytest.mark.parametrize("mode", [R.LISTED, R.NORMALIZED, R.TAIL])
def test_distill_by_sums(mode):
    H, W, ids, val, w = _case(mode)
    T = 1.3
    r = R.distill(H, W, ids, val, w, mode, T)
    V = W.shape[0]
    for m in range(H.shape[0]):
        z = (W @ H[m] / T).tolist()
        lse = math.log(sum(math.exp(x) for x in z))
        t = {}
        entries = [(i, v) for i, v in zip(ids[m].tolist(), val[m].tolist()) if i >= 0]
        if mode == R.NORMALIZED:
            s = sum(math.exp(v / T) for _, v in entries)
            entries = [(i, math.log(math.exp(v / T) / s)) for i, v in entries]
        for i, v in entries:
            t[i] = t.get(i, 0.0) + math.exp(v)
        loss = sum(p * (math.log(p) - (z[i] - lse)) for i, p in t.items())
        tail = 1 - sum(t.values())
        if mode == R.TAIL:
            rest = sum(math.exp(z[i] - lse) for i in range(V) if i not in t)
            loss += tail * math.log(tail / rest)
        assert abs(r["loss"][m].item() - (loss if w[m] != 0 else 0.0)) < 1e-12


@pytest.mark.parametrize("mode", [R.LISTED, R.NORMALIZED, R.TAIL])
def test_distill_gradients_by_differences(mode):
    H, W, ids, val, w = _case(mode, 1)
    r = R.distill(H, W, ids, val, w, mode, 0.8)
    eps = 1e-6
    for X, G in ((H, r["dH"]), (W, r["dW"])):
        for i in range(X.shape[0]):
            for j in range(X.shape[1]):
                keep = X[i, j].item()
                X[i, j] = keep + eps
                up = R.distill(H, W, ids, val, w, mode, 0.8)["stats"][0].item()
                X[i, j] = keep - eps
                down = R.distill(H, W, ids, val, w, mode, 0.8)["stats"][0].item()
                X[i, j] = keep
                assert abs((up - down) / (2 * eps) - G[i, j].item()) < 1e-8


def test_a_student_like_its_teacher_has_no_loss():
    H, W, ids, _, w = _case(R.TAIL, 2)
    lq = torch.log_softmax(H @ W.t(), 1)
    ids = torch.topk(lq, 5, 1).indices
    r = R.distill(H, W, ids, lq.gather(1, ids), w, R.TAIL)
    assert r["loss"].abs().max() < 1e-14 and r["dL"].abs().max() < 1e-14
    full = torch.arange(W.shape[0]).expand(H.shape[0], -1)
    other = torch.log_softmax(torch.randn_like(lq), 1)
    r = R.distill(H, W, full, other, w, R.LISTED)   # the whole vocabulary: the KL divergence
    assert torch.allclose(r["loss"][w != 0], (other.exp() * (other - lq)).sum(1)[w != 0])
