"""The gradients of a whole post-training step against fp64 without any 8-bit
codes, with every token's side of the clip settled by its data."""
import numpy as np
import pytest
import torch

from oracle import step_oracle as S
from tests._parity import assert_device_ok, f64, frob_err
from tests.test_gpu_step import D, NK, NQ, Step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [63, 300, 777])
def test_gradients_end_to_end(M):
    """The sampling log-probabilities put each token's ratio at 1 (unclipped)
    or at e^0.6 or e^-0.6 (0.35 past the borders of 0.8 and 1.28 in the
    logarithm): the codes' error of a log-probability, below 0.2 here, decides
    for no token, so dX and dW are compared at every size.

    Error, rms: e4m3 rounds to at most 2^-4 / sqrt(3) = 3.6 %, e5m2 to 7.2 %.
    qkv, from two e4m3 operands, 5.1 %, enters dqkv through the norm and,
    through H, through r and the softmax; dX then takes the gradient's and the
    weight's codes, dW the gradient's and the input's: 5.1 twice, 7.2 and 3.6 in
    quadrature make 11 %, the bar is 20 %."""
    s = Step(M, seed=M)
    x, w, gq, gk = f64(s.X), f64(s.W), f64(s.gq), f64(s.gk)
    e = x @ w.T
    eo = S.qknorm_rope(e, gq, gk, s.pos, NQ, NK, D, 1e-6)
    head = (eo[:, :NQ * D], f64(s.Wt), s.y, s.adv, s.w)
    lp = S.policy_loss(*head, None, None, 0.2, 0.28, 0.0, 0.9)["logp"]
    s.old = (lp - np.random.default_rng(M).choice([-0.6, 0.0, 0.6], M)).astype(np.float32)
    s.dev[4].copy_(torch.from_numpy(s.old))
    er = S.policy_loss(*head, s.old, None, 0.2, 0.28, 0.0, 0.9)
    s.run()
    assert_device_ok()
    assert np.abs(f64(s.logp) - er["logp"]).max() < 0.2
    # the same tokens carry a gradient, clipped ones among them
    got = np.abs(f64(s.dout)).sum(1) != 0
    assert (got == (er["g"] != 0)).all() and 0 < got.sum() < (s.w != 0).sum()
    ed = np.concatenate([er["dH"], np.zeros((M, 2 * NK * D))], 1)
    eg, _, _ = S.qknorm_rope_backward(e, ed, gq, gk, s.pos, NQ, NK, D, 1e-6)
    assert frob_err(s.dX, eg @ w) < 0.2
    assert frob_err(s.dW, eg.T @ x) < 0.2
