"""The policy loss's values for unusual arguments, against the 64-bit definition."""
import numpy as np
import pytest
import torch

import grad_plain as plain
import zero_sharded_mixed_shard_amd as zs
from test_gpu_r_policy import inputs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = plain.U


@pytest.mark.parametrize("vocab", [50, 20_000, 270_000])
@pytest.mark.parametrize("lo,hi,kl", [(1.0, float("inf"), 0.1), (0.0, 0.0, -0.2), (0.0, 0.0, 0.0),
                                      (1.0, 0.0, 0.3), (0.2, float("inf"), 0.0)])
def test_losses_of_unusual_arguments(vocab, lo, hi, kl):
    # no upper cut, a full or no lower one, a negative KL weight, negative weights and
    # advantages of both signs: every row's loss, the total and the log-probabilities
    z, a, old, ref, adv, w = inputs(12, vocab, "f32", 15, masked=False)
    adv[::2] = -adv[::2].abs()
    adv[1::2] = adv[1::2].abs()
    w[2], w[5] = -w[2], -w[5]
    got = [torch.empty(1, device=DEV), torch.empty(12, device=DEV), torch.empty(12, device=DEV)]
    zs.zero_policy_loss(*got, z.to(DEV), a.to(DEV), adv.to(DEV), w.to(DEV), old_logp=old.to(DEV),
                        ref_logp=ref.to(DEV), clip_low=lo, clip_high=hi, kl_coef=kl,
                        loss_scale=2.0)
    n = lambda t: t.double().numpy()
    args = (n(z), a.numpy(), n(old), n(ref), n(adv), n(w), lo, hi)
    ex = plain.policy(*args, kl, 2.0)
    by_size = plain.policy(*args, abs(kl), 2.0)      # the bounds count kl by its magnitude
    tol = by_size["b_token"] + (np.abs(ex["token_loss"]) + np.abs(by_size["token_loss"])) * 4 * U
    assert np.all(np.abs(plain.f64(got[1]) - ex["token_loss"]) <= tol)
    assert np.all(np.abs(plain.f64(got[2]) - ex["logp"]) <= ex["b_logp"] + np.abs(ex["logp"]) * U)
    assert abs(float(got[0]) - ex["loss"]) <= (tol * np.abs(n(w))).sum() + abs(ex["loss"]) * 2 * U
    # the cuts take part on both sides, and the KL term is part of it
    r = np.exp(ex["logp"] - n(old))
    if hi == 0.0:
        assert ((n(adv) > 0) & (r > 1)).any()
    if lo == 0.0:
        assert ((n(adv) < 0) & (r < 1)).any()
    if kl != 0:
        without = plain.policy(*args, 0.0, 2.0)["token_loss"]
        assert (np.abs(ex["token_loss"] - without) > 4 * tol).sum() >= 6
