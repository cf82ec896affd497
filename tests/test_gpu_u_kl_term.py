"""The policy loss's KL term to its last digits.

Two logits alike and every other token excluded make logp = -ln 2 to FP64, whatever the
vocabulary, so the distance d to the reference is known and only e^d - d - 1 itself is
measured, down to d = 1e-6, where a difference of e^d - 1 and d would keep no digits.

Bounds, in half steps of FP32 (U).  |d| <= 1: e^d - d - 1 is d^2 / 2 times a nested product
whose factors d / n are off by 2 U and its sums by U; the nesting divides them by three and
more, so the product is off by 2.4 U, d^2 and the last product by U each, and d's own rounding
by at most 2.5 U of the term: 8 U.  e^d - 1 is d and that term: 6 U with d's rounding.
Beyond, e^d by the hardware's 2^x is off by (4 + |d|) U, and each difference by one rounding.
"""
import numpy as np
import pytest
import torch

import grad_plain as plain
import zero_sharded_mixed_shard_amd as zs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = plain.U

DISTANCES = [s * d for d in (1e-6, 4e-6, 1e-5, 3e-5, 1e-4, 1e-3, 0.01, 0.1, 0.3, 0.7, 0.99, 1.01,
                             1.5, 3.0, 10.0) for s in (1.0, -1.0)]


def exact_terms(d):
    """(e^d - d - 1, e^d - 1): the first by its series where the difference cancels."""
    n = np.arange(2, 30)
    series = (d[:, None] ** n / np.cumprod(n.astype(float))).sum(1)
    return np.where(np.abs(d) < 0.5, series, np.expm1(d) - d), np.expm1(d)


@pytest.mark.parametrize("grads", [True, False])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("vocab", [2, 300, 3000, 30_000, 60_001, 98_304, 131_072, 250_000, 280_000])
def test_the_kl_term_near_the_reference(vocab, dt, grads):
    rows = len(DISTANCES)
    z = torch.full((rows, vocab), -float("inf"), dtype=plain.TORCH[dt], device=DEV)
    a = torch.arange(rows) * 37 % vocab
    other = (a + 1 + vocab // 3) % vocab if vocab > 2 else 1 - a
    r = torch.arange(rows)
    z[r, a], z[r, other] = 0.0, 0.0
    ref = torch.tensor([-np.log(2.0) + d for d in DISTANCES], dtype=torch.float32)
    d = plain.f64(ref) + np.log(2.0)
    one, zero = torch.ones(rows, device=DEV), torch.zeros(rows, device=DEV)
    loss, token, logp = torch.empty(1, device=DEV), torch.empty_like(one), torch.empty_like(one)
    dz = torch.empty_like(z) if grads else None
    zs.zero_policy_loss(loss, token, logp, z, a.to(DEV), zero, one, ref_logp=ref.to(DEV),
                        clip_low=0.2, clip_high=0.2, kl_coef=1.0, loss_scale=1.0, dlogits=dz)
    term, em = exact_terms(d)
    near = np.abs(d) <= 1
    far = (np.exp(d) * (4 + np.abs(d)) + np.abs(em) * (1 + np.abs(d)) + term) * U * 1.01
    err = np.abs(plain.f64(token) - term)
    worst = err / np.where(near, 8 * U * term, far)
    assert np.all(worst <= 1), list(zip(d, worst))
    assert bool((token >= 0).all())
    tol = np.where(near, 8 * U * term, far).sum() + term.sum() * U
    assert abs(float(loss) - term.sum()) <= tol
    if not grads:
        return
    g = -em / 2                         # the target's; the other logit's is its negative
    tol = plain.rounded(g, np.where(near, 6 * U * np.abs(em), far) / 2, dt)
    assert np.all(np.abs(plain.f64(dz[r, a]) - g) <= tol)
    assert torch.equal(dz[r, other], -dz[r, a])
