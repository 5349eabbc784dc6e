"""Many steps of 8-bit states on the GPU: the kernel's states after some hundred
steps are those of the oracle's chain of 32-bit steps bit for bit, and its
weights those of that chain in 64 bits."""
import types

import numpy as np
import pytest

import oracle.adamw_mixed_oracle as ao
from test_adamw_mixed_long_cpu import SEED, run_codes, stopping

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rounding", ["stochastic", "nearest"])
@pytest.mark.parametrize("beta1, beta2", [(0.9, 0.95), (0.9, 0.999)])
def test_states_after_many_steps(beta1, beta2, rounding):
    """Gradients stop in part of a block.  Stochastically rounded first moments
    have reached zero there and their weights rest; nearest ones have not.
    Bound on p: per step 4 |p| + 21 |change| half steps, as for single steps
    (moments and gradients have one sign here, so that the sum of their
    magnitudes is the new moment); errors of p do not enter the moments."""
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    lr, stop, steps, dead = 1e-3, 50, 700, 16
    grads = stopping(0.03, stop, dead)
    p, g = torch.zeros(ao.BLOCK, device="cuda"), torch.from_numpy(grads(1)).cuda()
    s = B.Adam8State.zeros(ao.BLOCK)
    count = torch.zeros(2, dtype=torch.int32, device="cuda")
    h = types.SimpleNamespace(lr=lr, beta1=beta1, beta2=beta2, eps=1e-8, weight_decay=0.0)
    run = B.adamw_mixed_bind([p], [g], [s], h, step_dev=count, rounding=rounding, seed=SEED)
    late = None
    for t in range(1, steps + 1):
        if t == stop + 1:
            g.copy_(torch.from_numpy(grads(t)))
        run()
        if t == steps - 100:
            late = p.clone()
    torch.cuda.synchronize()
    assert count.tolist() == [steps, 0]
    old, tol = np.zeros(ao.BLOCK), np.zeros(ao.BLOCK)
    for t, want, mc, r in run_codes(grads, beta1, beta2, rounding, lr):
        tol += 1.01 * 2.0 ** -24 * (4 * np.abs(old) + 21 * np.abs(want - old))
        old = want
        if t == steps:
            break
    assert np.array_equal(s.exp_avg.cpu().numpy(), mc)
    byte = s.scale.cpu().numpy()[1:]
    assert np.array_equal(ao.decode(s.root.cpu().numpy(), byte, ao.R_BITS), r)
    assert np.all(np.abs(p.cpu().numpy() - want) <= tol)
    moved = bool((p[:dead] != late[:dead]).any())
    assert moved == (rounding == "nearest") and bool((s.exp_avg[:dead] != 0).any()) == moved
