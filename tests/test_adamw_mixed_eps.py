"""The smallest eps of the mixed AdamW step.  Its kernel divides by a
denominator that it takes for 0 below fp32's normal range, so an eps down
there would make elements without moments (rows of tokens never seen)
0 / 0."""
import ctypes
import types

import numpy as np
import pytest

from muon_optimizer_step_02_b200 import binding as B

LEAST = 2.0 ** -126        # fp32's least normal value


def status(eps):
    """Of a call without elements: it returns before any device work."""
    from muon_optimizer_step_02_b200 import _build
    _build.build()
    hp = B.adamw_mixed_hyper_t(0.01, 0.9, 0.95, eps, 0.1, 0.99, 0, 0)
    return B.lib().adamw_mixed_batched(None, 0, ctypes.byref(hp), 1, None, None, None, None)


@pytest.mark.parametrize("eps", [LEAST * (1 - 2.0 ** -53), 1e-39, 2.0 ** -149, 1e-60, 5e-324])
def test_eps_below_the_normal_range_is_refused(eps):
    assert status(eps) == B.MUON_ERR_INVALID_ARG


@pytest.mark.parametrize("eps", [0.0, LEAST, 1e-30, 1.0])
def test_other_eps_are_taken(eps):
    assert status(eps) == B.MUON_OK


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
def test_elements_without_moments(eight):
    """At the least eps their weights only decay; at 0 they are 0 / 0, and the
    others are as ever.  Sizes of a full block and a ragged one.

    Bound: p (1 - lr wd) takes three roundings at most (of the product lr wd,
    of the difference from 1, of the product with p), half a step each."""
    import torch
    n = 256 + 77
    seen = np.arange(n) % 3 == 0
    g = torch.from_numpy(np.where(seen, 1e-3, 0).astype(np.float32)).cuda()
    p0 = np.random.default_rng(0).standard_normal(n).astype(np.float32)
    new = {}
    for eps in (LEAST, 0.0, 1e-8):
        p = torch.from_numpy(p0).cuda()
        state = B.Adam8State.zeros(n) if eight else (torch.zeros_like(p), torch.zeros_like(p))
        h = types.SimpleNamespace(lr=0.01, beta1=0.9, beta2=0.95, eps=eps, weight_decay=0.1)
        B.adamw_mixed_batched([p], [g], [state], h, step=1, rounding="nearest")
        torch.cuda.synchronize()
        new[eps] = p.cpu().numpy()
    kept = p0.astype(np.float64) * (1 - 0.01 * 0.1)
    for eps in (LEAST, 1e-8):
        assert np.all(np.abs(new[eps] - kept)[~seen] <= 1.01 * 3 * 2.0 ** -24 * np.abs(p0)[~seen])
    assert np.isnan(new[0.0][~seen]).all()
    # eps is far below the others' roots: the same weights at 0 and at the least
    assert np.array_equal(new[0.0][seen], new[LEAST][seen]) and np.isfinite(new[0.0][seen]).all()
