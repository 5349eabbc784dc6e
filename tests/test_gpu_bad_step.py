"""A step with a bad matrix gradient, withheld as a whole: the norm of all
gradients first, and the other calls only if its coefficient is a number."""
import math

import pytest

import oracle.adamw_mixed_oracle as ao
from muon_optimizer_step_02_b200 import workloads as wl
from test_gpu_adamw_mixed import DECAY, Case, host, hyper, near

pytestmark = pytest.mark.gpu


def test_a_bad_matrix_gradient_withholds_the_whole_step():
    import torch
    from gpu_harness import GpuMuon
    from muon_optimizer_step_02_b200 import binding as B
    h = wl.Hyper(momentum=0.95, lr=0.02, weight_decay=0.1)
    w = wl.custom([(128, 64), (64, 192)], h, [wl.FIXED_QUINTIC] * 5, name="bad step")
    mu = GpuMuon(w, with_out=False)
    mg = mu.grads(0)
    rest = Case([64 * 512, 512], lambda i: i == 0, "bf16")
    em = [x.clone().view(-1) for x in mu.W]
    out = torch.zeros(2, device="cuda")
    step = torch.zeros(2, dtype=torch.int32, device="cuda")
    norm = B.grad_norm_bind(mg + rest.G, 0.1, out, B.grad_norm_workspace())
    muon = mu.plan.bind(mu.W, mu.M, mg, h, w.coeffs, mu.ws, mu.scales)
    adam = B.adamw_mixed_bind(rest.P, rest.G, rest.S, hyper(), rest.E, rest.C, DECAY,
                              step_dev=step, grad_scale=out[1:], rounding="stochastic", seed=1)
    average = B.ema_bind(em, [x.view(-1) for x in mu.W], DECAY)

    def whole_step():
        norm()
        if not math.isnan(out[1].item()):
            muon()
            adam()
            average()
        torch.cuda.synchronize()

    arrays = [*mu.W, *mu.M, *em, *rest.arrays(), step]
    before = [x.clone() for x in arrays]
    good = mg[1][3, 5].clone()
    mg[1][3, 5] = float("inf")
    whole_step()
    assert math.isnan(out[1].item()) and not math.isfinite(out[0].item())
    assert all(torch.equal(x, y) for x, y in zip(before, arrays))
    mg[1][3, 5] = good
    whole_step()
    n, c = ao.grad_norm([host(g) for g in mg + rest.G], 0.1)
    assert near(out[0].item(), n) and near(out[1].item(), c) and step.tolist() == [1, 0]
    assert all(bool(x.isfinite().all()) for x in (*mu.W, *mu.M, *em))
    assert not any(torch.equal(x, y) for x, y in zip(before[:4], arrays[:4]))
    assert mu.plan.last_error() == 0
    mu.plan.close()
