"""Arguments of the AdamW bindings that are checked on the host, with host tensors
that the checks take for the device's: no call here is run."""
import types

import pytest

from muon_optimizer_step_02_b200 import binding as B


def on_device(x):
    import torch

    class Device(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return None
    return torch.Tensor._make_subclass(Device, x)


def hyper():
    return types.SimpleNamespace(lr=0.1, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0)


@pytest.mark.parametrize("step", [-(2 ** 31) - 1, -(2 ** 32) + 1, 2 ** 31, 2 ** 32 + 1])
def test_steps_past_32_bits_are_refused(step):
    """They would reach the library as other numbers, some of them valid steps."""
    with pytest.raises(ValueError, match="32 bits"):
        B.adamw_mixed_bind([], [], [], hyper(), step=step)
    run = B.adamw_mixed_bind([], [], [], hyper())
    with pytest.raises(ValueError, match="32 bits"):
        run(step_now=step)


@pytest.mark.parametrize("step", [-(2 ** 31), -1, 0])
def test_steps_below_one_are_refused(step):
    with pytest.raises(B.MuonError):
        B.adamw_mixed_bind([], [], [], hyper(), step=step)(stream=0)
    with pytest.raises(B.MuonError):
        B.adamw_mixed_bind([], [], [], hyper())(step_now=step, stream=0)
