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


def states_with(**kw):
    """An Adam8State of 300 elements (two blocks) whose tensors are replaced after
    it was made, as by a checkpoint's loader."""
    import torch
    u = lambda n: on_device(torch.zeros(n, dtype=torch.uint8))  # noqa: E731
    s = B.Adam8State(u(300), u(300), u(4))
    for key, t in kw.items():
        setattr(s, key, on_device(t))
    return s


def bound(call, s):
    import torch
    f = lambda d=torch.float32: on_device(torch.zeros(300, dtype=d))  # noqa: E731
    if call == "step":
        return B.adamw_mixed_bind([f()], [f()], [s], hyper(), rounding="stochastic")
    return getattr(B, call)([s], [f()], [f()])


CALLS = ["step", "adam8_read_bind", "adam8_write_bind"]


@pytest.mark.parametrize("call", CALLS)
def test_states_as_they_were_made_bind(call):
    bound(call, states_with())


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("key, numel, match", [
    ("exp_avg", 299, "exp_avg has 299"), ("root", 299, "root has 299"), ("root", 301, "root has 301"),
    ("scale", 2, "scale has 2"), ("scale", 6, "scale has 6")])
def test_states_whose_tensors_were_replaced_are_checked(call, key, numel, match):
    """A root or scale of another size would be read and written past its end."""
    import torch
    s = states_with(**{key: torch.zeros(numel, dtype=torch.uint8)})
    with pytest.raises(ValueError, match=match):
        bound(call, s)


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("key", ["root", "scale"])
def test_states_whose_tensors_have_another_type_are_refused(call, key):
    import torch
    s = states_with(**{key: torch.zeros(4 if key == "scale" else 300)})
    with pytest.raises(ValueError, match=f"{key} must be torch.uint8"):
        bound(call, s)


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("key", ["exp_avg", "root", "scale"])
def test_states_whose_tensors_are_on_the_host_are_refused(call, key):
    import torch
    s = states_with()
    setattr(s, key, torch.zeros(4 if key == "scale" else 300, dtype=torch.uint8))
    with pytest.raises(ValueError, match=f"{key} must be a CUDA tensor"):
        bound(call, s)


@pytest.mark.parametrize("call", CALLS)
def test_bound_calls_keep_the_state_tensors_that_they_write(call):
    """Replacing a state's tensors after a bind leaves the bound ones alive: the
    call still writes to them."""
    import gc
    import weakref

    import torch
    s = states_with()
    refs = [weakref.ref(t) for t in (s.exp_avg, s.root, s.scale)]
    run = bound(call, s)
    s.exp_avg, s.root, s.scale = (on_device(torch.zeros(n, dtype=torch.uint8)) for n in (300, 300, 4))
    gc.collect()
    assert all(r() is not None for r in refs)
    del run
    gc.collect()
    assert all(r() is None for r in refs)
