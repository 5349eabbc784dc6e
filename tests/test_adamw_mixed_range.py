"""Settings of the mixed AdamW step that fit 64 bits but not the 32 that its
kernel takes them in, where they would be infinite and make weights NaN that
the formula leaves alone.  Calls without elements: they return before any
device work."""
import ctypes

import pytest

from muon_optimizer_step_02_b200 import binding as B

LARGEST = (2 - 2.0 ** -23) * 2.0 ** 127        # of fp32
PAST = LARGEST + 2.0 ** 103                    # half a step further: rounds to infinity


def status(**kw):
    from muon_optimizer_step_02_b200 import _build
    _build.build()
    h = dict(lr=0.01, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, ema_decay=0.99, seed=0,
             rounding=0)
    h.update(kw)
    return B.lib().adamw_mixed_batched(None, 0, ctypes.byref(B.adamw_mixed_hyper_t(*h.values())), 1,
                                       None, None, None, None)


@pytest.mark.parametrize("key", ["lr", "weight_decay", "ema_decay"])
@pytest.mark.parametrize("value", [PAST, 1e39, 1e300, -1e39])
def test_settings_past_fp32_are_refused(key, value):
    assert status(**{key: value}) == B.MUON_ERR_INVALID_ARG


@pytest.mark.parametrize("key", ["lr", "weight_decay", "ema_decay"])
@pytest.mark.parametrize("value", [LARGEST, -LARGEST, 0.0, 1e-300])
def test_settings_within_fp32_are_taken(key, value):
    assert status(**{key: value}) == B.MUON_OK
