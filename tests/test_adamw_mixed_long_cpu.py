"""8-bit moments over many steps, where single steps show nothing: the oracle's
32-bit steps carrying their own 8-bit state against AdamW in 64 bits carrying
its own, for both roundings; and the binding's choice between them.  No GPU."""
import types
import warnings

import numpy as np
import pytest

import oracle.adamw_mixed_oracle as ao
from muon_optimizer_step_02_b200 import binding as B

SEED = 7


def run_codes(grads, beta1, beta2, rounding, lr=1e-3):
    """Steps of one tensor through 8-bit states; yields (t, p, m codes, r), p in
    64 bits from the moments before their rounding, as the kernel has it."""
    h = types.SimpleNamespace(beta1=beta1, beta2=beta2)
    n = grads(1).size
    m = r = p = np.zeros(n)
    for t in range(1, 1 << 30):
        m32, _, r32 = ao.moments_f32(grads(t), m, None, h, root=r)
        with np.errstate(invalid="ignore"):
            p = p - lr * (m32.astype(np.float64) / (1 - beta1 ** t)) / (
                r32.astype(np.float64) / np.sqrt(1 - beta2 ** t) + 1e-8)
        lo = hi = None
        if rounding == "stochastic":
            w = ao.random_words(SEED, t, 0, n)
            lo, hi = (w & np.uint32(0xFFFF)).astype(np.int64), (w >> np.uint32(16)).astype(np.int64)
        mc, mb = ao.codes_f32(m32, ao.M_BITS, lo)
        rc, rb = ao.codes_f32(r32, ao.R_BITS, hi)
        m, r = ao.decode(mc, mb, ao.M_BITS), ao.decode(rc, rb, ao.R_BITS)
        yield t, p, mc, r


def stopping(ratio, stop, dead):
    """Gradients of one block: 1, and `ratio` in the first `dead` elements until
    step `stop`, 0 there after it."""
    def grads(t):
        g = np.ones(ao.BLOCK, np.float32)
        g[:dead] = ratio if t <= stop else 0.0
        return g
    return grads


@pytest.mark.parametrize("ratio", [0.03, 0.003])
@pytest.mark.parametrize("beta1, beta2", [(0.9, 0.95), (0.95, 0.95), (0.9, 0.999)])
def test_stochastic_moments_of_stopped_gradients_end_at_zero(beta1, beta2, ratio):
    """Part of a block stops having gradients.  The mean of a stochastically
    rounded first moment is b1^k m, below 2^11 units of its last code, and a
    moment that is not zero is one unit at least: after k steps it is not zero
    with a probability below b1^k 2^11, 1e-9 for 16 elements and the k below.  A zero moment without a gradient stays zero: the weights have come
    to rest."""
    dead, stop = 16, 50
    k = int(np.ceil(np.log(1e-9 / 16 / 2 ** 11) / np.log(beta1)))
    rest = None
    for t, p, mc, _ in run_codes(stopping(ratio, stop, dead), beta1, beta2, "stochastic"):
        if t == stop + k:
            assert not (mc[:dead] & 0x7F).any()
            rest = p[:dead].copy()
        if t == stop + k + 200:
            assert np.array_equal(p[:dead], rest)
            return


@pytest.mark.parametrize("beta1, stuck", [(0.9, 4), (0.95, 10)])
def test_nearest_moments_of_stopped_gradients_stay(beta1, stuck):
    """What the header says of nearest rounding: a first moment of k units below
    the least normal code stays where (1 - b1) k is under half a unit (or ties
    to its own, even, code), and its weight goes on moving, by about the
    learning rate each step."""
    dead, lr, seen = 16, 1e-3, {}
    for t, p, mc, r in run_codes(stopping(0.03, 50, dead), beta1, 0.95, "nearest", lr):
        seen[t] = p[:dead].copy()
        if t == 2000:
            break
    assert np.all(mc[:dead] == stuck)
    assert np.all(seen[1900] - seen[2000] > 100 * lr * 0.1)


@pytest.mark.parametrize("beta2", [0.95, 0.99, 0.999])
def test_stochastic_roots_follow_the_second_moment(beta2):
    """Gradients of size 1, then 20 times smaller.  A root's rounding leaves its
    mean and adds at most (2^-5 / 2)^2 = 2^-12 of v to the mean of its square
    (codes are 2^-5 of their value apart at most), so the mean second moment lies
    between AdamW's v and the same recursion with (1 + 2^-12) a step; the mean
    over the elements is within 5 of its standard errors of that."""
    n, steps = 1024, 1200
    signs = np.where(np.random.default_rng(3).random(n) < 0.5, -1, 1).astype(np.float32)
    low = high = 0.0

    def size(t):
        return 1.0 if t <= steps else 0.05
    for t, _, _, r in run_codes(lambda t: signs * np.float32(size(t)), 0.9, beta2, "stochastic"):
        g2 = float(np.float32(size(t))) ** 2
        low = beta2 * low + (1 - beta2) * g2
        high = (1 + 2.0 ** -12) * (beta2 * high + (1 - beta2) * g2)
        if t in (steps, 2 * steps):
            v = r * r
            error = 5 * v.std() / np.sqrt(n) + 1e-5 * low     # (fp32's own, of all steps)
            assert low - error <= v.mean() <= high + error, t
        if t == 2 * steps:
            return


# ---- the binding's choice --------------------------------------------------------

def on_device(x):
    """A host tensor that the binding's checks take for one of the device; no call
    made with it may be run."""
    import torch

    class Device(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return None
    return torch.Tensor._make_subclass(Device, x)


def bind(eight, **kw):
    import torch
    h = types.SimpleNamespace(lr=0.1, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0)
    f = lambda: on_device(torch.zeros(300))  # noqa: E731
    u = lambda n: on_device(torch.zeros(n, dtype=torch.uint8))  # noqa: E731
    state = B.Adam8State(u(300), u(300), u(4)) if eight else (f(), f())
    return B.adamw_mixed_bind([f(), f()], [f(), f()], [(f(), f()), state], h, **kw)


def test_nearest_rounding_of_states_is_not_taken_silently():
    with pytest.warns(UserWarning, match="rounding='stochastic'"):
        bind(True)


def test_a_stated_rounding_does_not_warn():
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        bind(True, rounding="nearest")
        bind(True, rounding="stochastic")
        bind(False)
