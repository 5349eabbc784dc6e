"""Refusals of the mixed AdamW step, the gradient norm and the 8-bit state
conversions that come before any device work, through the C ABI and the
binding.  The pointers are made up: no call here may reach a launch."""
import ctypes
import types

import pytest

from muon_optimizer_step_02_b200 import binding as B

E, A, W, U = (B.MUON_ERR_INVALID_ARG, B.MUON_ERR_ALIGNMENT, B.MUON_ERR_WORKSPACE,
              B.MUON_ERR_UNSUPPORTED)
P = 0x10000


@pytest.fixture(scope="module")
def L():
    from muon_optimizer_step_02_b200 import _build
    _build.build()
    return B.lib()


def tensor(**kw):
    t = dict(param=P, grad=2 * P, exp_avg=3 * P, exp_avg_sq=4 * P, scale=None, ema=None,
             copy_bf16=None, numel=4, lr_scale=1.0, wd_scale=1.0, grad_dtype=0)
    t.update(kw)
    return B.adamw_mixed_tensor_t(*t.values())


def hyper(**kw):
    h = dict(lr=0.01, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, ema_decay=0.99, seed=0,
             rounding=0)
    h.update(kw)
    return B.adamw_mixed_hyper_t(*h.values())


def step(L, t=None, h=None, n=1, step=1, step_dev=None, lr=None, coef=None):
    arr = (B.adamw_mixed_tensor_t * 1)(t if t is not None else tensor())
    hp = hyper() if h is None else h
    return L.adamw_mixed_batched(arr, n, ctypes.byref(hp), step, step_dev, lr, coef, None)


@pytest.mark.parametrize("kw", [
    dict(lr=float("nan")), dict(lr=float("inf")), dict(beta1=1.0), dict(beta1=-0.1),
    dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=-1.0), dict(weight_decay=float("inf")),
    dict(ema_decay=float("nan")), dict(rounding=2), dict(rounding=-1)])
def test_step_refuses_bad_settings(L, kw):
    assert step(L, h=hyper(**kw)) == E


@pytest.mark.parametrize("kw, status", [
    (dict(numel=-1), E), (dict(param=None), E), (dict(grad=None), E), (dict(exp_avg=None), E),
    (dict(exp_avg_sq=None), E), (dict(grad_dtype=2), E), (dict(lr_scale=float("nan")), E),
    (dict(wd_scale=float("inf")), E), (dict(param=P + 2), A), (dict(grad=P + 2), A),
    (dict(grad=P + 1, grad_dtype=1), A), (dict(exp_avg=P + 1), A), (dict(exp_avg_sq=P + 2), A),
    (dict(ema=P + 1), A), (dict(copy_bf16=P + 1), A), (dict(numel=(1 << 39) + 1), U)])
def test_step_refuses_bad_tensors(L, kw, status):
    assert step(L, tensor(**kw)) == status


def test_step_refuses_bad_calls(L):
    hp = hyper()
    assert L.adamw_mixed_batched(None, 1, ctypes.byref(hp), 1, None, None, None, None) == E
    arr = (B.adamw_mixed_tensor_t * 1)(tensor())
    assert L.adamw_mixed_batched(arr, 1, None, 1, None, None, None, None) == E
    assert step(L, n=-1) == E
    assert step(L, step=0) == E
    assert step(L, step_dev=P + 2) == A
    assert step(L, lr=P + 1) == A
    assert step(L, coef=P + 2) == A
    two = (B.adamw_mixed_tensor_t * 2)(tensor(numel=1 << 38), tensor(numel=(1 << 38) + 1))
    assert L.adamw_mixed_batched(two, 2, ctypes.byref(hp), 1, None, None, None, None) == U
    # nothing to do: no device is asked for
    assert step(L, tensor(numel=0, param=None)) == B.MUON_OK
    assert L.adamw_mixed_batched(None, 0, ctypes.byref(hp), 1, None, None, None, None) == B.MUON_OK


def norm(L, grad=P, numel=4, dtype=0, limit=1.0, ws=P, ws_n=None, out=P, n=1):
    arr = (B.grad_tensor_t * 1)(B.grad_tensor_t(grad, numel, dtype))
    ws_n = L.grad_norm_workspace_bytes() if ws_n is None else ws_n
    return L.grad_norm_batched(arr, n, limit, ws, ws_n, out, None)


def test_norm_refuses(L):
    need = L.grad_norm_workspace_bytes()
    assert norm(L, limit=0.0) == E and norm(L, limit=-1.0) == E and norm(L, limit=float("nan")) == E
    assert norm(L, grad=None) == E and norm(L, numel=-1) == E and norm(L, dtype=2) == E
    assert norm(L, out=None) == E and norm(L, out=P + 2) == A and norm(L, n=-1) == E
    assert norm(L, ws=None) == W and norm(L, ws=P + 8) == W and norm(L, ws_n=need - 1) == W
    assert norm(L, grad=P + 2) == A and norm(L, grad=P + 1, dtype=1) == A
    assert norm(L, numel=(1 << 39) + 1) == U
    assert L.grad_norm_batched(None, 1, 1.0, P, need, P, None) == E


@pytest.mark.parametrize("name", ["adam8_write_batched", "adam8_read_batched"])
def test_conversions_refuse(L, name):
    fn = getattr(L, name)

    def call(dtype=0, n=1, **kw):
        t = dict(exp_avg8=P, root8=2 * P, scale=3 * P, exp_avg=4 * P, second=5 * P, numel=4)
        t.update(kw)
        return fn((B.adam8_tensor_t * 1)(B.adam8_tensor_t(*t.values())), n, dtype, None)
    for key in ("exp_avg8", "root8", "scale", "exp_avg", "second"):
        assert call(**{key: None}) == E
    assert call(numel=-1) == E and call(n=-1) == E and call(dtype=2) == E
    assert call(exp_avg=P + 2) == A and call(second=P + 1, dtype=1) == A
    assert call(numel=(1 << 39) + 1) == U
    assert fn(None, 1, 0, None) == E
    assert call(numel=0, scale=None) == B.MUON_OK and fn(None, 0, 0, None) == B.MUON_OK


def test_launch_counts(L):
    assert [B.adamw_mixed_launches(n) for n in (0, 1, 400, 401, 801)] == [1, 1, 1, 2, 3]
    assert [B.grad_norm_launches(n) for n in (0, 1, 1300, 1301)] == [1, 1, 1, 2]
    assert [B.adam8_launches(n) for n in (0, 1, 500, 501)] == [0, 1, 1, 2]


def test_structures_match_the_header(L):
    """Sizes of the structures under the C rules of the header."""
    assert ctypes.sizeof(B.adamw_mixed_hyper_t) == 64
    assert ctypes.sizeof(B.adamw_mixed_tensor_t) == 80
    assert ctypes.sizeof(B.grad_tensor_t) == 24
    assert ctypes.sizeof(B.adam8_tensor_t) == 48


def test_binding_refuses_host_tensors():
    import torch
    x, u = torch.zeros(4), torch.zeros(4, dtype=torch.uint8)
    h = types.SimpleNamespace(lr=0.1, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0)
    for call in (lambda: B.Adam8State(u, u, u[:2]),
                 lambda: B.adamw_mixed_bind([x], [x], [(x, x)], h),
                 lambda: B.grad_norm_bind([x], 1.0, x[:2], u),
                 lambda: B.adamw_mixed_bind([3.0], [x], [(x, x)], h)):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="one grad"):
        B.adamw_mixed_bind([x], [], [(x, x)], h)
    with pytest.raises(ValueError, match="one grad"):
        B.adamw_mixed_bind([x], [x], [(x, x)], h, lr_scales=[1.0, 2.0])
    with pytest.raises(ValueError, match="rounding"):
        B.adamw_mixed_bind([], [], [], h, rounding="up")
    with pytest.raises(ValueError, match="one exp_avg"):
        B.adam8_read_bind([], [x], [])


def test_overlap_check():
    import torch
    a = torch.arange(10.0)

    def bad(written, read):
        with pytest.raises(ValueError, match="overlaps"):
            B._check_overlap([(t, "w{}", i) for i, t in enumerate(written)],
                             [(t, "r{}", i) for i, t in enumerate(read)])

    def good(written, read):
        B._check_overlap([(t, "w{}", i) for i, t in enumerate(written)],
                         [(t, "r{}", i) for i, t in enumerate(read)])
    bad([a, a], [])
    bad([a[:5]], [a[4:]])
    bad([a[2:3]], [a])
    bad([a[2:3], a[5:6]], [a[:3], a[:1]])
    bad([a[5:]], [a[:3], a[:9], a[:1]])
    good([], [a, a])
    good([a[:5], None], [a[5:], a[5:], a[:0]])
    good([a[5:]], [a[:5], a[:5]])
