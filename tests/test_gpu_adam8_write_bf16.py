"""Plain bf16 moments to 8-bit states where they have to be rounded: codes and
scale bytes bit for bit those of the oracle's 32-bit restatement on the bf16
values."""
import numpy as np
import pytest

import oracle.adamw_mixed_oracle as ao
from test_gpu_adamw_mixed import SIZES, Arrays, host, state

pytestmark = pytest.mark.gpu


def bf16(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16()


def moments(n, seed):
    """(m, root) of bf16's 8 bits each, of which codes keep 5 and 6: blocks of very
    different size, elements far below and near their block's largest, zeros of
    both signs, and bf16's subnormal numbers."""
    r = np.random.default_rng(seed)
    rows = np.repeat(10.0 ** r.uniform(-25, 25, -(-n // 256)), 256)[:n]
    out = []
    for _ in range(2):
        x = r.standard_normal(n) * np.exp(2.5 * r.standard_normal(n)) * rows
        x[r.random(n) < 0.05] = 0.0
        x[r.random(n) < 0.02] = 1e-39
        out.append(x)
    m = np.where(r.random(n) < 0.02, -0.0, out[0])
    return bf16(m), bf16(np.abs(out[1]))


def check(s, m, r):
    b = host(s.scale).reshape(-1, 2)
    for got, byte, x, bits in ((s.exp_avg, b[:, 0], host(m), ao.M_BITS),
                               (s.root, b[:, 1], host(r), ao.R_BITS)):
        codes, want = ao.codes_f32(x, bits)
        assert np.array_equal(byte, want)
        assert np.array_equal(host(got), codes)


@pytest.mark.parametrize("shift", [0, 1, None])
@pytest.mark.parametrize("sizes", [SIZES, [1024 * (9 + i % 7) + 100 * (i % 3) for i in range(60)]])
def test_rounding_bf16_moments(sizes, shift):
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    new = Arrays()
    states, M, R = [], [], []
    for i, n in enumerate(sizes):
        new.shift = (0, 1, 0, 4, 8)[i % 5] if shift is None else shift
        m, r = moments(n, i)
        M.append(new.tensor(m))
        R.append(new.tensor(r))
        states.append(state(np.full(n, 5), np.full(n, 5), np.full(2 * -(-n // 256), 5), new))
    B.adam8_write_batched(states, M, R)
    torch.cuda.synchronize()
    for s, m, r in zip(states, M, R):
        check(s, m, r)
    new.check_guards()


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("bits", [ao.M_BITS, ao.R_BITS])
def test_every_bf16_of_the_codes_range(bits, shift):
    """All bf16 values of the exponents that a block's codes span and two below,
    under one scale: every tie between two codes among them."""
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    new = Arrays(shift)
    e = np.arange(-13 - bits, 1)
    v = ((1 + np.arange(128) / 128.0)[None, :] * np.exp2(e)[:, None]).reshape(-1)
    v = v[v <= 2.0 - 2.0 ** -bits]
    top = 2.0 - 2.0 ** -bits                       # each block starts with the top code's value
    rows = [np.concatenate([[top], v[k:k + 255]]) for k in range(0, v.size, 255)]
    v = np.concatenate(rows)
    x = bf16(np.where(np.arange(v.size) % 2 == 1, -v, v) if bits == ao.M_BITS else v)
    assert np.array_equal(np.abs(x.float().numpy()), v)          # (bf16 holds them)
    n = v.size
    m, r = (new.tensor(x if b == bits else torch.zeros(n, dtype=torch.bfloat16))
            for b in (ao.M_BITS, ao.R_BITS))
    s = state(np.full(n, 5), np.full(n, 5), np.full(2 * -(-n // 256), 5), new)
    B.adam8_write_batched([s], [m], [r])
    torch.cuda.synchronize()
    check(s, m, r)
    byte = host(s.scale).reshape(-1, 2)[:, 0 if bits == ao.M_BITS else 1]
    assert np.all(byte == 127)
    # and the definition in 64 bits: the same codes wherever fp32 keeps all bits
    codes, _ = ao.round_to_codes(v.astype(np.float64), bits)
    got = host(s.exp_avg) & 0x7F if bits == ao.M_BITS else host(s.root)
    assert np.array_equal(got, codes)
    new.check_guards()
