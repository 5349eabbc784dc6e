"""Pins of the oracle of AdamW with 8-bit moments: the codes against their
definition and brute force, the roundings, the random bits, the 32-bit
restatement against the 64-bit one, and the step against the AdamW oracle."""
import numpy as np
import pytest

import oracle.adamw_mixed_oracle as ao
import oracle.muon_oracle as mo

BITS = [ao.M_BITS, ao.R_BITS]


def _values(bits, seed=0, n=1000, spread=3.0):
    r = np.random.default_rng(seed)
    x = (r.standard_normal(n) * np.exp(spread * r.standard_normal(n)) * 1e-3).astype(np.float32)
    return x if bits == ao.M_BITS else np.abs(x)


@pytest.mark.parametrize("bits", BITS)
def test_code_values(bits):
    v = ao.code_values(bits)
    mag = v[:128] if bits == ao.M_BITS else v
    assert mag[0] == 0 and np.all(np.diff(mag) > 0)
    assert mag[-1] == 2.0 - 2.0 ** -bits and mag[7 << bits] == 1.0
    assert mag[1] == 2.0 ** (-6 - bits) and mag[1 << bits] == 2.0 ** -6
    if bits == ao.M_BITS:
        assert np.array_equal(v[128:], -v[:128])
    # spacing: relative to the value at most 2^-bits from the least normal on
    normal = mag[1 << bits:]
    assert np.max(np.diff(normal) / normal[:-1]) == 2.0 ** -bits


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("n", [1, 255, 256, 257, 1000])
def test_nearest_is_the_closest_of_all_codes(bits, n):
    x = _values(bits, n, n).astype(np.float64)
    codes, b = ao.round_to_codes(x, bits)
    got = ao.decode(codes, b, bits)
    every = ao.code_values(bits)[None, :] * np.exp2(np.repeat(b, ao.BLOCK)[:n] - 127.0)[:, None]
    best = np.min(np.abs(every - x[:, None]), axis=1)
    off = np.abs(got - x)
    lifted = (bits == ao.R_BITS) & (codes == 1)    # a root below half of code 1 is lifted to it
    assert np.all((off == best) | lifted)
    # the byte is the least that reaches the largest
    top = 2.0 - 2.0 ** -bits
    for k in range(b.size):
        big = np.max(np.abs(x[k * ao.BLOCK:(k + 1) * ao.BLOCK]))
        assert top * 2.0 ** (b[k] - 127.0) >= big > top * 2.0 ** (b[k] - 128.0)


@pytest.mark.parametrize("bits", BITS)
def test_ties_go_to_the_even_code(bits):
    mag = ao.code_values(bits)[:128 if bits == ao.M_BITS else 256]
    mid = (mag[1:-1] + mag[2:]) / 2
    x = np.concatenate([[mag[-1]], mid])[:ao.BLOCK]     # one block at byte 127
    codes, b = ao.round_to_codes(x, bits)
    assert b[0] == 127 and codes[0] == mag.size - 1
    assert np.all(codes[1:] % 2 == 0)
    c32, b32 = ao.codes_f32(x.astype(np.float32), bits)
    assert np.array_equal(c32, codes) and b32[0] == 127


@pytest.mark.parametrize("bits", BITS)
def test_values_on_codes_stay_when_the_scale_moves(bits):
    """A value on a code keeps its value exactly when the block's largest grows
    up to fourfold, as long as it stays above the subnormal codes."""
    v = ao.code_values(bits)
    v = v[(np.abs(v) >= 2.0 ** -4)]
    for up in (1.0, 2.0, 4.0):
        x = np.concatenate([[up * 1.5], v])[:ao.BLOCK]
        for enc in (lambda y: ao.round_to_codes(y, bits),
                    lambda y: ao.codes_f32(y.astype(np.float32), bits)):
            codes, b = enc(x)
            assert np.array_equal(ao.decode(codes, b, bits), x)


@pytest.mark.parametrize("bits", BITS)
def test_special_blocks(bits):
    x = np.zeros(3 * ao.BLOCK, np.float32)
    x[256] = np.inf
    x[512] = np.nan
    for enc in (ao.round_to_codes, ao.codes_f32):
        codes, b = enc(x, bits)
        assert list(b) == [ao.LOW, ao.NAN_BYTE, ao.NAN_BYTE] and not codes.any()
        v = ao.decode(codes, b, bits)
        assert np.all(v[:256] == 0) and np.all(np.isnan(v[256:]))
    # magnitudes past the top code of byte 245 do not fit
    for enc in (ao.round_to_codes, ao.codes_f32):
        assert enc(np.float32([2.0 ** 118 * (2 - 2.0 ** -bits)]), bits)[1][0] == ao.HIGH
        assert enc(np.float32([2.0 ** 119]), bits)[1][0] == ao.NAN_BYTE


def test_a_root_above_zero_stays_above_zero():
    x = np.array([1.0, 1e-30, 0.0, 1e-5], np.float32)
    for enc in (ao.round_to_codes, ao.codes_f32):
        for six in (None, np.zeros(4, np.int64)):
            codes, _ = enc(x, ao.R_BITS, six)
            assert codes[1] == 1 and codes[2] == 0 and codes[3] >= 1


@pytest.mark.parametrize("bits", BITS)
def test_stochastic_rounding_is_unbiased(bits):
    """Over all 2^16 random halves the mean of a value's roundings is the value
    to 2^-16 of the gap between its codes (the bits' own step)."""
    x = _values(bits, 5, 40, 1.0)
    x[0] = np.max(np.abs(x)) * 1.5
    codes, b = ao.codes_f32(x, bits)
    unit = np.exp2(b[0] - 127.0)
    total = np.zeros(40)
    for part in np.split(np.arange(65536), 16):
        block = np.zeros((part.size, ao.BLOCK), np.float32)
        block[:, :40] = x
        c, bb = ao.codes_f32(block.reshape(-1), bits, np.repeat(part, ao.BLOCK))
        assert np.all(bb == b[0])
        total += ao.decode(c, bb, bits).reshape(block.shape)[:, :40].sum(axis=0)
    total /= 65536
    gap = np.maximum(np.abs(x.astype(np.float64)) * 2.0 ** -bits, unit * 2.0 ** (-6 - bits))
    far = np.abs(total - x.astype(np.float64))
    small = (bits == ao.R_BITS) & (np.abs(x) < unit * 2.0 ** (-6 - bits))
    assert np.all((far <= gap * 2.0 ** -16) | small)


def test_random_words_look_random():
    """Means of the bits, of both halves, and correlations between neighbours,
    steps, tensors and seeds: within 5 standard deviations of independence."""
    n = 1 << 16
    a = ao.random_words(1, 1, 0, n)
    others = [np.roll(a, 1), np.roll(a, ao.BLOCK), ao.random_words(1, 2, 0, n),
              ao.random_words(1, 1, 1, n), ao.random_words(2, 1, 0, n),
              ao.random_words(1 + (1 << 32), 1, 0, n)]
    bound = 5 / np.sqrt(n)
    for k in range(32):
        bit = ((a >> np.uint32(k)) & 1).astype(np.float64) * 2 - 1
        assert abs(bit.mean()) <= bound
        for o in others:
            assert abs((bit * (((o >> np.uint32(k)) & 1) * 2.0 - 1)).mean()) <= bound
    lo, hi = (a & np.uint32(0xFFFF)) / 65536.0 - 0.5, (a >> np.uint32(16)) / 65536.0 - 0.5
    assert abs((lo * hi).mean() * 12) <= bound


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("stochastic", [False, True])
def test_32_bit_codes_agree_with_64_bit_ones(bits, stochastic):
    """On 32-bit values both levels give the same codes; below the least normal
    code the 32-bit pattern keeps 2^-(23 - bits) of a gap, so there a value
    nearer than that to a border may fall either way (at most one code)."""
    x = _values(bits, 9, 60000)
    six = (ao.random_words(3, 4, 5, x.size) & np.uint32(0xFFFF)).astype(np.int64) if stochastic else None
    c64, b64 = ao.round_to_codes(x, bits, six)
    c32, b32 = ao.codes_f32(x, bits, six)
    assert np.array_equal(b64, b32)
    differ = c64 != c32
    subnormal = (c64 & (0x7F if bits == ao.M_BITS else 0xFF)) <= (1 << bits)
    assert not np.any(differ & ~subnormal) and differ.mean() < 1e-4
    assert np.all(np.abs(c64[differ].astype(int) - c32[differ].astype(int)) == 1)


def test_step_is_adamw():
    """The 64-bit step equals the AdamW oracle's, and its clip coefficient and
    factors act as on the inputs."""
    r = np.random.default_rng(2)
    p, g, m, e = (r.standard_normal(50) for _ in range(4))
    v = r.random(50)
    h = mo.AdamWHyper(lr=0.01, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
    got = ao.adamw_step(p, g, m, v, h, 7, e, 0.99)
    want = mo.adamw_ema(p, g, m, v, e, h, 7, 0.99)
    for a, b in zip(got, want):
        assert np.allclose(a, b, rtol=1e-14, atol=0)
    a = ao.adamw_step(p, g, m, v, h, 7, coef=0.25)
    b = mo.adamw_update(p, 0.25 * g, m, v, h, 7)
    assert all(np.allclose(x, y, rtol=1e-14, atol=0) for x, y in zip(a, b))
    h2 = mo.AdamWHyper(lr=0.005, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0)
    a = ao.adamw_step(p, g, m, v, h, 7, lr_scale=0.5, wd_scale=0.0)
    b = mo.adamw_update(p, g, m, v, h2, 7)
    assert all(np.allclose(x, y, rtol=1e-14, atol=0) for x, y in zip(a, b))
    m32, v32, r32 = ao.moments_f32(g, m, v, h)
    assert np.allclose(m32, got[1], rtol=1e-5, atol=1e-6) and np.allclose(v32, got[2], rtol=1e-6)
    assert np.allclose(r32 ** 2, got[2], rtol=1e-6)


def test_grad_norm():
    assert ao.grad_norm([np.array([3.0, 0.0]), np.array([-4.0])], 1.0) == (5.0, 1 / (5 + 1e-6))
    assert ao.grad_norm([], 2.0) == (0.0, 1.0)
    assert ao.grad_norm([np.array([0.3])], 1.0)[1] == 1.0
    n, c = ao.grad_norm([np.array([1.0, np.inf])], 1.0)
    assert n == np.inf and np.isnan(c)
    n, c = ao.grad_norm([np.array([np.inf]), np.array([np.nan])], 1.0)
    assert np.isnan(n) and np.isnan(c)
