"""AdamW with 32-bit or 8-bit moments, the gradient norm it clips with and the
conversions of its states, through the binding, against the 64-bit oracle and,
where the library fixes every rounding (moments and codes), bit for bit
against its restatement in 32 bits."""
import os
import types

import numpy as np
import pytest

import oracle.adamw_mixed_oracle as ao
from muon_optimizer_step_02_b200 import workloads as wl

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -24      # half a step of fp32, relative
GUARD = 64             # elements around every array, checked after the call
DECAY = 0.9965
# none, one, around one block's end, several blocks, odd, a vector, a table
SIZES = [0, 1, 3, 255, 256, 257, 512, 1000, 4096, 4099, 70001]


def hyper(**kw):
    return types.SimpleNamespace(**{**dict(lr=0.01, beta1=0.9, beta2=0.95, eps=1e-8,
                                           weight_decay=0.1), **kw})


class Arrays:
    """Device arrays inside guarded buffers, `shift` elements off their start."""

    def __init__(self, shift=0):
        self.shift, self.held = shift, []

    def __call__(self, a):
        import torch
        a = torch.from_numpy(np.ascontiguousarray(a))
        return self.tensor(a)

    def tensor(self, a):
        import torch
        lead = GUARD + self.shift
        buf = torch.full((lead + a.numel() + GUARD,), 77, dtype=a.dtype, device="cuda")
        buf[lead:lead + a.numel()] = a.cuda()
        self.held.append((buf, lead, a.numel()))
        return buf[lead:lead + a.numel()]

    def check_guards(self):
        for buf, lead, n in self.held:
            assert bool((buf[:lead] == 77).all()) and bool((buf[lead + n:] == 77).all())


def host(t):
    import torch
    return t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


class Case:
    """Tensors of one call with their host copies.  eight(i): whether tensor i
    has an 8-bit state; shift: elements that its arrays lie off their buffers'
    starts, or a function of i."""

    def __init__(self, sizes, eight, grad="f32", ema=True, copy=True, shift=0, seed=0, empty=False):
        import torch
        from muon_optimizer_step_02_b200 import binding as B
        self.sizes, self.new = sizes, Arrays()
        shift = shift if callable(shift) else lambda i, k=shift: k
        self.eight = [bool(eight(i)) for i in range(len(sizes))]
        self.P, self.G, self.S, self.E, self.C = [], [], [], [], []
        for i, n in enumerate(sizes):
            self.new.shift = shift(i)
            p, m, v, e = wl.adamw_state(n, i, seed, wid=300)
            m, v = (m * 0, v * 0) if empty else (m, v)
            self.P.append(self.new(p))
            g = torch.from_numpy(wl.adamw_grad(n, i, 1, seed, wid=300))
            half = grad == "bf16" or (grad == "both" and i % 3 != 1)
            self.G.append(self.new.tensor(g.bfloat16() if half else g))
            if self.eight[i]:
                (m8, mb), (r8, rb) = (ao.codes_f32(m, ao.M_BITS),
                                      ao.codes_f32(np.sqrt(v), ao.R_BITS))
                self.S.append(B.Adam8State(*(self.new(x.astype(np.uint8)) for x in (
                    m8, r8, np.stack([mb, rb], 1).reshape(-1)))))
            else:
                self.S.append((self.new(m), self.new(v)))
            self.E.append(self.new(e) if ema and i % 5 != 2 else None)
            self.C.append(self.new.tensor(torch.zeros(n, dtype=torch.bfloat16))
                          if copy and i % 5 != 3 else None)

    def set_grads(self, step, seed=0):
        import torch
        for i, n in enumerate(self.sizes):
            self.G[i].copy_(torch.from_numpy(wl.adamw_grad(n, i, step, seed, wid=300)))

    def arrays(self):
        """Every array of every tensor, the written ones first."""
        out = []
        for i in range(len(self.sizes)):
            s = self.S[i]
            s = (s.exp_avg, s.root, s.scale) if self.eight[i] else s
            out += [t for t in (self.P[i], *s, self.E[i], self.C[i]) if t is not None]
        return out

    def snapshot(self):
        out = []
        for i in range(len(self.sizes)):
            s = self.S[i]
            d = {"p": host(self.P[i]), "g": host(self.G[i]),
                 "e": None if self.E[i] is None else host(self.E[i])}
            if self.eight[i]:
                b = host(s.scale).reshape(-1, 2)
                d["m8"], d["r8"], d["mb"], d["rb"] = host(s.exp_avg), host(s.root), b[:, 0], b[:, 1]
                d["m"] = ao.decode(d["m8"], d["mb"], ao.M_BITS)
                d["r"] = ao.decode(d["r8"], d["rb"], ao.R_BITS)
                d["v"] = d["r"] ** 2
            else:
                d["m"], d["v"] = host(s[0]), host(s[1])
            out.append(d)
        return out


def check(c, before, h, t, coef=1.0, lr_scales=None, wd_scales=None, rounding="nearest", seed=0,
          decay=DECAY):
    """The state after one step against the oracles.  The bound on p': with
    A = |b1 m| + |(1-b1) g| and S = A / (1-b1^t) / (r' / sqrt(1-b2^t) + eps),
    in half steps (relative 2^-24): m' is off by at most 4 A (factors,
    products, sum), r' by 4 r', the denominator by 6, the quotient by 6 S + 10 S
    (its own division 2 ulp = 4), lr by 3 with its product, p's decay by
    1.1 |p| + the sum's |p| + lr S: together under 4 |p| + 21 lr S.  e' adds
    2 |d e| + 4 |(1-d) p'| to (1-d) times that."""
    after = c.snapshot()
    for i, n in enumerate(c.sizes):
        b, a = before[i], after[i]
        ls = 1.0 if lr_scales is None else lr_scales[i]
        ws = 1.0 if wd_scales is None else wd_scales[i]
        p, m, v, e = ao.adamw_step(b["p"], b["g"], b["m"], b["v"], h, t, b["e"], decay, coef, ls, ws)
        big = np.abs(h.beta1 * b["m"]) + np.abs((1 - h.beta1) * coef * b["g"].astype(np.float64))
        s = big / (1 - h.beta1 ** t) / (np.sqrt(v / (1 - h.beta2 ** t)) + h.eps)
        tol = 1.01 * HALF * (4 * np.abs(b["p"]) + 21 * h.lr * ls * s) + 1e-40
        what = f"tensor {i} ({n} elements)"
        assert np.all(np.abs(a["p"] - p) <= tol), what
        if e is not None:
            tol_e = (1 - decay) * tol + 1.01 * HALF * (2 * np.abs(decay * b["e"])
                                                       + 4 * np.abs((1 - decay) * p)) + 1e-40
            assert np.all(np.abs(a["e"] - e) <= tol_e), what
        if c.C[i] is not None:
            import torch
            assert torch.equal(c.C[i], c.P[i].bfloat16()), what
        if c.eight[i]:
            m32, _, r32 = ao.moments_f32(b["g"], b["m"], None, h, coef, root=b["r"])
            w = ao.random_words(seed, t, i, n) if rounding == "stochastic" else None
            lo = None if w is None else (w & np.uint32(0xFFFF)).astype(np.int64)
            hi = None if w is None else (w >> np.uint32(16)).astype(np.int64)
            for got, gb, x, bits, six in ((a["m8"], a["mb"], m32, ao.M_BITS, lo),
                                          (a["r8"], a["rb"], r32, ao.R_BITS, hi)):
                codes, byte = ao.codes_f32(x, bits, six)
                assert np.array_equal(got, codes) and np.array_equal(gb, byte), what
        else:
            m32, v32, _ = ao.moments_f32(b["g"], b["m"], b["v"], h, coef)
            assert np.array_equal(a["m"], m32) and np.array_equal(a["v"], v32), what
    c.new.check_guards()


FORMATS = {"32": lambda i: False, "8": lambda i: True, "mixed": lambda i: i % 2 == 0}


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
@pytest.mark.parametrize("form", list(FORMATS))
def test_step_matches_the_oracle(form, rounding, grad, shift):
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    h, seed = hyper(), 0x123456789ABCDEF
    c = Case(SIZES, FORMATS[form], grad, shift=shift)
    run = B.adamw_mixed_bind(c.P, c.G, c.S, h, c.E, c.C, DECAY, rounding=rounding, seed=seed)
    for t in (1, 2, 1000):
        before = c.snapshot()
        run(step_now=t)
        torch.cuda.synchronize()
        check(c, before, h, t, rounding=rounding, seed=seed)


@pytest.mark.parametrize("form", list(FORMATS))
@pytest.mark.parametrize("beta2", [0.0, 0.999])
def test_from_empty_states_with_factors(form, beta2):
    """First steps from zero states, with per-tensor factors, a coefficient and
    no averages or copies; also b1 = 0."""
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    for b1 in (0.0, 0.9):
        h = hyper(beta1=b1, beta2=beta2, eps=1e-6)
        c = Case(SIZES, FORMATS[form], "f32", ema=False, copy=False, empty=True)
        ls = [0.25 * (1 + i % 3) for i in range(len(SIZES))]
        ws = [0.5 * (i % 2) for i in range(len(SIZES))]
        coef = torch.tensor([0.375], device="cuda")
        run = B.adamw_mixed_bind(c.P, c.G, c.S, h, lr_scales=ls, wd_scales=ws, grad_scale=coef)
        for t in (1, 2):
            before = c.snapshot()
            run(step_now=t)
            torch.cuda.synchronize()
            check(c, before, h, t, 0.375, ls, ws)


@pytest.mark.parametrize("large", [1e-12, 1e12])
def test_gradients_of_very_different_size(large):
    """Elements far below their block's largest, and blocks far apart: codes
    down to the subnormal ones and the least byte, bit for bit."""
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    h = hyper(eps=1e-20)
    c = Case([5000, 256], FORMATS["8"], empty=True)
    r = np.random.default_rng(4)
    for i, n in enumerate(c.sizes):
        g = (r.standard_normal(n) * np.exp(5 * r.standard_normal(n)) * large).astype(np.float32)
        c.G[i].copy_(torch.from_numpy(g))
    run = B.adamw_mixed_bind(c.P, c.G, c.S, h, c.E, c.C, DECAY, rounding="stochastic", seed=5)
    for t in (1, 2, 3):
        before = c.snapshot()
        run(step_now=t)
        torch.cuda.synchronize()
        check(c, before, h, t, rounding="stochastic", seed=5)


@pytest.mark.parametrize("form", list(FORMATS))
def test_device_counter_and_graph_replay(form):
    """Steps counted on the device and replayed from one graph give the host
    steps' results bit for bit, random bits included."""
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    h = hyper()
    a, b, c = (Case(SIZES, FORMATS[form]) for _ in range(3))
    kw = dict(ema_decay=DECAY, rounding="stochastic", seed=77)
    run_a = B.adamw_mixed_bind(a.P, a.G, a.S, h, a.E, a.C, **kw)
    sb, sc = (torch.zeros(2, dtype=torch.int32, device="cuda") for _ in range(2))
    run_b = B.adamw_mixed_bind(b.P, b.G, b.S, h, b.E, b.C, step_dev=sb, **kw)
    run_c = B.adamw_mixed_bind(c.P, c.G, c.S, h, c.E, c.C, step_dev=sc, **kw)
    for t in range(1, 6):
        a.set_grads(t)
        run_a(step_now=t)
        b.set_grads(t)
        run_b()
    c.set_grads(1)
    run_c()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_c()
    for t in range(2, 6):
        c.set_grads(t)
        graph.replay()
    torch.cuda.synchronize()
    assert sb.tolist() == [5, 0] and sc.tolist() == [5, 0]
    for x, y, z in zip(a.arrays(), b.arrays(), c.arrays()):
        assert torch.equal(x, y) and torch.equal(x, z)
    del graph


def test_many_tensors_take_several_launches():
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    sizes = [(7 * i) % 37 + 300 * (i % 97 == 5) for i in range(900)]
    c = Case(sizes, FORMATS["mixed"])
    h, step = hyper(), torch.tensor([3, 0], dtype=torch.int32, device="cuda")
    run = B.adamw_mixed_bind(c.P, c.G, c.S, h, c.E, c.C, DECAY, step_dev=step,
                             rounding="stochastic", seed=9)
    before = c.snapshot()
    run()
    torch.cuda.synchronize()
    assert step.tolist() == [4, 0]
    check(c, before, h, 4, rounding="stochastic", seed=9)


@pytest.mark.parametrize("ema", [False, True])
@pytest.mark.parametrize("form", ["8", "mixed"])
def test_gradient_types_change_between_tensors(form, ema):
    """A thread block goes from tensors with bf16 gradients to ones with fp32
    gradients and back, full and ragged blocks in turn, while it copies one
    block ahead: enough tensors of a few units that each block sees several."""
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    h = hyper()
    sizes = [1024 * (20 + 7 * (i % 5)) + (0, 0, 300, 77)[i % 4] for i in range(380)]
    c = Case(sizes, FORMATS[form], "both", ema=ema, copy=False)
    run = B.adamw_mixed_bind(c.P, c.G, c.S, h, c.E, c.C, DECAY, rounding="stochastic", seed=8)
    for t in (1, 2):
        before = c.snapshot()
        run(step_now=t)
        torch.cuda.synchronize()
        check(c, before, h, t, rounding="stochastic", seed=8)


@pytest.mark.parametrize("form", list(FORMATS))
def test_alignment_changes_between_tensors(form):
    """Aligned and unaligned tensors (off by 1 to 16 elements, so that some arrays
    are and others are not aligned), ragged or not, in turn."""
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    h = hyper()
    sizes = [1024 * (9 + 5 * (i % 4)) + (0, 256, 300, 77, 0)[i % 5] for i in range(390)]
    c = Case(sizes, FORMATS[form], "both", shift=lambda i: (0, 0, 1, 0, 4, 8, 0, 16)[i % 8])
    run = B.adamw_mixed_bind(c.P, c.G, c.S, h, c.E, c.C, DECAY, rounding="stochastic", seed=8)
    for t in (1, 2):
        before = c.snapshot()
        run(step_now=t)
        torch.cuda.synchronize()
        check(c, before, h, t, rounding="stochastic", seed=8)


@pytest.mark.parametrize("case", range(int(os.environ.get("MUONB200_FUZZ_MIXED_CASES", "10"))))
def test_random_calls(case):
    """Random lists of tensors (sizes, state forms, gradient types, alignments),
    settings, coefficients, factors and steps, against the oracles."""
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    r = np.random.default_rng(1000 + case)
    count = int(np.exp(r.uniform(0, np.log(500))))
    top = np.log(3e5 if count > 30 else 3e6)
    sizes = [int(np.exp(r.uniform(0, top))) for _ in range(count)]
    while sum(sizes) > 6_000_000:
        sizes.pop(int(np.argmax(sizes)))
    sizes = sizes or [1]
    n = len(sizes)
    eight, off = r.random(n) < r.choice([0.0, 0.5, 1.0]), r.choice([0, 0, 0, 1, 2, 4, 8], n)
    c = Case(sizes, lambda i: eight[i], r.choice(["f32", "bf16", "both"]), ema=bool(r.random() < 0.6),
             copy=bool(r.random() < 0.6), shift=lambda i: int(off[i]), seed=case,
             empty=bool(r.random() < 0.3))
    h = hyper(lr=float(10 ** r.uniform(-4, -1)), beta1=float(r.choice([0.0, 0.9, 0.95])),
              beta2=float(r.choice([0.9, 0.95, 0.99, 0.999])), eps=float(r.choice([1e-8, 1e-12])),
              weight_decay=float(r.choice([0.0, 0.1])))
    rounding, seed = str(r.choice(["nearest", "stochastic"])), int(r.integers(0, 1 << 62))
    ls, ws = ([float(x) for x in r.choice([0.25, 0.5, 1.0, 2.0], n)] for _ in range(2))
    coef = float(np.float32(r.choice([1.0, r.uniform(0.01, 1.0)])))
    step = torch.tensor([int(r.choice([0, 5, 12345])), 0], dtype=torch.int32, device="cuda")
    run = B.adamw_mixed_bind(c.P, c.G, c.S, h, c.E, c.C, DECAY, step_dev=step, lr_scales=ls,
                             wd_scales=ws, rounding=rounding, seed=seed,
                             grad_scale=torch.tensor([coef], device="cuda"))
    for _ in range(2):
        before, t = c.snapshot(), step[0].item() + 1
        run()
        torch.cuda.synchronize()
        assert step.tolist() == [t, 0]
        check(c, before, h, t, coef, ls, ws, rounding, seed)
    norm, k = ao.grad_norm([host(g) for g in c.G], 0.1)
    got = norm_of(c.G, 0.1)
    assert near(got[0], norm) and near(got[1], k)


def test_a_call_without_elements_counts_its_step():
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    step = torch.zeros(2, dtype=torch.int32, device="cuda")
    empty = torch.zeros(0, device="cuda")
    runs = [B.adamw_mixed_bind([], [], [], hyper(), step_dev=step),
            B.adamw_mixed_bind([empty], [empty], [B.Adam8State.zeros(0)], hyper(), step_dev=step)]
    for k, run in enumerate(runs):
        run()
        torch.cuda.synchronize()
        assert step.tolist() == [k + 1, 0]
    B.adamw_mixed_batched([empty], [empty], [(empty, empty)], hyper())
    B.adam8_read_batched([B.Adam8State.zeros(0)], [empty], [empty])
    B.adam8_write_batched([], [], [])
    torch.cuda.synchronize()


def test_same_inputs_same_bits():
    """Two runs of several steps on many thread blocks give the same bits."""
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    runs = []
    for _ in range(2):
        c = Case([3 << 20, 4099, 77], FORMATS["mixed"], "bf16")
        step = torch.zeros(2, dtype=torch.int32, device="cuda")
        run = B.adamw_mixed_bind(c.P, c.G, c.S, hyper(beta2=0.999), c.E, c.C, DECAY,
                                 step_dev=step, rounding="stochastic", seed=-1)
        for _ in range(4):
            run()
        torch.cuda.synchronize()
        runs.append(c.arrays() + [step])
    for x, y in zip(*runs):
        assert torch.equal(x, y)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_coefficient_that_is_not_finite_skips_the_step(bad):
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    h = hyper()
    c = Case(SIZES, FORMATS["mixed"])
    step = torch.tensor([6, 0], dtype=torch.int32, device="cuda")
    coef = torch.tensor([bad], device="cuda")
    run = B.adamw_mixed_bind(c.P, c.G, c.S, h, c.E, c.C, DECAY, step_dev=step, grad_scale=coef)
    old = [x.clone() for x in c.arrays()]
    run()
    torch.cuda.synchronize()
    assert step.tolist() == [6, 0]
    assert all(torch.equal(x, y) for x, y in zip(old, c.arrays()))
    coef.fill_(0.5)
    before = c.snapshot()
    run()
    torch.cuda.synchronize()
    assert step.tolist() == [7, 0]
    check(c, before, h, 7, 0.5)


def test_learning_rate_from_the_device():
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    c = Case([4099, 300], FORMATS["mixed"])
    lr = torch.tensor([0.002], device="cuda")
    run = B.adamw_mixed_bind(c.P, c.G, c.S, hyper(lr=123.0), c.E, c.C, DECAY, lr_dev=lr)
    for t, x in ((1, 0.002), (2, 0.0005), (3, 0.0)):
        lr.fill_(x)
        before = c.snapshot()
        run(step_now=t)
        torch.cuda.synchronize()
        check(c, before, hyper(lr=float(np.float32(x))), t)


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_gradient_that_is_not_finite(bad, shift):
    """Without a coefficient it reaches its own element; an 8-bit state's block
    reads as NaN from then on, the other blocks are as ever."""
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    h, n, at = hyper(), 1000, 300
    c = Case([n, n], FORMATS["mixed"], shift=shift)
    for g in c.G:
        g[at] = bad
    before = c.snapshot()
    run = B.adamw_mixed_bind(c.P, c.G, c.S, h, c.E, c.C, DECAY)
    run(step_now=4)
    torch.cuda.synchronize()
    after = c.snapshot()
    block = slice(256, 512)
    for i in range(2):
        p = ao.adamw_step(before[i]["p"], before[i]["g"], before[i]["m"], before[i]["v"], h, 4)[0]
        fine = np.arange(n) != at
        assert np.isnan(after[i]["p"][at]) and np.isnan(after[i]["e"][at])
        assert np.allclose(after[i]["p"][fine], p[fine], rtol=1e-5, atol=1e-7)
    assert np.isfinite(after[1]["m"][fine]).all() and not np.isfinite(after[1]["m"][at])
    for key in ("m", "r"):
        assert np.isnan(after[0][key][block]).all()
        assert np.isfinite(np.delete(after[0][key], np.arange(n)[block])).all()
    assert after[0]["mb"].tolist()[1] == ao.NAN_BYTE and after[0]["rb"].tolist()[1] == ao.NAN_BYTE
    for g in c.G:
        g[at] = 0.0
    run(step_now=5)
    torch.cuda.synchronize()
    last = c.snapshot()
    assert np.isnan(last[0]["p"][block]).all() and np.isnan(last[0]["m"][block]).all()
    assert np.isfinite(np.delete(last[0]["p"], np.arange(n)[block])).all()
    c.new.check_guards()


def test_on_another_stream_and_two_calls_at_once():
    """Calls on side streams with counters of their own, at the same time."""
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    h = hyper()
    cases = [Case([200000, 77], FORMATS["mixed"], seed=k) for k in range(3)]
    runs, steps, streams = [], [], []
    for c in cases:
        steps.append(torch.zeros(2, dtype=torch.int32, device="cuda"))
        runs.append(B.adamw_mixed_bind(c.P, c.G, c.S, h, c.E, c.C, DECAY, step_dev=steps[-1]))
        streams.append(torch.cuda.Stream())
    before = [c.snapshot() for c in cases]
    torch.cuda.synchronize()
    for r, s in zip(runs, streams):
        r(stream=s)
    torch.cuda.synchronize()
    for c, b, s in zip(cases, before, steps):
        assert s.tolist() == [1, 0]
        check(c, b, h, 1)


def test_past_32_bits_of_elements():
    """One tensor of 2^32 + 777 elements: the first, the middle (around 2^31 and
    2^32) and the last blocks against the oracle, and the norm of its
    gradient."""
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    n, h = (1 << 32) + 777, hyper()
    p = torch.zeros(n, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    s = B.Adam8State.zeros(n)
    spots = [0, (1 << 31) - 512, (1 << 32) - 768, (1 << 32) + 256]    # apart from each other
    r = np.random.default_rng(0)
    sums = 0.0
    for at in spots:
        k = min(1024, n - at)
        p[at:at + k] = torch.from_numpy(r.standard_normal(k).astype(np.float32))
        g[at:at + k] = torch.from_numpy(r.standard_normal(k).astype(np.float32)).bfloat16()
    sums = sum(float(g[at:at + 1024].double().square().sum()) for at in spots)
    old = [(host(p[at:at + 1024]), host(g[at:at + 1024])) for at in spots]
    out = torch.zeros(2, device="cuda")
    B.grad_norm_batched([g], 1.0, out, B.grad_norm_workspace())
    run = B.adamw_mixed_bind([p], [g], [s], h, grad_scale=out[1:], rounding="stochastic", seed=3)
    run(step_now=1)
    torch.cuda.synchronize()
    assert abs(out[0].item() - sums ** 0.5) <= 1.01 * HALF * sums ** 0.5
    coef = out[1].item()
    words = {}
    for at, (p0, g0) in zip(spots, old):
        k = p0.size
        z = np.zeros(k)
        ref = ao.adamw_step(p0, g0, z, z, h, 1, coef=coef)[0]
        # A = (1-b1) |c g|: S = |c g| / (|c g| + eps) <= 1 on the first step
        tol = 1.01 * HALF * (4 * np.abs(p0) + 21 * h.lr)
        assert np.all(np.abs(host(p[at:at + k]) - ref) <= tol), at
        m32, _, r32 = ao.moments_f32(g0, z, None, h, coef, root=z)
        first = at // ao.BLOCK
        u = np.uint32
        key = ao.mix32(ao.mix32(u(3)) ^ u(0))
        key = ao.mix32(ao.mix32(key ^ u(1)) ^ u(0))
        i = np.arange(k)
        w = ao.mix32(ao.mix32(key ^ (first + i // ao.BLOCK).astype(u)) ^ (i % ao.BLOCK).astype(u))
        bytes_ = host(s.scale[2 * first:2 * (first + -(-k // ao.BLOCK))]).reshape(-1, 2)
        for got, col, x, bits, six in (
                (s.exp_avg, 0, m32, ao.M_BITS, (w & u(0xFFFF)).astype(np.int64)),
                (s.root, 1, r32, ao.R_BITS, (w >> u(16)).astype(np.int64))):
            codes, b = ao.codes_f32(x, bits, six)
            assert np.array_equal(host(got[at:at + k]), codes), at
            assert np.array_equal(bytes_[:, col], b), at
    assert not s.exp_avg[1024:(1 << 31) - 512].any()
    del words


def test_roots_are_correctly_rounded(tmp_path):
    """Every fp32 value from 2^-98 up to the largest: the kernels' square root
    equals the correctly rounded one."""
    import ctypes
    import shutil
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc is not available")
    lib = str(tmp_path / "root_check.so")
    subprocess.run([nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-std=c++17",
                    "-Xcompiler", "-fPIC", "-shared", "--expt-relaxed-constexpr",
                    "-I", os.path.join(root, "muon_optimizer_step_02_b200", "csrc"),
                    "-o", lib, os.path.join(root, "tests", "cpp", "root_check.cu")], check=True)
    check = ctypes.CDLL(lib).root_differences
    check.argtypes, check.restype = [ctypes.c_uint32, ctypes.c_uint32], ctypes.c_longlong
    first, end = (127 - 98) << 23, 255 << 23        # 2^-98, infinity
    assert check(first, end - first) == 0


# ---- the norm -----------------------------------------------------------------

def norm_of(grads, limit=1.0, ws=None):
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    out = torch.full((2,), 9.0, device="cuda")
    B.grad_norm_batched(grads, limit, out, B.grad_norm_workspace() if ws is None else ws)
    return out.tolist()


def near(got, ref):
    """A 64-bit value rounded once: half a step, and 1e-9 for the sum's order."""
    return abs(got - ref) <= HALF * (1 + 1e-3) * abs(ref) + 1e-9 * abs(ref) + 1e-45


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("kind", ["f32", "bf16", "both"])
@pytest.mark.parametrize("sizes", [[1], [0, 3], [255, 256, 257], [70001, 0, 5, 4096],
                                   [(3 * i) % 301 for i in range(2700)]])
def test_norm_matches_the_oracle(sizes, kind, shift):
    import torch
    new = Arrays(shift)
    r = np.random.default_rng(len(sizes))
    grads = []
    for i, n in enumerate(sizes):
        g = torch.from_numpy((r.standard_normal(n) * 10.0 ** r.integers(-4, 2)).astype(np.float32))
        grads.append(new.tensor(g.bfloat16() if kind == "bf16" or (kind == "both" and i % 2) else g))
    for limit in (1e-3, 1e9, float("inf")):
        norm, coef = ao.grad_norm([host(g) for g in grads], limit)
        got = norm_of(grads, limit)
        assert near(got[0], norm) and near(got[1], coef)
    new.check_guards()


@pytest.mark.parametrize("scale", [1e-30, 1e25, 3e38])
def test_norm_of_extreme_gradients(scale):
    import torch
    g = np.full(1000, scale, np.float32)
    norm, coef = ao.grad_norm([g], 1e-3)
    got = norm_of([torch.from_numpy(g).cuda()], 1e-3)
    assert got[0] == np.float32(norm) if norm < 3.4e38 else got[0] == np.inf
    assert near(got[1], coef)


def test_norm_of_nothing_and_of_bad_gradients():
    import torch
    assert norm_of([]) == [0.0, 1.0]
    assert norm_of([torch.zeros(1000, device="cuda")], 1e-7) == [0.0, float(np.float32(1e-7 / 1e-6))]
    for bad in (float("inf"), -float("inf"), float("nan")):
        for dtype in (torch.float32, torch.bfloat16):
            g = torch.ones(5000, dtype=dtype, device="cuda")
            g[4321] = bad
            norm, coef = norm_of([torch.ones(3, device="cuda"), g])
            assert not np.isfinite(norm) and np.isnan(coef)


def test_norm_is_deterministic_and_its_workspace_returns_ready():
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    r = torch.Generator(device="cuda").manual_seed(1)
    g = [torch.randn(n, generator=r, device="cuda") for n in (3 << 20, 777, 12345)]
    ws = B.grad_norm_workspace()
    first = norm_of(g, 0.5, ws)
    out = torch.zeros(2, device="cuda")
    run = B.grad_norm_bind(g, 0.5, out, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(5):
        out.zero_()
        graph.replay()
        assert out.tolist() == first and norm_of(g, 0.5, ws) == first
    assert norm_of(g[1:], 0.5, ws) != first
    del graph


# ---- states in and out --------------------------------------------------------

def state(codes_m, codes_r, bytes_, new):
    from muon_optimizer_step_02_b200 import binding as B
    return B.Adam8State(new(codes_m.astype(np.uint8)), new(codes_r.astype(np.uint8)),
                        new(bytes_.astype(np.uint8)))


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_reading_every_code_under_every_byte(dtype, shift):
    """All 256 codes under all 256 scale bytes (those past 245 read as NaN),
    exact in both types; bf16 as far as its own range goes (bytes from 20)."""
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    new = Arrays(shift)
    codes = np.tile(np.arange(256), 256)
    byte = np.arange(256)
    s = state(codes, codes, np.stack([byte, byte], 1).reshape(-1), new)
    kind = torch.float32 if dtype == "f32" else torch.bfloat16
    m, v = (new.tensor(torch.zeros(codes.size, dtype=kind)) for _ in range(2))
    B.adam8_read_batched([s], [m], [v])
    torch.cuda.synchronize()
    want_m, want_r = ao.decode(codes, byte, ao.M_BITS), ao.decode(codes, byte, ao.R_BITS)
    with np.errstate(over="ignore", under="ignore"):
        want_v = (want_r.astype(np.float32) ** 2) if dtype == "f32" else want_r
    use = np.repeat(byte >= ao.LOW, 256)
    for got, want in ((m, want_m), (v, want_v)):
        got, want = host(got)[use], np.asarray(want, np.float64)[use]
        assert np.array_equal(np.isnan(got), np.isnan(want))
        ok = ~np.isnan(want)
        assert np.array_equal(got[ok], want[ok])
    new.check_guards()


@pytest.mark.parametrize("shift", [0, 1, None])
@pytest.mark.parametrize("sizes", [SIZES, [(5 * i) % 41 for i in range(1100)],
                                   [1024 * (9 + i % 7) + 100 * (i % 3) for i in range(450)]])
def test_writing_and_reading_back(sizes, shift):
    """fp32 moments to the nearest codes, bit for bit; read back in bf16 and
    written again they give the same values; a state read in fp32 squares its
    roots."""
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    new = Arrays()
    states, M, V, M16, R16 = [], [], [], [], []
    for i, n in enumerate(sizes):
        new.shift = (0, 1, 0, 4, 8)[i % 5] if shift is None else shift
        _, m, v, _ = wl.adamw_state(n, i, 3, wid=301)
        M.append(new(m))
        V.append(new(v))
        M16.append(new.tensor(torch.zeros(n, dtype=torch.bfloat16)))
        R16.append(new.tensor(torch.zeros(n, dtype=torch.bfloat16)))
        states.append(state(np.full(n, 5), np.full(n, 5), np.full(2 * -(-n // 256), 5), new))
    B.adam8_write_batched(states, M, V)
    B.adam8_read_batched(states, M16, R16)
    torch.cuda.synchronize()
    for i, s in enumerate(states):
        b = host(s.scale).reshape(-1, 2)
        for got, byte, x, bits, value in ((s.exp_avg, b[:, 0], host(M[i]), ao.M_BITS, M16[i]),
                                          (s.root, b[:, 1], np.sqrt(host(V[i])), ao.R_BITS, R16[i])):
            codes, want = ao.codes_f32(x, bits)
            assert np.array_equal(host(got), codes) and np.array_equal(byte, want), i
            assert np.array_equal(host(value), ao.decode(codes, want, bits)), i
    again = [state(np.full(n, 9), np.full(n, 9), np.full(2 * -(-n // 256), 9), new) for n in sizes]
    B.adam8_write_batched(again, M16, R16)
    M2, R2 = ([new.tensor(torch.zeros_like(x)) for x in y] for y in (M16, R16))
    B.adam8_read_batched(again, M2, R2)
    B.adam8_read_batched(states, M, V)
    torch.cuda.synchronize()
    for i in range(len(sizes)):
        assert torch.equal(M2[i], M16[i]) and torch.equal(R2[i], R16[i])
        assert torch.equal(M[i], M16[i].float()) and torch.equal(V[i], R16[i].float().square())
    new.check_guards()


def test_writing_what_is_no_moment():
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    for dtype in (torch.float32, torch.bfloat16):
        s = B.Adam8State.zeros(768)
        m, v = torch.ones(768, dtype=dtype, device="cuda"), torch.ones(768, dtype=dtype, device="cuda")
        v[3] = -1.0
        m[300] = float("nan")
        v[300] = float("inf")
        m[700], v[700] = -0.0, -0.0
        B.adam8_write_batched([s], [m], [v])
        M, V = torch.zeros(768, device="cuda"), torch.zeros(768, device="cuda")
        B.adam8_read_batched([s], [M], [V])
        torch.cuda.synchronize()
        assert bool(V[:256].isnan().all()) and bool((M[:256] == 1).all())
        assert bool(V[256:512].isnan().all()) and bool(M[256:512].isnan().all())
        assert M[700].item() == 0 and V[700].item() == 0 and bool((V[512:700] == 1).all())


# ---- what runs before and after, on the stream and in graphs --------------------

def _chain(B, c, h):
    """norm -> clipped step -> read-back of one case, as bound calls."""
    import torch
    out = torch.zeros(2, device="cuda")
    step = torch.zeros(2, dtype=torch.int32, device="cuda")
    m = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in c.sizes]
    r = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in c.sizes]
    calls = (B.grad_norm_bind(c.G, 0.01, out, B.grad_norm_workspace()),
             B.adamw_mixed_bind(c.P, c.G, c.S, h, c.E, c.C, DECAY, step_dev=step,
                                grad_scale=out[1:], rounding="stochastic", seed=4),
             B.adam8_read_bind(c.S, m, r))
    return calls, [out, step, *m, *r, *c.arrays()]


@pytest.mark.parametrize("n", [1000, 3 << 20])
def test_calls_see_what_ran_before_them(n):
    """The kernels may be set up while what precedes them still runs: each of a
    copy, a fill, a library kernel, a plain kernel of another stream and a
    call of the same kind, eagerly and in a graph, is seen whole; and what
    follows sees the calls' results."""
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    h = hyper(beta2=0.99)
    sizes = [n, 77]
    ref, eager, graphed = (Case(sizes, FORMATS["8"], seed=2) for _ in range(3))
    src = [torch.from_numpy(wl.adamw_grad(k, i, 7, 2, wid=300)).cuda() for i, k in enumerate(sizes)]
    big = torch.randn(2048, 2048, device="cuda")

    def program(c, calls, after, wait):
        side = torch.cuda.Stream()
        norm, step, read = calls

        def passes():
            for g, x in zip(c.G, src):
                g.copy_(x)                       # a copy, then the norm
            wait()
            norm()
            wait()
            step()
            wait()
            c.G[0].fill_(0.25)                   # a fill, then the norm
            wait()
            norm()
            wait()
            step()
            wait()
            y = big @ big                        # a library's product, then the step
            c.G[1].copy_(y[0, :77] * 1e-3)
            wait()
            step()
            wait()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):        # another stream's work, joined
                c.G[0].mul_(0.5)
                c.G[1].add_(1e-3)
            torch.cuda.current_stream().wait_stream(side)
            wait()
            norm()
            wait()
            step()
            wait()
            step()
            wait()
            read()
            wait()
            after[0].copy_(c.P[0])               # a kernel that reads the results
            after[1].copy_(c.G[0] * 2)
        return passes

    results = []
    for c, how in ((ref, "waits"), (eager, "eager"), (graphed, "graph")):
        calls, arrays = _chain(B, c, h)
        after = [torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")]
        run = program(c, calls, after, torch.cuda.synchronize if how == "waits" else lambda: None)
        if how == "graph":
            run()                                # workspaces of the product, once
            torch.cuda.synchronize()
            fresh = Case(sizes, FORMATS["8"], seed=2)
            for x, y in zip(c.arrays(), fresh.arrays()):
                x.copy_(y)
            arrays[1].zero_()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                run()
            graph.replay()
            torch.cuda.synchronize()
            del graph
        else:
            run()
            torch.cuda.synchronize()
        results.append(arrays + after)
    for x, y, z in zip(*results):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_first_calls_of_a_process_may_be_captured():
    """A process whose first calls are captured ones: no warm-up is needed."""
    import subprocess
    import sys
    code = """
import types, torch
from muon_optimizer_step_02_b200 import binding as B
h = types.SimpleNamespace(lr=0.01, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
def side():
    g = torch.Generator(device="cuda").manual_seed(1)
    P = [torch.randn(n, generator=g, device="cuda") for n in (5000, 300)]
    G = [torch.randn(n, generator=g, device="cuda") for n in (5000, 300)]
    S = [B.Adam8State.zeros(5000), (torch.zeros(300, device="cuda"), torch.zeros(300, device="cuda"))]
    out, step = torch.zeros(2, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    V = [torch.ones(5000, device="cuda") for _ in range(2)]
    calls = [B.adam8_write_bind(S[:1], V[:1], V[1:]), B.grad_norm_bind(G, 1.0, out, B.grad_norm_workspace()),
             B.adamw_mixed_bind(P, G, S, h, step_dev=step, grad_scale=out[1:], rounding="stochastic"),
             B.adam8_read_bind(S[:1], V[:1], V[1:])]
    return calls, [*P, S[0].exp_avg, S[0].root, S[0].scale, *S[1], out, step, *V]
calls, a = side()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for c in calls:
        c()
graph.replay()
torch.cuda.synchronize()
calls, b = side()
for c in calls:
    c()
torch.cuda.synchronize()
assert b[-3].tolist() == [1, 0], b[-3]
assert all(torch.equal(x, y) for x, y in zip(a, b))
print("captured first")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                         timeout=300)
    assert res.returncode == 0 and "captured first" in res.stdout, res.stderr[-2000:]


def test_interleaved_with_the_other_optimizer_calls():
    """Between Muon steps (whose tensor-core kernel is itself a dependent
    launch), with 0 and 5 Newton-Schulz steps, and EMA passes: bit for bit what
    the same calls give with waits between them."""
    import torch
    from gpu_harness import GpuMuon
    from muon_optimizer_step_02_b200 import binding as B
    h, ah = wl.Hyper(momentum=0.95, lr=0.02, weight_decay=0.1), hyper()
    results = []
    for wait in (torch.cuda.synchronize, lambda: None):
        kept = []
        for coeffs in ([wl.FIXED_QUINTIC] * 5, []):
            w = wl.custom([(512, 256), (128, 384)], h, coeffs, name="interleaved")
            mu = GpuMuon(w, with_out=False)
            mg = mu.grads(0)
            c = Case([4099, 512], FORMATS["mixed"])
            calls, arrays = _chain(B, Case([3000], FORMATS["8"]), ah)
            em = [x.clone().view(-1) for x in mu.W]
            adam = B.adamw_mixed_bind(c.P, c.G, c.S, ah, c.E, c.C, DECAY)
            for t in range(1, 4):
                for call in (calls[0], lambda: mu.step(mg), lambda: adam(step_now=t), calls[1],
                             lambda: B.ema_update_batched(em, [x.view(-1) for x in mu.W], DECAY),
                             calls[2], lambda: mu.step(mg), calls[1]):
                    call()
                    wait()
            torch.cuda.synchronize()
            assert mu.plan.last_error() == 0
            kept += [*mu.W, *mu.M, *em, *c.arrays(), *arrays]
            mu.plan.close()
        results.append(kept)
    for x, y in zip(*results):
        assert torch.equal(x, y)


# ---- refusals that need device tensors ----------------------------------------

def test_binding_refusals():
    import torch
    from muon_optimizer_step_02_b200 import binding as B
    f = lambda n, d=torch.float32: torch.zeros(n, dtype=d, device="cuda")  # noqa: E731
    h, s8 = hyper(), B.Adam8State.zeros(300)

    def bad(match, *a, **kw):
        with pytest.raises(ValueError, match=match):
            B.adamw_mixed_bind(*a, **kw)
    p, g = f(300), f(300)
    bad("expected 300", [p], [f(299)], [s8], h)
    bad("params", [f(300, torch.bfloat16)], [g], [s8], h)
    bad("grads", [p], [f(300, torch.float16)], [s8], h)
    bad("contiguous", [f(600)[::2]], [g], [s8], h)
    bad("expected 300", [p], [g], [B.Adam8State.zeros(299)], h)
    bad("emas", [p], [g], [s8], h, emas=[f(300, torch.bfloat16)])
    bad("copies", [p], [g], [s8], h, copies=[f(300)])
    bad("overlaps", [p], [g], [s8], h, emas=[p])
    bad("overlaps", [p], [p], [s8], h)
    bad("overlaps", [p, f(300)], [g, g], [s8, s8], h)
    bad("overlaps", [p], [g], [s8], h, grad_scale=p[:1])
    bad("step_dev", [p], [g], [s8], h, step_dev=f(1, torch.int32))
    bad("lr_dev", [p], [g], [s8], h, lr_dev=f(1, torch.float64))
    B.adamw_mixed_bind([p, f(300)], [g, g], [s8, (f(300), f(300))], h)     # one gradient read twice
    with pytest.raises(ValueError, match="scale"):
        B.Adam8State(s8.exp_avg, s8.root, f(3, torch.uint8))
    with pytest.raises(ValueError, match="expected"):
        B.Adam8State(s8.exp_avg, f(299, torch.uint8), s8.scale)
    ws = B.grad_norm_workspace()
    for a in (([f(3, torch.float16)], 1.0, f(2), ws), ([g], 1.0, f(3), ws),
              ([ws.view(torch.float32)], 1.0, f(2), ws), ([g], 1.0, g[:2], ws)):
        with pytest.raises(ValueError):
            B.grad_norm_bind(*a)
    for call in (lambda: B.grad_norm_batched([g], -1.0, f(2), ws),
                 lambda: B.grad_norm_batched([g], 1.0, f(2), ws[:100]),
                 lambda: B.adamw_mixed_bind([p], [g], [s8], h)(step_now=0)):
        with pytest.raises(B.MuonError):
            call()
    with pytest.raises(ValueError, match="exp_avgs"):
        B.adam8_write_bind([s8], [f(299)], [f(300)])
    with pytest.raises(ValueError, match="seconds"):
        B.adam8_write_bind([s8], [f(300)], [f(300, torch.bfloat16)])
    with pytest.raises(ValueError, match="overlaps"):
        B.adam8_read_bind([s8], [p], [p])


# ---- together -----------------------------------------------------------------

def test_clip_muon_adamw_and_averages_in_one_graph():
    """A training step as it is used: the norm of all gradients, the Muon step
    of the matrices with their EMA, and the clipped AdamW step of the rest
    (8-bit table, 32-bit vectors), captured once and replayed; against the
    same steps made eagerly, and each AdamW step against the oracle.  A step
    with a bad gradient leaves what AdamW keeps untouched."""
    import torch
    from gpu_harness import GpuMuon
    from muon_optimizer_step_02_b200 import binding as B
    h, ah = wl.Hyper(momentum=0.95, lr=0.02, weight_decay=0.1), hyper(beta2=0.99)
    w = wl.custom([(128, 64), (64, 192)], h, [wl.FIXED_QUINTIC] * 5, name="together")
    kw = dict(ema_decay=DECAY, rounding="stochastic", seed=11)

    class Side:
        def __init__(self):
            self.mu = GpuMuon(w, with_out=False)
            self.mg = self.mu.grads(0)
            self.rest = Case([64 * 512, 512, 512, 1], lambda i: i == 0, "bf16")
            self.em = [x.clone().view(-1) for x in self.mu.W]
            self.out = torch.zeros(2, device="cuda")
            self.step = torch.zeros(2, dtype=torch.int32, device="cuda")
            r = self.rest
            self.norm = B.grad_norm_bind(self.mg + r.G, 0.1, self.out, B.grad_norm_workspace())
            self.muon = self.mu.plan.bind(self.mu.W, self.mu.M, self.mg, h, w.coeffs, self.mu.ws,
                                          self.mu.scales)
            self.adam = B.adamw_mixed_bind(r.P, r.G, r.S, ah, r.E, r.C, step_dev=self.step,
                                           grad_scale=self.out[1:], **kw)
            self.avg = B.ema_bind(self.em, [x.view(-1) for x in self.mu.W], DECAY)

        def grads(self, t):
            for a, b in zip(self.mg, self.mu.grads(t)):
                a.copy_(b)
            self.rest.set_grads(t)

        def __call__(self):
            self.norm()
            self.muon()
            self.adam()
            self.avg()

        def arrays(self):
            return [*self.mu.W, *self.mu.M, *self.em, self.out, self.step, *self.rest.arrays()]

    a, b = Side(), Side()
    for s in (a, b):
        s.grads(1)
    before = a.rest.snapshot()
    a()
    b()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b()
    for t in range(1, 5):
        norm, coef = ao.grad_norm([host(g) for g in a.mg + a.rest.G], 0.1)
        assert near(a.out[0].item(), norm) and near(a.out[1].item(), coef) and coef < 1
        check(a.rest, before, ah, t, a.out[1].item(), rounding="stochastic", seed=11)
        for x, y in zip(a.arrays(), b.arrays()):
            assert torch.equal(x, y)
        for s in (a, b):
            s.grads(t + 1)
        before = a.rest.snapshot()
        a()
        graph.replay()
        torch.cuda.synchronize()
    b.rest.G[1][7] = float("inf")
    old = [x.clone() for x in (*b.rest.arrays(), b.step)]
    graph.replay()
    torch.cuda.synchronize()
    assert np.isnan(b.out[1].item())
    assert all(torch.equal(x, y) for x, y in zip(old, (*b.rest.arrays(), b.step)))
    del graph
    for s in (a, b):
        assert s.mu.plan.last_error() == 0
        s.mu.plan.close()
