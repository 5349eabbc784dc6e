"""The cases on which the AdamW step with 8-bit or 32-bit states, the gradient norm it clips
with, and the conversions of its 8-bit states are measured.

Every tensor list lies in arenas: one flat buffer for each kind of array, every tensor starting on
a block of 256 elements, the rest of its last block zero.  A program that keeps its parameters in
flat buffers does the same; the plain forms then need no loop over tensors, and the framework's
calls take the tensors one by one, as views.
"""

import math
import random

import numpy as np
import torch

own = False

DEVICE = "cuda"
BLOCK = 256          # elements that share one scale
M_BITS, R_BITS = 4, 5   # mantissa bits of the first moment's codes and of the root's
LOW, HIGH = 20, 245  # the range of a block's scale byte

LR, BETA1, EPS, DECAY, EMA = 1e-3, 0.9, 1e-8, 0.1, 0.9965
MAX_NORM = 1.0
SEED = 0x5DEECE66D1234567   # of the random bits of stochastic rounding
EIGHT_FROM = 4096    # "mixed": tensors from this size on have 8-bit states


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------

def listed():
    """`set`: whose tensors; `grad`: their gradients' type; `bits`: of the states; `clip`: the
    norm of all gradients is taken first and scales them; `taken`: steps taken before."""
    return [
        # the least a call can do: the gradient of one vector of the 24L model
        {"name": "norm one vector", "op": "norm", "set": "one", "size": 2048, "grad": "f32", "shift": 0},
        # the whole 11L model: bf16 gradients of the matrices, fp32 of the rest
        {"name": "norm 11L", "op": "norm", "set": "11L all", "size": 0, "grad": "both", "shift": 0},
        # the 16L model's matrices, 184 million bf16 gradients
        {"name": "norm 16L matrices", "op": "norm", "set": "16L matrices", "size": 0, "grad": "bf16", "shift": 0},
        # the vectors and scalars that stay in 32 bits beside 8-bit embeddings: 210 small tensors
        adamw("adamw 32 vectors", "11L vectors", "32", grad="f32", ema=True),
        # the 11L model's non-matrix tensors from bf16 gradients, clipped, with the copy that the forward pass reads
        adamw("adamw 32 11L clipped", "11L", "32", grad="bf16", ema=True, copy=True, clip=True),
        # one small tensor of an odd size, the first step
        adamw("adamw 8 one tensor", "one", "8", size=4099, grad="f32", taken=0),
        # the 11L model's non-matrix tensors with fp32 gradients and the average
        adamw("adamw 8 11L", "11L", "8", grad="f32", ema=True),
        # the 24L model: its embedding in 8 bits, its vectors in 32, in one call, clipped
        adamw("adamw mixed 24L clipped", "24L", "mixed", grad="bf16", ema=True, copy=True, clip=True, stochastic=True, beta2=0.999),
        # a large embedding table, 65,536 x 1024
        adamw("adamw 8 large table", "one", "8", size=65536 * 1024, grad="bf16", copy=True, stochastic=True, beta2=0.99),
        # odd sizes that start off a 16-byte boundary: views into somebody else's buffers
        adamw("adamw mixed unaligned", "spread", "mixed", size=1 << 18, count=40, grad="bf16", stochastic=True, shift=1),
        # a 32-bit run moved over to 8-bit states, and their values read back for a checkpoint
        {"name": "convert 11L", "op": "convert", "set": "11L", "size": 0, "count": 0, "pick": 0, "shift": 0},
        # the same for a few odd sizes
        {"name": "convert odd sizes", "op": "convert", "set": "spread", "size": 1 << 16, "count": 7, "pick": 3, "shift": 0},
    ]


def adamw(name, tensors, bits, size=0, count=0, pick=1, grad="f32", ema=False, copy=False, clip=False, stochastic=False,
          beta2=0.95, taken=9, shift=0):
    return {"name": name, "op": "adamw", "set": tensors, "bits": bits, "size": size, "count": count, "pick": pick,
            "grad": grad, "ema": ema, "copy": copy, "clip": clip, "stochastic": stochastic, "beta2": beta2, "taken": taken,
            "shift": shift}


def draw(rng):
    size = int(round(math.exp(rng.uniform(0.0, math.log(1 << 24)))))
    count = int(round(math.exp(rng.uniform(0.0, math.log(600)))))
    spread = {"set": "spread", "size": size, "count": count, "pick": rng.randrange(1 << 20), "shift": rng.choice([0, 0, 1])}
    op = rng.choice(["norm", "adamw", "adamw", "adamw", "convert"])
    if op == "norm":
        return {"op": op, "grad": rng.choice(["f32", "bf16"]), **spread}
    if op == "convert":
        return {"op": op, **spread}
    grad = rng.choice(["f32", "bf16"])
    # the first step from empty states only with fp32 gradients: a tenth of a bf16 value often lies half-way between two codes,
    # where 32 and 64 bits may take either
    return {"op": op, "bits": rng.choice(["8", "8", "32", "mixed"]), "grad": grad,
            "ema": rng.random() < 0.5, "copy": rng.random() < 0.5, "clip": rng.random() < 0.4,
            "stochastic": rng.random() < 0.5, "beta2": rng.choice([0.95, 0.99, 0.999]),
            "taken": rng.choice([9, 999, 100000] + [0] * (grad == "f32")), **spread}


def gpt_matrices(layers, d, kv):
    return [d * d, kv * d, kv * d, d * d, 4 * d * d, 4 * d * d] * layers


def sizes(case):
    """The numbers of elements of the case's tensors."""
    which = case["set"]
    vectors = [512] * 118 + [1] * 92
    if which == "one":
        return [case["size"]]
    if which == "11L vectors":
        return vectors
    if which == "11L":
        return [8192 * 512, 4096 * 512] + vectors
    if which == "11L all":
        return gpt_matrices(11, 512, 256) + [8192 * 512, 4096 * 512] + vectors
    if which == "16L matrices":
        return gpt_matrices(16, 1024, 512)
    if which == "24L":
        return [8192 * 2048] + [2048] * 96
    pick, got, left = random.Random(case["pick"]), [case["size"]], 48 << 20
    for _ in range(case["count"] - 1):
        n = int(round(math.exp(pick.uniform(0.0, math.log(max(2, case["size"]))))))
        left -= n
        if left < 0:
            break
        got.append(n)
    return got


def parts(case):
    """[(bits, [(place in the call, number of elements)])]: the tensors of each state format."""
    every = list(enumerate(sizes(case)))
    if case["bits"] != "mixed":
        return [(int(case["bits"]), every)]
    big = [x for x in every if x[1] >= EIGHT_FROM]
    small = [x for x in every if x[1] < EIGHT_FROM]
    return [(b, p) for b, p in ((8, big), (32, small)) if p]


def work(case):
    n = sum(sizes(case))
    if case["op"] == "norm":
        wide = sum(sizes(case)[66:]) if case["grad"] == "both" else n if case["grad"] == "f32" else 0
        return {"bytes": 4 * wide + 2 * (n - wide) + 8, "flops": 2 * n}
    if case["op"] == "convert":
        # both moments in 32 bits read; codes and scales written; their values in bf16 written
        return {"bytes": n * (8 + 2 + 4) + n / 128, "flops": 20 * n}
    # parameter in and out, gradient, average in and out, copy out
    per = 8 + (4 if case["grad"] == "f32" else 2) + (8 if case["ema"] else 0) + (2 if case["copy"] else 0)
    moved, flops = n * per, 0
    for bits, some in parts(case):
        k = sum(x[1] for x in some)
        # both moments in and out; for 8 bits the scales too, and the values they stand for
        moved += k * 16 if bits == 32 else k * (4 + 4) + 4 * k / BLOCK
        flops += k * (16 if bits == 32 else 40)
    return {"bytes": moved, "flops": flops + (2 * n if case["clip"] else 0)}


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

class Arena:
    """Where the tensors of one list lie in flat buffers, and what of it the plain forms go by."""

    def __init__(self, some, shift):
        self.some, self.shift = some, shift
        blocks = [-(-n // BLOCK) for _, n in some]
        self.first = np.concatenate([[0], np.cumsum(blocks)])
        self.blocks = int(self.first[-1])
        per = torch.tensor(blocks)
        rows = lambda v: torch.repeat_interleave(torch.tensor(v), per).to(DEVICE)  # noqa: E731
        self.tensor = rows([i for i, _ in some])                          # of each block: its tensor's place in the call,
        self.number = torch.arange(self.blocks, device=DEVICE) - rows(self.first[:-1].tolist())  # its place in the tensor,
        left = rows([n for _, n in some]) - BLOCK * self.number           # and the elements that are the tensor's
        self.there = torch.arange(BLOCK, device=DEVICE) < left[:, None]
        # small tensors (vectors, scalars) are not decayed; the first tensor learns at half the rate
        self.lr = rows([0.5 if i == 0 else 1.0 for i, _ in some])[:, None]
        self.wd = rows([0.0 if n < EIGHT_FROM else 1.0 for _, n in some])[:, None]

    def buffer(self, values):
        """`values` (blocks x 256) as a flat buffer, `shift` elements off its allocation's start."""
        held = torch.zeros(values.numel() + self.shift, dtype=values.dtype, device=DEVICE)
        held[self.shift:] = values.reshape(-1)
        return held[self.shift:]

    def views(self, flat, unit=BLOCK):
        """The tensors of a buffer of `unit` elements a block."""
        return [flat[f * unit:f * unit + (n if unit == BLOCK else -(-n // BLOCK) * unit)]
                for f, (_, n) in zip(self.first.tolist(), self.some)]


def gradients(arena, g, kind, scale):
    """Gradients of rows of very different size; a tenth of the rows saw no token and have none."""
    v = torch.randn(arena.blocks, BLOCK, generator=g, device=DEVICE) * scale
    seen = torch.rand(arena.blocks, 1, generator=g, device=DEVICE) >= 0.1
    v = v * (arena.there & seen)
    return arena.buffer(v if kind == "f32" else v.to(torch.bfloat16))


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    s = {"case": case, "arenas": []}
    if case["op"] == "norm":
        every = list(enumerate(sizes(case)))
        lists = [("bf16", every[:66]), ("f32", every[66:])] if case["grad"] == "both" else [(case["grad"], every)]
        for kind, some in lists:
            a = Arena(some, case["shift"])
            scale = 1e-3 * torch.exp(torch.randn(a.blocks, 1, generator=g, device=DEVICE))
            s["arenas"].append({"arena": a, "grad": gradients(a, g, kind, scale)})
        s["norm"] = torch.zeros(2, device=DEVICE)
    elif case["op"] == "convert":
        a = Arena(list(enumerate(sizes(case))), case["shift"])
        m, v = moments(a, g, 1e-3 * torch.exp(torch.randn(a.blocks, 1, generator=g, device=DEVICE)))
        nothing = torch.zeros(a.blocks, BLOCK, dtype=torch.uint8, device=DEVICE)
        s["arenas"].append({"arena": a, "m": a.buffer(m), "v": a.buffer(v), "m8": a.buffer(nothing), "r8": a.buffer(nothing),
                            "scale": a.buffer(nothing[:, :2]), "m_value": a.buffer(nothing.bfloat16()),
                            "r_value": a.buffer(nothing.bfloat16())})
    else:
        for bits, some in parts(case):
            a = Arena(some, case["shift"])
            scale = 1e-3 * torch.exp(torch.randn(a.blocks, 1, generator=g, device=DEVICE))
            p = torch.randn(a.blocks, BLOCK, generator=g, device=DEVICE) * 0.02 * a.there
            d = {"arena": a, "bits": bits, "p": a.buffer(p), "grad": gradients(a, g, case["grad"], scale)}
            m, v = moments(a, g, scale)
            if case["taken"] == 0:
                m, v = m * 0, v * 0
            if bits == 8:
                (m8, me), (r8, re) = encode(m, M_BITS), encode(v.sqrt(), R_BITS)
                d |= {"m8": a.buffer(m8), "r8": a.buffer(r8), "scale": a.buffer(torch.cat([me, re], 1).to(torch.uint8)),
                      "m_value": a.buffer(torch.zeros_like(m, dtype=torch.bfloat16)),
                      "r_value": a.buffer(torch.zeros_like(m, dtype=torch.bfloat16))}
            else:
                d |= {"m": a.buffer(m), "v": a.buffer(v)}
            if case["ema"]:
                d["ema"] = a.buffer(p + torch.randn(a.blocks, BLOCK, generator=g, device=DEVICE) * 1e-3 * a.there)
            if case["copy"]:
                d["copy"] = a.buffer(p.bfloat16())
            s["arenas"].append(d)
        s["norm"] = torch.zeros(2, device=DEVICE)
        s["step"] = torch.tensor([case["taken"], 0], dtype=torch.int32, device=DEVICE)  # steps taken; a word of the call's
    if own:
        bind(s)
    return s


def moments(arena, g, scale):
    """Both moments as after some steps: the second near the square of the gradients' size; rows of tokens never seen have none."""
    seen = (torch.rand(arena.blocks, 1, generator=g, device=DEVICE) >= 0.03) & arena.there
    m = 0.4 * scale * torch.randn(arena.blocks, BLOCK, generator=g, device=DEVICE)
    v = scale * scale * (0.1 + torch.randn(arena.blocks, BLOCK, generator=g, device=DEVICE) ** 2)
    return m * seen, v * seen


def bind(s):
    """What a program does once, before its loop: the framework's calls with their arguments marshalled."""
    from muon_optimizer_step_02_b200 import binding as B

    class Hyper:
        lr, beta1, beta2, eps, weight_decay = LR, BETA1, s["case"].get("beta2", 0.95), EPS, DECAY

    def gathered(key, unit=BLOCK):
        """The views of one kind of array, in the order of the call."""
        found = {}
        for d in s["arenas"]:
            a = d["arena"]
            found |= {i: v for (i, _), v in zip(a.some, a.views(d[key], unit))} if key in d else {i: None for i, _ in a.some}
        return [found[i] for i in sorted(found)]

    case = s["case"]
    if case["op"] == "norm" or case.get("clip"):
        s["run_norm"] = B.grad_norm_bind(gathered("grad"), MAX_NORM, s["norm"], B.grad_norm_workspace())
    if case["op"] == "norm":
        return
    states = [B.Adam8State(m, r, c) if m is not None else None
              for m, r, c in zip(gathered("m8"), gathered("r8"), gathered("scale", 2))]
    eight = [i for i, x in enumerate(states) if x is not None]
    if eight:
        values = [[x[i] for i in eight] for x in (gathered("m_value"), gathered("r_value"))]
        s["run_read"] = B.adam8_read_bind([states[i] for i in eight], *values)
    if case["op"] == "convert":
        s["run_write"] = B.adam8_write_bind(states, gathered("m"), gathered("v"))
        return
    states = [x if x is not None else (m, v) for x, m, v in zip(states, gathered("m"), gathered("v"))]
    n = sizes(case)
    s["run_step"] = B.adamw_mixed_bind(
        gathered("p"), gathered("grad"), states, Hyper, emas=gathered("ema"), copies=gathered("copy"), ema_decay=EMA,
        step_dev=s["step"], grad_scale=s["norm"][1:] if case["clip"] else None,
        lr_scales=[0.5 if i == 0 else 1.0 for i in range(len(n))], wd_scales=[0.0 if k < EIGHT_FROM else 1.0 for k in n],
        rounding="stochastic" if case["stochastic"] else "nearest", seed=SEED)


# ---------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------

def run(s):
    case = s["case"]
    if case["op"] == "norm":
        if own:
            s["run_norm"]()
        else:
            s["norm"].copy_(plain_norm(s))
        return {"norm": s["norm"]}
    if case["op"] == "convert":
        if own:
            s["run_write"]()
            s["run_read"]()
        else:
            d = s["arenas"][0]
            (m8, me), (r8, re) = (encode(blocks(d["m"]), M_BITS), encode(blocks(d["v"]).sqrt(), R_BITS))
            keep(d, m8, me, r8, re)
        return states(s)
    if own:
        if case["clip"]:
            s["run_norm"]()
        s["run_step"]()
        if "run_read" in s:
            s["run_read"]()
    else:
        if case["clip"]:
            s["norm"].copy_(plain_norm(s))
        s["step"][0] += 1
        for d in s["arenas"]:
            plain_adamw(case, d, s["norm"][1] if case["clip"] else None, s["step"][0])
    return states(s)


def states(s):
    """The arrays that a pass writes; 8-bit states as the values that they stand for, which bf16 holds exactly."""
    out = {"taken": s["step"][:1]} if "step" in s else {}
    if s["case"].get("clip"):
        out["norm"] = s["norm"]
    for k, d in enumerate(s["arenas"]):
        written = ("m_value", "r_value") if "m8" in d else ("m", "v")
        out |= {"%s %d" % (key, k): d[key] for key in ("p", "ema", "copy", *written) if key in d}
    return out


def blocks(flat, unit=BLOCK):
    return flat.view(-1, unit)


def plain_norm(s):
    """The norm of all gradients together and the factor that brings it to MAX_NORM at most; a long sum: in 64 bits."""
    total = sum(d["grad"].double().square().sum() for d in s["arenas"])
    norm = total.sqrt()
    return torch.stack([norm, (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)]).float()


def power(e):
    """2^(e - 127) for whole e from 1 to 254."""
    return (e.int() << 23).view(torch.float32)


def encode(x, bits, random_bits=None):
    """Codes of 3 exponent bits and `bits` mantissa bits (and the sign, where x has one) for blocks x 256 values of 32 bits,
    and the blocks' scale bytes.  A byte is the exponent of the top codes' values, biased by 127: the least that holds
    the block's largest.  What is rounded is a definite function of the 32-bit values: the bits below the code in the pattern of
    x scaled so that the codes' subnormal numbers are the type's own."""
    low = 23 - bits
    largest = x.abs().amax(1, keepdim=True).view(torch.int32)
    e = ((largest + ((1 << low) - 1)) >> 23).clamp(min=LOW)
    pattern = (x.abs() * power(246 - e) * 2.0 ** -112).view(torch.int32)
    if random_bits is None:
        pattern = pattern + ((1 << (low - 1)) - 1) + ((pattern >> low) & 1)     # to the nearest, ties to even
    else:
        pattern = pattern + (random_bits << (low - 16))
    code = pattern >> low
    if bits == R_BITS:
        code = torch.where(x > 0, code.clamp(min=1), code)                     # a root above zero stays above it
    else:
        code = code | ((x.view(torch.int32) >> 24) & 0x80)
    return code.to(torch.uint8), e


def decode(code, e, bits):
    code, e = code.int(), e.int()
    size = code & 0x7F if bits == M_BITS else code
    value = (size << (23 - bits)).view(torch.float32) * 2.0 ** 112 * power(e + 8)
    return torch.where(code >= 128, -value, value) if bits == M_BITS else value


def mix(x):
    """A mixing of 32 bits: exclusive-or with its upper bits, and products with odd constants."""
    x = ((x ^ (x >> 16)) * 0x57735285) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x4746E6A3) & 0xFFFFFFFF
    return x ^ (x >> 16)


def random_words(arena, t):
    """32 random bits for each element, from the seed, the step, the tensor's place, the block's and the element's."""
    key = mix(mix(SEED & 0xFFFFFFFF) ^ (SEED >> 32)) ^ t.long()
    key = mix(mix(mix(key) ^ arena.tensor) ^ arena.number)
    return mix(key[:, None] ^ torch.arange(BLOCK, device=DEVICE))


def plain_adamw(case, d, coefficient, t):
    a, eight, beta2 = d["arena"], d["bits"] == 8, case["beta2"]
    g = blocks(d["grad"]).float()
    if coefficient is not None:
        g = g * coefficient
    if eight:
        m = decode(blocks(d["m8"]), blocks(d["scale"], 2)[:, :1], M_BITS)
        r = decode(blocks(d["r8"]), blocks(d["scale"], 2)[:, 1:], R_BITS)
        v = r * r
    else:
        m, v = blocks(d["m"]), blocks(d["v"])
    m = m * BETA1 + g * (1 - BETA1)
    v = v * beta2 + g * g * (1 - beta2)
    r = v.sqrt()
    step = t.double()
    m_by = 1 / (1 - BETA1 ** step)
    r_by = (1 / (1 - beta2 ** step)).sqrt()
    lr = LR * a.lr
    p = blocks(d["p"])
    new = p * (1 - lr * DECAY * a.wd) - lr * ((m * m_by) / (r * r_by + EPS))
    p.copy_(new)
    if case["ema"]:
        e = blocks(d["ema"])
        e.copy_(e * EMA + new * (1 - EMA))
    if case["copy"]:
        blocks(d["copy"]).copy_(new)
    if eight:
        words = random_words(a, t) if case["stochastic"] else None
        m8, me = encode(m, M_BITS, (words & 0xFFFF).int() if words is not None else None)
        r8, re = encode(r, R_BITS, (words >> 16).int() if words is not None else None)
        keep(d, m8, me, r8, re)
    else:
        blocks(d["m"]).copy_(m)
        blocks(d["v"]).copy_(v)


def keep(d, m8, me, r8, re):
    """Writes codes and scales, and the values that they stand for."""
    blocks(d["m8"]).copy_(m8)
    blocks(d["r8"]).copy_(r8)
    blocks(d["scale"], 2).copy_(torch.cat([me, re], 1))
    blocks(d["m_value"]).copy_(decode(m8, me, M_BITS))
    blocks(d["r_value"]).copy_(decode(r8, re, R_BITS))


# ---------------------------------------------------------------------------------------------
# The same from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    out = {}
    if case["op"] == "norm" or case.get("clip"):
        norm = math.sqrt(math.fsum(float(torch.dot(x, x)) for x in (d["grad"].double() for d in s["arenas"])))
        factor = min(1.0, MAX_NORM / (norm + 1e-6))
        out["norm"] = torch.tensor([norm, factor], dtype=torch.float64)
    if case["op"] == "norm":
        return out
    out["taken"] = None
    for k, d in enumerate(s["arenas"]):
        a = d["arena"]
        if case["op"] == "convert":
            m, r = d["m"].double().view(-1, BLOCK), d["v"].double().view(-1, BLOCK).sqrt()
            out["m_value %d" % k], out["r_value %d" % k] = on_grid(m, 4, None).view(-1), on_grid(r, 5, None, least=True).view(-1)
            continue
        t, beta2 = case["taken"] + 1, case["beta2"]
        g = d["grad"].double().view(-1, BLOCK) * (float(np.float32(factor)) if case["clip"] else 1.0)
        if d["bits"] == 8:
            scale = d["scale"].double().view(-1, 2) - 127
            m = stands_for(d["m8"].view(-1, BLOCK), scale[:, :1], 4)
            v = stands_for(d["r8"].view(-1, BLOCK), scale[:, 1:], 5) ** 2
        else:
            m, v = d["m"].double().view(-1, BLOCK), d["v"].double().view(-1, BLOCK)
        m = BETA1 * m + (1 - BETA1) * g
        v = beta2 * v + (1 - beta2) * g ** 2
        lr, wd = LR * a.lr.double(), DECAY * a.wd.double()
        p = d["p"].double().view(-1, BLOCK)
        p = (1 - lr * wd) * p - lr * (m / (1 - BETA1 ** t)) / ((v / (1 - beta2 ** t)) ** 0.5 + EPS)
        out["p %d" % k] = p.view(-1)
        if case["ema"]:
            out["ema %d" % k] = EMA * d["ema"].double() + (1 - EMA) * p.view(-1)
        if case["copy"]:
            out["copy %d" % k] = p.view(-1)
        if d["bits"] == 32:
            out["m %d" % k], out["v %d" % k] = m.view(-1), v.view(-1)
            continue
        words = exact_words(a, t) if case["stochastic"] else None
        out["m_value %d" % k] = on_grid(m, 4, None if words is None else words % 65536).view(-1)
        out["r_value %d" % k] = on_grid(v.sqrt(), 5, None if words is None else torch.floor(words / 65536), least=True).view(-1)
    return out


def stands_for(code, top, bits):
    """The value of a code: (-1)^sign (1 + mantissa / 2^bits) 2^(top - 7 + exponent), without the 1 where the exponent is 0."""
    code = code.double()
    sign = 1.0
    if bits == 4:
        sign = torch.where(code >= 128, -1.0, 1.0).double()
        code = code % 128
    exponent = torch.floor(code / 2 ** bits)
    fraction = code / 2 ** bits - exponent
    return sign * (fraction + (exponent > 0)) * torch.exp2(top - 7 + exponent.clamp(min=1))


def on_grid(x, bits, sixteen, least=False):
    """x on its block's grid: `bits` bits after the first down to 2^(top - 6), even spacing below."""
    mantissa, exponent = torch.frexp(x.abs().amax(1, keepdim=True))          # mantissa from 1/2 to 1
    top = (exponent - 1 + (mantissa > 1 - 2.0 ** -(bits + 1)).int()).double()
    top = torch.where(mantissa == 0, LOW - 127.0, top).clamp(min=LOW - 127.0)
    own_exponent = torch.maximum(torch.frexp(x.abs())[1].double() - 1, top - 6)
    own_exponent = torch.where(x == 0, top - 6, own_exponent)
    space = torch.exp2(own_exponent - bits)
    number = x.abs() / space
    number = torch.round(number) if sixteen is None else torch.floor(number + sixteen / 65536.0)
    size = number * space
    if least:
        size = torch.where(x > 0, torch.maximum(size, torch.exp2(top - 6 - bits)), size)
    return torch.copysign(size, x)


def exact_words(a, t):
    """random_words() once more, in 32-bit unsigned arithmetic on the host."""
    def stir(x):
        x = np.asarray(x, dtype=np.uint32)
        x = (x ^ (x >> np.uint32(16))) * np.uint32(0x57735285)
        x = (x ^ (x >> np.uint32(15))) * np.uint32(0x4746E6A3)
        return x ^ (x >> np.uint32(16))

    with np.errstate(over="ignore"):
        key = stir(stir(np.uint32(SEED & 0xFFFFFFFF)) ^ np.uint32(SEED >> 32))
        key = stir(key ^ np.uint32(t))
        key = stir(stir(key ^ a.tensor.cpu().numpy().astype(np.uint32)) ^ a.number.cpu().numpy().astype(np.uint32))
        words = stir(key[:, None] ^ np.arange(BLOCK, dtype=np.uint32))
    return torch.from_numpy(words.astype(np.int64)).to(DEVICE).double()
