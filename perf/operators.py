"""The operators of a tensor set, and what is measured of them: the global norm of many gradient tensors, the AdamW
step over many tensors with states in 32 bits, the same step with states in 8 bits, and the conversion of states
between the two.

A case names a list of tensors, laid back to back in flat buffers without padding as a rank's partition holds them, so
that most tensors start at an odd place:

  "decoder"  the parameter tensors of a GPT-2-style decoder (layers, hidden, vocab), or the pieces of them that the
             last of `ranks` equal shards of the flattened model holds
  "ragged"   `tensors` tensors with sizes log-uniform in [1, most], drawn from `layout`

With scale S the gradients' loss scale, the step is (every gradient finite)

  norm = sqrt(sum g^2) / S           c = max_norm / norm where norm > max_norm, else 1 (max_norm 0: 1)
  g = (c / S) grad
  m = beta1 m + (1 - beta1) g        v = beta2 v + (1 - beta2) g^2
  p = p - (lr wd p + lr / (1 - beta1^t) m / (sqrt(v) / sqrt(1 - beta2^t) + eps))

and out is p rounded to 16 bits.  States in 8 bits: blocks of 32 consecutive elements of a tensor (the last one may be
shorter) hold e4m3 numbers and one power of two, the least that brings the block's largest magnitude to 448 or below (at
least 2^-126).  m is rounded to nearest (ties to even).  v is rounded up or down at random, with a probability that
keeps its mean, from 16 bits of a hash of the set's seed, the tensor, the step and the element; a v above zero does not
become zero.  The update itself uses the new m and v before they are rounded.  A conversion from 32 bits rounds both to
nearest.
"""

import math
import random

import torch

own = False

SCALE = 1024.0
T0 = 1000                                   # steps taken before the pass
LR, BETA1, BETA2, EPS, DECAY = 1e-4, 0.9, 0.999, 1e-8, 0.1
BLOCK = 32
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32, "none": None}


def listed():
    return [
        # a handful of bias and norm vectors: what the call itself costs
        {"name": "norm small fp16", "op": "norm", "kind": "ragged", "tensors": 12, "most": 1600, "layout": 1, "grad": "fp16"},
        # fp32 gradients of a model with thousands of tensors of every size
        {"name": "norm ragged fp32", "op": "norm", "kind": "ragged", "tensors": 1500, "most": 1 << 20, "layout": 2, "grad": "fp32"},
        # one rank's share of a 13B model: pieces of its last layer
        {"name": "norm 13B shard bf16", "op": "norm", "kind": "decoder", "layers": 40, "hidden": 5120, "vocab": 50257, "ranks": 64, "grad": "bf16"},
        # the smallest step: norm, clip and update of a few vectors
        {"name": "adamw32 small fp16 clip", "op": "adamw32", "kind": "ragged", "tensors": 12, "most": 1600, "layout": 1, "grad": "fp16", "out": "fp16", "clip": True},
        # one rank's share of GPT-2 1.5B
        {"name": "adamw32 1.5B shard fp16", "op": "adamw32", "kind": "decoder", "layers": 48, "hidden": 1600, "vocab": 50257, "ranks": 64, "grad": "fp16", "out": "fp16", "clip": False},
        # thousands of tensors of every size, gradients accumulated in fp32, clipped
        {"name": "adamw32 ragged fp32 clip", "op": "adamw32", "kind": "ragged", "tensors": 1500, "most": 1 << 20, "layout": 2, "grad": "fp32", "out": "none", "clip": True},
        # one rank's share of a 13B model, the usual clipped step
        {"name": "adamw32 13B shard bf16 clip", "op": "adamw32", "kind": "decoder", "layers": 40, "hidden": 5120, "vocab": 50257, "ranks": 64, "grad": "bf16", "out": "bf16", "clip": True},
        # states in 8 bits: the smallest step, a whole small decoder on one rank, and the 13B share
        {"name": "adamw8 small fp16 clip", "op": "adamw8", "kind": "ragged", "tensors": 12, "most": 1600, "layout": 3, "grad": "fp16", "out": "fp16", "clip": True},
        {"name": "adamw8 decoder fp16 clip", "op": "adamw8", "kind": "decoder", "layers": 2, "hidden": 1600, "vocab": 50257, "ranks": 1, "grad": "fp16", "out": "fp16", "clip": True},
        {"name": "adamw8 13B shard bf16", "op": "adamw8", "kind": "decoder", "layers": 40, "hidden": 5120, "vocab": 50257, "ranks": 64, "grad": "bf16", "out": "bf16", "clip": False},
        # a run in 32 bits that goes on in 8, and a state in 8 bits read back
        {"name": "states to 8 bits, ragged", "op": "to8", "kind": "ragged", "tensors": 1500, "most": 1 << 18, "layout": 4},
        {"name": "states to 32 bits, 1.5B shard", "op": "to32", "kind": "decoder", "layers": 48, "hidden": 1600, "vocab": 50257, "ranks": 64},
    ]


def draw(rng):
    op = rng.choice(["norm", "adamw32", "adamw32", "adamw8", "adamw8", "to8", "to32"])
    if rng.random() < 0.5:
        case = {"op": op, "kind": "ragged", "tensors": int(10 ** rng.uniform(0, 3.2)), "most": int(2 ** rng.uniform(3, 20)), "layout": rng.randrange(1 << 20)}
    else:
        hidden = 8 * int(2 ** rng.uniform(3, 8))
        layers = rng.randint(1, 24)
        case = {"op": op, "kind": "decoder", "layers": layers, "hidden": hidden, "vocab": rng.randint(1000, 60000), "ranks": rng.choice([1, 2, 3, 5, 8, 17, 64])}
        while _total(case) > 150_000_000:
            case["ranks"] *= 2
    if op in ("norm", "adamw32", "adamw8"):
        case["grad"] = rng.choice(["fp16", "bf16", "fp32"])
    if op in ("adamw32", "adamw8"):
        case["out"] = rng.choice(["fp16", "bf16", "none"])
        case["clip"] = rng.random() < 0.6
    return case


def _numels(case):
    """Sizes of the case's tensors, none of them zero."""
    if case["kind"] == "ragged":
        r = random.Random(case["layout"])
        top = math.log(case["most"] + 1.0)
        return [min(case["most"], max(1, int(math.exp(r.uniform(0.0, top))))) for _ in range(case["tensors"])]
    h = case["hidden"]
    sizes = [case["vocab"] * h, 1024 * h] + [h, h, 3 * h * h, 3 * h, h * h, h, h, h, 4 * h * h, 4 * h, 4 * h * h, h] * case["layers"] + [h, h]
    if case["ranks"] == 1:
        return sizes
    psi = sum(sizes)
    shard = -(-psi // case["ranks"])
    begin, at, pieces = psi - (psi - shard * (case["ranks"] - 1)), 0, []
    for n in sizes:
        if at + n > begin:
            pieces.append(at + n - max(at, begin))
        at += n
    return pieces


def _total(case):
    return sum(_numels(case))


def _groups(case, numels):
    """Vectors take no weight decay (group 1), matrices do (group 0)."""
    most = 4 * case["hidden"] if case["kind"] == "decoder" else 2047
    return [1 if n <= most else 0 for n in numels]


def work(case):
    numels = _numels(case)
    n, blocks = sum(numels), sum(-(-k // BLOCK) for k in numels)
    size = {"fp16": 2, "bf16": 2, "fp32": 4, "none": 0}
    g, o = size[case.get("grad", "none")], size[case.get("out", "none")]
    if case["op"] == "norm":
        return {"bytes": n * g + 8, "flops": 2 * n}
    if case["op"] == "adamw32":
        return {"bytes": n * (g + 24 + o), "flops": 16 * n}
    if case["op"] == "adamw8":
        return {"bytes": n * (g + 8 + 4 + o) + 4 * blocks, "flops": 20 * n}
    return {"bytes": n * (8 + 2) + 2 * blocks, "flops": 4 * n}


# What a program has in hand.

def _fill(n, std, gen):
    return torch.randn(n, generator=gen, device="cuda").mul_(std)


def _split(flat, sizes):
    return list(torch.split(flat, sizes))


def prepare(case, seed):
    numels = _numels(case)
    n = sum(numels)
    op = case["op"]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"
    s = {"case": case, "numels": numels, "n": n, "seed": seed & 0xFFFFFFFF, "t": torch.full((), T0, dtype=torch.int64, device=dev)}
    s["counts"] = torch.tensor(numels, dtype=torch.int64, device=dev)
    s["blocks"] = [-(-k // BLOCK) for k in numels]
    s["first"] = torch.tensor([0] + s["blocks"][:-1], dtype=torch.int64, device=dev).cumsum(0)     # each tensor's first block
    s["groups"] = _groups(case, numels)
    s["group"] = torch.tensor(s["groups"], dtype=torch.int64, device=dev)
    if "grad" in case:
        g = _fill(n, 1e-3 * SCALE, gen).to(DTYPES[case["grad"]])
        g[: n // 16] = 0                     # rows of the embedding that no token of the batch named
        s["grad"] = g
    if op != "norm":
        s["p"] = _fill(n, 0.02, gen)
        m = _fill(n, 3e-4, gen)
        v = _fill(n, 1e-3, gen).square_()
        m[: n // 32] = 0                     # rows that no batch has named so far
        v[: n // 32] = 0
        if op in ("adamw32", "to8"):
            s["m"], s["v"] = m, v
        else:
            at = _places(s, _tensors(s))
            s["m"], s["m_scale"] = _encode(m, at, sum(s["blocks"]), None)
            s["v"], s["v_scale"] = _encode(v, at, sum(s["blocks"]), None)
        if op in ("to8", "to32"):            # where the states go
            b = sum(s["blocks"])
            s["to"] = [torch.zeros(n, dtype=torch.uint8 if op == "to8" else torch.float32, device=dev) for _ in range(2)]
            if op == "to8":
                s["to"] += [torch.zeros(b, dtype=torch.uint8, device=dev) for _ in range(2)]
        s["out"] = torch.zeros(n, dtype=DTYPES[case["out"]], device=dev) if DTYPES[case.get("out", "none")] is not None else None
    if own:
        _hand_over(s)
    return s


def _hand_over(s):
    """The handles that a program makes once: the tensor set and the step's control block."""
    import sharded_zero_partition_amd as zp
    case, sizes, blocks = s["case"], s["numels"], s["blocks"]
    op = case["op"]
    s["hparams"] = [zp.AdamHParams(LR, BETA1, BETA2, EPS, DECAY), zp.AdamHParams(LR, BETA1, BETA2, EPS, 0.0)]
    s["control"] = zp.StepControl(scale=SCALE, t=T0)
    if op == "norm":
        s["set"] = zp.TensorSet(grads=_split(s["grad"], sizes))
        return
    grads = _split(s["grad"], sizes) if "grad" in s else None
    out = _split(s["out"], sizes) if s["out"] is not None else None
    p = _split(s["p"], sizes)

    def states(m, v, ms=None, vs=None):
        return dict(m=_split(m, sizes), v=_split(v, sizes), m_scale=None if ms is None else _split(ms, blocks),
                    v_scale=None if vs is None else _split(vs, blocks))

    s["set"] = zp.TensorSet(p=p, grads=grads, out=out, groups=s["groups"], seed=s["seed"], **states(s["m"], s["v"], s.get("m_scale"), s.get("v_scale")))
    if op in ("to8", "to32"):
        s["target"] = zp.TensorSet(p=p, seed=s["seed"], **states(*s["to"]))


# The plain forms.

def _tensors(s):
    """Each element's tensor."""
    return torch.bucketize(torch.arange(s["n"], device="cuda"), s["counts"].cumsum(0), right=True, out_int32=True)


def _places(s, of):
    """Where each element stands when every tensor starts a block of its own."""
    shift = s["first"] * BLOCK - (s["counts"].cumsum(0) - s["counts"])
    return torch.arange(s["n"], device="cuda") + shift[of]


def _mix(x):
    """MurmurHash3's 32-bit finaliser on int32 (products wrap; shifts are made logical by masks)."""
    x = x ^ ((x >> 16) & 0xFFFF)
    x = x * -2048144789                      # 0x85EBCA6B
    x = x ^ ((x >> 13) & 0x7FFFF)
    x = x * -1028477387                      # 0xC2B2AE35
    return x ^ ((x >> 16) & 0xFFFF)


def _chances(s, of, at, t):
    """20 bits for each element: the upper 16 from the hash of its pair, then 8."""
    tensor = torch.arange(len(s["numels"]), dtype=torch.int32, device="cuda")
    low = torch.full((), s["seed"] - (1 << 32) if s["seed"] >> 31 else s["seed"], dtype=torch.int32, device="cuda")
    key = _mix(_mix(low) + tensor)
    key = _mix(key + t.to(torch.int32) * -1640531527)             # 0x9E3779B9
    element = at - (s["first"] * BLOCK)[of]
    pair = _mix((element >> 1).to(torch.int32) + key[of])
    half = torch.where((element & 1) == 0, pair & 0xFFFF, (pair >> 16) & 0xFFFF)
    return (half << 4) | 8


def _encode(x, at, blocks, positive, chances=None):
    """(codes, scales) of x in blocks: to nearest, or at random where chances are given. Of x that is never negative, no value above zero becomes zero."""
    padded = torch.zeros(blocks * BLOCK, device="cuda")
    padded[at] = x.abs()
    top = padded.view(blocks, BLOCK).amax(1)
    scale = (((top.view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp(min=1)
    y = x * ((254 - scale) << 23).view(torch.float32)[at >> 5]
    if chances is not None:
        lift = torch.where(y < 2.0 ** -6, 2.0 ** -6, 0.0)           # below it the numbers' steps are all 2^-9, as in [2^-6, 2^-5)
        y = (((y + lift).view(torch.int32) + chances) & ~0xFFFFF).view(torch.float32) - lift
    code = y.to(torch.float8_e4m3fn).view(torch.uint8)
    if positive:
        code = torch.maximum(code, (x > 0).to(torch.uint8))
    return code, scale.to(torch.uint8)


def _decode(code, scale, at):
    return code.view(torch.float8_e4m3fn).to(torch.float32) * (scale.to(torch.int32) << 23).view(torch.float32)[at >> 5]


def _begin(s):
    """(whether the step is taken, the new t, the norm, what gradients are multiplied by), all on the GPU."""
    t, norm = s["t"], torch.zeros((), dtype=torch.float64, device="cuda")
    ok, factor = torch.ones((), dtype=torch.bool, device="cuda"), torch.full((), 1.0 / SCALE, dtype=torch.float64, device="cuda")
    if s["case"]["clip"]:
        norm = s["grad"].to(torch.float64).square().sum().sqrt() / SCALE
        ok = norm < 2.0 ** 62
        factor = torch.where(norm > 1.0, 1.0 / norm, 1.0) / SCALE
    return ok, t + ok, norm.to(torch.float32), factor.to(torch.float32)


def _adamw(s, of, m, v, t, factor):
    """(p, m, v) after the step."""
    t = t.to(torch.float64)
    b1, b2 = torch.tensor([BETA1, BETA2], dtype=torch.float32).tolist()
    step = (LR / (1.0 - torch.pow(b1, t))).to(torch.float32)
    root = torch.rsqrt(1.0 - torch.pow(b2, t)).to(torch.float32)
    g = s["grad"].to(torch.float32) * factor
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + g.square() * (1.0 - b2)
    decay = torch.where(s["group"] == 0, LR * DECAY, 0.0).to(torch.float32)[of]
    return s["p"] - (s["p"] * decay + m / (v.sqrt() * root + EPS) * step), m, v


def _commit(s, ok, new):
    """Writes what the step gives, where it is taken."""
    if not s["case"]["clip"]:                # nothing was looked at: always taken
        ok = None
    torch._foreach_copy_([s[k] for k in new], [x if ok is None else torch.where(ok, x, s[k]) for k, x in new.items()])
    if s["out"] is not None:
        s["out"].copy_(s["p"])


def _adamw32_plain(s):
    ok, t, norm, factor = _begin(s)
    p, m, v = _adamw(s, _tensors(s), s["m"], s["v"], t, factor)
    _commit(s, ok, {"p": p, "m": m, "v": v, "t": t})
    return {"p": s["p"], "m": s["m"], "v": s["v"], "out": s["out"], "t": s["t"], "norm": norm}


def _adamw8_plain(s):
    ok, t, norm, factor = _begin(s)
    of, blocks = _tensors(s), sum(s["blocks"])
    at = _places(s, of)
    p, m, v = _adamw(s, of, _decode(s["m"], s["m_scale"], at), _decode(s["v"], s["v_scale"], at), t, factor)
    m, m_scale = _encode(m, at, blocks, False)
    v, v_scale = _encode(v, at, blocks, True, _chances(s, of, at, t))
    _commit(s, ok, {"p": p, "m": m, "v": v, "m_scale": m_scale, "v_scale": v_scale, "t": t})
    return {"p": s["p"], "out": s["out"], "t": s["t"], "norm": norm, **_numbers(s["m"], s["v"], s["m_scale"], s["v_scale"])}


def _numbers(m, v, m_scale, v_scale):
    """States in 8 bits as the numbers that they hold: the blocks' powers of two and what these multiply."""
    return {"m": m.view(torch.float8_e4m3fn), "v": v.view(torch.float8_e4m3fn), "m_scale": m_scale.view(torch.float8_e8m0fnu), "v_scale": v_scale.view(torch.float8_e8m0fnu)}


def _plain(s):
    op = s["case"]["op"]
    if op == "norm":
        return {"sumsq": s["grad"].to(torch.float64).square().sum()}
    if op == "adamw32":
        return _adamw32_plain(s)
    if op == "adamw8":
        return _adamw8_plain(s)
    at, blocks, to = _places(s, _tensors(s)), sum(s["blocks"]), s["to"]
    if op == "to8":
        m, m_scale = _encode(s["m"], at, blocks, False)
        v, v_scale = _encode(s["v"], at, blocks, True)
        torch._foreach_copy_(to, [m, v, m_scale, v_scale])
        return _numbers(*to)
    torch._foreach_copy_(to, [_decode(s["m"], s["m_scale"], at), _decode(s["v"], s["v_scale"], at)])
    return {"m": to[0], "v": to[1]}


# The framework's calls.

def _calls(s):
    op = s["case"]["op"]
    if op in ("to8", "to32"):
        s["target"].states_from(s["set"])
        return _numbers(*s["to"]) if op == "to8" else {"m": s["to"][0], "v": s["to"][1]}
    c = s["control"]
    if op == "norm":
        s["set"].grad_sumsq(c.sumsq)
        return {"sumsq": c.sumsq}
    if s["case"]["clip"]:
        s["set"].grad_sumsq(c.sumsq)
        c.begin(s["hparams"], max_norm=1.0)
    else:
        c.begin(s["hparams"], check=False)
    s["set"].adamw_step(c)
    got = {"p": s["p"], "out": s["out"], "t": c.t, "norm": c.norm}
    if op == "adamw32":
        return {**got, "m": s["m"], "v": s["v"]}
    return {**got, **_numbers(s["m"], s["v"], s["m_scale"], s["v_scale"])}


def run(state):
    return _calls(state) if own else _plain(state)


# What the outputs are, from the definition, in 64 bits.

def _exact_blocks(s):
    """For each element, its block, and for each block a number of its own, from the sizes alone."""
    sizes = torch.tensor(s["numels"], device="cuda")
    of = torch.repeat_interleave(torch.arange(len(s["numels"]), device="cuda"), sizes)
    inside = torch.arange(s["n"], device="cuda") - torch.cat([sizes.new_zeros(1), sizes.cumsum(0)[:-1]])[of]
    count = torch.div(sizes + BLOCK - 1, BLOCK, rounding_mode="floor")
    return of, inside, torch.cat([count.new_zeros(1), count.cumsum(0)[:-1]])[of] + torch.div(inside, BLOCK, rounding_mode="floor")


def _exact_e4m3(y, up=None):
    """y (448 at most in magnitude) to an e4m3 number: to nearest, ties to even, or up where the part that does not fit reaches 1 - up."""
    _, e = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), e.clamp(min=-5) - 4)
    return torch.round(y / step) * step if up is None else torch.floor(y / step + up) * step


def _exact_pack(x, block, positive, up=None):
    """(numbers, powers of two) of the blocks of x."""
    top = torch.zeros(int(block[-1]) + 1, dtype=torch.float64, device="cuda").scatter_reduce_(0, block, x.abs(), "amax")
    fraction, e = torch.frexp(top)
    e = e - 1 - 8 + (fraction > 0.875)                             # top = 2 fraction 2^(e - 1)
    e = torch.where(top > 0, e, -126).clamp(min=-126)
    power = torch.ldexp(torch.ones_like(top), e)
    y = _exact_e4m3(x / power[block], up)
    return torch.where((x > 0) & (y == 0), 2.0 ** -9, y) if positive else y, power


def _exact_up(s, of, inside, t):
    """The share of a step from which v is rounded up, as 1 - share: the hash over whole numbers of 64 bits."""
    full = 0xFFFFFFFF

    def mix(x):
        x = ((x ^ (x >> 16)) * 0x85EBCA6B) & full
        x = ((x ^ (x >> 13)) * 0xC2B2AE35) & full
        return x ^ (x >> 16)

    seed = mix(torch.tensor(s["seed"], device="cuda"))
    key = mix((mix((seed + of) & full) + t * 0x9E3779B9) & full)
    h = mix((torch.div(inside, 2, rounding_mode="floor") + key) & full)
    bits = torch.where(inside % 2 == 0, h % 65536, h >> 16)
    return (bits.to(torch.float64) * 16 + 8) / 2.0 ** 20


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op, wide = case["op"], torch.float64
    if op == "norm":
        return {"sumsq": (s["grad"].to(wide) ** 2).sum()}
    of, inside, block = _exact_blocks(s)
    if op == "to8":
        (m, ms), (v, vs) = _exact_pack(s["m"].to(wide), block, False), _exact_pack(s["v"].to(wide), block, True)
        return {"m": m, "v": v, "m_scale": ms, "v_scale": vs}
    m, v = s["m"], s["v"]
    if "m_scale" in s:
        m, v = ((k.view(torch.float8_e4m3fn).to(wide) * torch.exp2(e.to(wide) - 127)[block]) for k, e in ((m, s["m_scale"]), (v, s["v_scale"])))
    m, v = m.to(wide), v.to(wide)
    if op == "to32":
        return {"m": m, "v": v}
    t, norm, c = T0 + 1, 0.0, 1.0
    g = s["grad"].to(wide)
    if case["clip"]:
        norm = math.sqrt(float((g ** 2).sum())) / SCALE
        c = 1.0 / norm if norm > 1.0 else 1.0
    g *= c / SCALE
    b1, b2 = (float(torch.tensor(b, dtype=torch.float32)) for b in (BETA1, BETA2))
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g ** 2
    p = s["p"].to(wide)
    p = p - (LR * DECAY * p * (s["group"] == 0).to(wide)[of] + LR / (1 - b1 ** t) * m / (torch.sqrt(v) / math.sqrt(1 - b2 ** t) + EPS))
    got = {"p": p, "out": None if s["out"] is None else p, "t": None, "norm": torch.tensor(norm, dtype=wide)}
    if op == "adamw32":
        return {**got, "m": m, "v": v}
    (m, ms), (v, vs) = _exact_pack(m, block, False), _exact_pack(v, block, True, _exact_up(s, of, inside, t))
    return {**got, "m": m, "v": v, "m_scale": ms, "v_scale": vs}
