"""Plain numpy forms of the tensor-set operators: AdamW with fp32 or MXFP8 states, the begin of a step, the state
conversion.  Two kinds: `adamw`, `encode` and `decode` round every operation to fp32 as the definition orders them (a
device result equals them bit for bit), `adamw_wide` computes in 64 bits what they approximate, with a bound on how far
they may be from it."""

from dataclasses import dataclass, field

import numpy as np

BLOCK = 32
U = 2.0 ** -24          # half a unit of fp32's last place, relative


def e4m3_values():
    """The number of every e4m3 code (OCP: bias 7, no infinities, 0x7F and 0xFF NaN)."""
    c = np.arange(256)
    e, f, sign = (c >> 3) & 15, c & 7, np.where(c & 128, -1.0, 1.0)
    v = sign * np.where(e == 0, f / 8.0 * 2.0 ** -6, (1 + f / 8.0) * 2.0 ** (e - 7.0))
    v[[0x7F, 0xFF]] = np.nan
    return v


E4M3 = e4m3_values()
_POSITIVE = E4M3[:127]   # ascending


def e4m3_nearest(y):
    """Codes of y (448 at most in magnitude), to nearest, ties to the even code."""
    y = np.asarray(y, np.float64)
    a = np.abs(y)
    hi = np.clip(np.searchsorted(_POSITIVE, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    down, up = a - _POSITIVE[lo], _POSITIVE[hi] - a
    pick = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    return (pick + np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def mix32(x):
    x = np.asarray(x, np.uint64) & 0xFFFFFFFF
    x ^= x >> np.uint64(16)
    x = (x * 0x85EBCA6B) & 0xFFFFFFFF
    x ^= x >> np.uint64(13)
    x = (x * 0xC2B2AE35) & 0xFFFFFFFF
    return x ^ (x >> np.uint64(16))


# m in 8 bits is rounded to nearest up to this beta1 (as fp32 has it), at random above: 1.125 beta1 has to come below
# 1.0625, or an m without gradient stays where it is.
NEAREST_BETA1 = float(np.float32(0.9444))


def chances(n, seed, tensor, t, start=0, of_m=False):
    """16 random bits for each of elements start .. start + n of a tensor at step t, of v or of m."""
    key = mix32(mix32(mix32(seed) + np.uint64(tensor)) + np.uint64((t * 0x9E3779B9) & 0xFFFFFFFF))
    if of_m:
        key = mix32(key ^ np.uint64(0xFFFFFFFF))
    e = np.arange(start, start + n, dtype=np.uint64)
    h = mix32((e >> np.uint64(1)) + key)
    return np.where(e & np.uint64(1), h >> np.uint64(16), h & np.uint64(0xFFFF)).astype(np.uint32)


def scale_bytes(top):
    """The least s >= 1 with top * 2^(127 - s) <= 448."""
    f, e = np.frexp(np.asarray(top, np.float64))          # top = f 2^e, f in [0.5, 1)
    s = e - 9 + (f > 0.875) + 127                         # 448 = 0.875 2^9
    return np.where(top > 0, np.maximum(s, 1), 1).astype(np.int64)


def _blocks(x):
    n = x.size
    pad = np.zeros(-(-n // BLOCK) * BLOCK, x.dtype)
    pad[:n] = x
    return pad.reshape(-1, BLOCK)


def encode(x, positive, chance=None):
    """(codes, scale bytes) of an fp32 tensor: to nearest, or with 16 random bits an element to a neighbour."""
    x = np.asarray(x, np.float32)
    s = scale_bytes(np.abs(_blocks(x)).max(1) if x.size else np.zeros(0))
    with np.errstate(under="ignore"):
        y = x * np.repeat(np.ldexp(np.float32(1), 127 - s).astype(np.float32), BLOCK)[:x.size]
    if positive:
        y = np.maximum(y, np.where(x > 0, np.float32(2.0 ** -9), np.float32(0))) + np.float32(0)    # -0: +0
    if chance is None:
        return e4m3_nearest(y), s.astype(np.uint8)
    # the next number below in magnitude and the share of the step to the one above, in which 20 bits are added and cut
    # off; below 2^-6 the steps are 2^-9
    up = (chance.astype(np.int64) << 4) | 8
    a = np.abs(y)
    _, e = np.frexp(np.maximum(a, np.float32(2.0 ** -6)))
    step = np.ldexp(1.0, e - 4)
    code = e4m3_nearest(np.copysign(np.floor(a.astype(np.float64) / step + up / 2.0 ** 20) * step, y))
    return code, s.astype(np.uint8)


def encode_m(m, beta1, seed, tensor, t, always_random=False):
    """(codes, scale bytes) of the m that a step with beta1 leaves."""
    if always_random or beta1 > NEAREST_BETA1:
        return encode(m, False, chances(m.size, seed, tensor, t, of_m=True))
    return encode(m, False)


def decode(code, s):
    f = np.ldexp(1.0, np.asarray(s, np.int64) - 127)
    with np.errstate(under="ignore"):
        return (E4M3[code] * np.repeat(f, BLOCK)[:code.size]).astype(np.float32)


@dataclass
class HParams:
    lr: float = 1e-3
    beta1: float = 0.9
    beta2: float = 0.999
    eps: float = 1e-8
    weight_decay: float = 0.0

    def __post_init__(self):     # as the ABI takes them
        for k in ("lr", "beta1", "beta2", "eps", "weight_decay"):
            setattr(self, k, float(np.float32(getattr(self, k))))


@dataclass
class Control:
    """zero_step_control and zero_step_begin."""
    t: int = 0
    skipped: int = 0
    scale: float = 1.0
    lr_mult: float = 1.0
    good_steps: int = 0
    skip: int = 0
    norm: float = 0.0
    grad_mult: float = 0.0
    sumsq: float = 0.0
    consts: list = field(default_factory=list)
    groups: list = field(default_factory=list)

    def begin(self, groups, max_norm=0.0, check=True, scaler=None):
        scale = float(np.float32(self.scale))
        ok = scale >= 2.0 ** -24 and np.isfinite(scale) and np.isfinite(self.lr_mult)
        norm, clip = 0.0, 1.0
        if check:
            norm = float(np.sqrt(np.float64(self.sumsq))) / scale
            clip = max_norm / norm if max_norm > 0 and norm > max_norm else 1.0
            ok = bool(ok and norm * clip < 2.0 ** 62)
        ok = bool(ok and clip / scale >= 2.0 ** -126)
        self.norm = float(np.float32(norm))
        self.grad_mult = float(np.float32(clip / scale)) if ok else 0.0
        self.skip = 0 if ok else 1
        self.groups = list(groups)
        if ok:
            self.t += 1
            self.consts = []
            for h in groups:
                lr = h.lr * float(np.float32(self.lr_mult))
                self.consts.append(dict(
                    beta1=h.beta1, omb1=float(np.float32(1) - np.float32(h.beta1)), beta2=h.beta2,
                    omb2=float(np.float32(1) - np.float32(h.beta2)), decay=float(np.float32(lr * h.weight_decay)),
                    step=float(np.float32(lr / (1.0 - h.beta1 ** self.t))),
                    rbc2=float(np.float32(1.0 / np.sqrt(1.0 - h.beta2 ** self.t))), eps=h.eps))
        else:
            self.skipped += 1
        if scaler is not None:
            if not ok:
                s = float(np.float32(scale * scaler.backoff))
                self.scale = s if np.isfinite(s) and s >= scaler.min_scale else float(np.float32(scaler.min_scale))
                self.good_steps = 0
            else:
                self.good_steps += 1
                if scaler.growth_interval > 0 and self.good_steps >= scaler.growth_interval:
                    with np.errstate(over="ignore"):
                        s = np.float32(scale) * np.float32(scaler.growth)
                    if np.isfinite(s):
                        self.scale = float(s)
                    self.good_steps = 0
        return ok


def adamw(c, grad, mult, p, m, v):
    """(p, m, v), fp32, one rounding an operation.  grad: fp32 values."""
    f = {k: np.float32(x) for k, x in c.items()}
    with np.errstate(under="ignore", over="ignore", invalid="ignore"):
        g = grad.astype(np.float32) * np.float32(mult)
        m = f["beta1"] * m + f["omb1"] * g
        v = f["beta2"] * v + f["omb2"] * (g * g)
        den = np.sqrt(v) * f["rbc2"] + f["eps"]
        p = p - (f["decay"] * p + f["step"] * (m / den))
    return p, m, v


def adamw_wide(h, lr_mult, t, grad, mult, p, m, v, fast=False):
    """((p, m, v) in 64 bits, how far fp32 results may be from each).  `mult` is the exact factor, clip / scale.

    Each rounding to fp32 is off by U relative at most.  g: the factor's and the product's.  beta1 m: the product's and
    the sum's; (1 - beta1) g: g's two, the product's and the sum's; so m is off by 4 U of its terms' magnitudes.  g^2:
    twice g's two and its own; v: those 5, its product's and the sum's: 7 U of its terms, none of them negative.  den:
    half of v's 7 and sqrt's own, the constant's, the product's and the sum's: 7.5 U.  m / den: m's error over den, den's
    7.5 and the quotient's; times the step: 2 more; the term with p: 2; the sum of the two and the difference: 1 each.
    fast (the step with MXFP8 states): root and reciprocal are within 1 ulp, 2 U, each where sqrt and the quotient were
    within 1: a product takes the quotient's place, so 12 become 14; v counts as 2^-126 at least under the root.
    U stands for U (1 + 16 U); subnormal results add 2^-149 a rounding."""
    w = np.float64
    p, m, v, g = p.astype(w), m.astype(w), v.astype(w), grad.astype(w) * mult
    lr, tiny, u = h.lr * lr_mult, 8 * 2.0 ** -149, U * (1 + 16 * U)
    m1, m2 = h.beta1 * m, (1 - h.beta1) * g
    m_new = m1 + m2
    m_off = 4 * u * (np.abs(m1) + np.abs(m2)) + tiny
    v_new = h.beta2 * v + (1 - h.beta2) * g * g
    v_off = 7 * u * v_new + tiny
    den = np.sqrt(np.maximum(v_new, 2.0 ** -126) if fast else v_new) / np.sqrt(1 - h.beta2 ** t) + h.eps
    step = lr / (1 - h.beta1 ** t)
    update = step * m_new / den
    decay = lr * h.weight_decay * p
    p_new = p - (decay + update)
    p_off = np.abs(step) * m_off / den + (14 if fast else 12) * u * np.abs(update) + 4 * u * np.abs(decay) + u * np.abs(p_new) + tiny
    # where v is subnormal its absolute error reaches den through a root
    p_off += np.abs(update) / den * np.sqrt(tiny) * (v_new < 2.0 ** -120)
    return (p_new, m_new, v_new), (p_off, m_off, v_off)
