"""A tensor set on the device and its numpy twin: tensors laid into one buffer a kind with guarded gaps between them, so
that every start is possible and a write outside a tensor shows."""

import numpy as np
import torch

import sharded_zero_partition_amd as zp
from oracle import tensor_set as T

GRAD = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
OUT = {"fp16": torch.float16, "bf16": torch.bfloat16, "none": None}
GUARD = 0x5A

# one to a few elements, the ends of a block (32), of a 256-element group and of a tile (1024), several tiles
SIZES = [1, 0, 2, 3, 4, 5, 31, 32, 33, 63, 255, 256, 257, 1023, 1024, 1025, 2047, 2048, 4099, 1, 7, 10240, 50001]


def guarded(arrays, dtype, gaps):
    """Device views of one buffer, GUARD bytes between them; (buffer, views, starts in elements)."""
    size = torch.empty(0, dtype=dtype).element_size()
    starts, at = [], 0
    for a, gap in zip(arrays, gaps):
        at += int(gap)
        starts.append(at)
        at += len(a)
    buf = torch.full(((at + 16) * size,), GUARD, dtype=torch.uint8, device="cuda")
    flat = buf.view(dtype)
    views = [flat[s:s + len(a)] for s, a in zip(starts, arrays)]
    return buf, views, starts


def bits(t):
    t = t.detach().contiguous()
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).cpu().numpy()


def to_bits(x, dtype):
    """Numpy fp32 values (or codes) to the dtype's bits, rounded to nearest even by torch on the CPU."""
    t = torch.from_numpy(np.ascontiguousarray(x))
    return bits(t.to(dtype) if t.dtype != dtype else t)


class Twin:
    """A set with its own inputs from a seed.  state: "fp32" or "mx".  The tensors of each kind lie up to `gap` elements
    apart, drawn for each kind, or in all kinds by the same `gaps` (buffers start on 512 bytes)."""

    def __init__(self, sizes, grad="fp16", out="fp16", state="fp32", seed=0, groups=None, std=1e-3, scale=1024.0, gap=5, gaps=None):
        rng = np.random.default_rng(seed)
        self.sizes, self.state, self.seed, self.grad_dtype, self.out_dtype = list(sizes), state, seed, GRAD[grad], OUT[out]
        self.groups = [i % 2 for i in range(len(sizes))] if groups is None else groups
        self.rng, self.std, self.scale = rng, std, scale
        self.kinds = {"p": torch.float32, "g": self.grad_dtype}
        host = {"p": [(rng.standard_normal(n) * 0.02).astype(np.float32) for n in sizes]}
        m = [(rng.standard_normal(n) * 3e-4 * 10.0 ** rng.uniform(-2, 1, n)).astype(np.float32) for n in sizes]
        v = [np.square(rng.standard_normal(n) * 1e-3).astype(np.float32) for n in sizes]
        for a, b in zip(m[::3], v[::3]):        # tensors, and the first half of others, that have seen no gradient
            a[:] = 0
            b[:] = 0
        for a, b in zip(m[1::3], v[1::3]):
            a[:len(a) // 2] = 0
            b[:len(b) // 2] = 0
        if state == "fp32":
            self.kinds.update(m=torch.float32, v=torch.float32)
            host.update(m=m, v=v)
        else:
            self.kinds.update(m=torch.uint8, v=torch.uint8, ms=torch.uint8, vs=torch.uint8)
            em, ev = [T.encode(a, False) for a in m], [T.encode(b, True) for b in v]
            host.update(m=[c for c, _ in em], v=[c for c, _ in ev], ms=[s for _, s in em], vs=[s for _, s in ev])
        if self.out_dtype is not None:
            self.kinds["out"] = self.out_dtype
            host["out"] = [np.zeros(n, np.float32) for n in sizes]
        host["g"] = [np.zeros(n, np.float32) for n in sizes]
        self.host, self.buf, self.view, self.start, self.bound = host, {}, {}, {}, {}
        for k, dtype in self.kinds.items():
            apart = rng.integers(0, gap + 1, len(sizes)) if gaps is None else gaps
            if gaps is not None and k in ("ms", "vs"):
                apart = [0] * len(sizes)
            self.buf[k], self.view[k], self.start[k] = guarded(host[k], dtype, apart)
            for t, a in zip(self.view[k], host[k]):
                t.copy_(torch.from_numpy(a))
        self.new_grads()
        opt = dict(m_scale=self.view["ms"], v_scale=self.view["vs"]) if state == "mx" else {}
        self.set = zp.TensorSet(p=self.view["p"], grads=self.view["g"], m=self.view["m"], v=self.view["v"],
                                out=self.view.get("out"), groups=self.groups, seed=seed, **opt)

    def new_grads(self, values=None):
        """New gradients on both sides (host: the values that the dtype holds)."""
        for i, t in enumerate(self.view["g"]):
            x = (self.rng.standard_normal(t.numel()) * self.std * self.scale).astype(np.float32) if values is None else values[i]
            if values is None and i % 4 == 3:
                x[: len(x) // 3] = 0
            h = torch.from_numpy(x).to(self.grad_dtype)
            t.copy_(h)
            self.host["g"][i] = h.to(torch.float32).numpy()

    def sumsq(self):
        return float(sum(np.sum(np.square(g.astype(np.float64))) for g in self.host["g"]))

    def expect(self, c):
        """The host side's step with the oracle's control `c` (begun)."""
        if c.skip:
            return
        for i, n in enumerate(self.sizes):
            h = self.host
            mx = self.state == "mx"
            m = T.decode(h["m"][i], h["ms"][i]) if mx else h["m"][i]
            v = T.decode(h["v"][i], h["vs"][i]) if mx else h["v"][i]
            if mx:      # p by the hardware's root and reciprocal: compared within its bound, then taken over
                w, off = T.adamw_wide(c.groups[self.groups[i]], float(np.float32(c.lr_mult)), c.t, h["g"][i], c.grad_mult, h["p"][i], m, v, fast=True)
                self.bound[i] = w[0], off[0]
            p, m, v = T.adamw(c.consts[self.groups[i]], h["g"][i], c.grad_mult, h["p"][i], m, v)
            h["p"][i] = p
            if mx:
                h["m"][i], h["ms"][i] = T.encode(m, False)
                h["v"][i], h["vs"][i] = T.encode(v, True, T.chances(n, self.seed & 0xFFFFFFFF, i, c.t))
            else:
                h["m"][i], h["v"][i] = m, v
            if "out" in h:
                h["out"][i] = p

    def compare(self, what=""):
        """Every byte of every buffer: tensors as the host has them, guards untouched."""
        for i, (w, off) in self.bound.items():
            p = self.view["p"][i].cpu().numpy()
            d = np.abs(p.astype(np.float64) - w)
            assert (d <= off).all(), f"{what} p of tensor {i}: {np.max(d / off)} of its bound"
            self.host["p"][i] = p
            if "out" in self.host:
                self.host["out"][i] = p
        self.bound = {}
        for k, dtype in self.kinds.items():
            size = torch.empty(0, dtype=dtype).element_size()
            want = np.full(self.buf[k].numel(), GUARD, np.uint8)
            for a, s in zip(self.host[k], self.start[k]):
                if len(a):
                    want[s * size:(s + len(a)) * size] = to_bits(a, dtype).view(np.uint8)
            got = self.buf[k].cpu().numpy()
            if not np.array_equal(got, want):
                bad = int(np.flatnonzero(got != want)[0]) // size
                i = max(j for j, s in enumerate(self.start[k]) if s <= bad)
                raise AssertionError(f"{what} {k}: differs first at element {bad - self.start[k][i]} of tensor {i} (of {self.sizes[i]})")


def read(control):
    """The control block as the binding's struct."""
    return zp.binding.StepControlC.from_buffer_copy(bytes(control.buffer.cpu().numpy()))


def same_control(control, c, rel=0.0):
    """The device's block against the oracle's.  The norm's and factor's last bits hang on the sum's order: `rel`."""
    d = read(control)
    assert (d.t, d.skipped, d.scale, d.good_steps, d.skip) == (c.t, c.skipped, c.scale, c.good_steps, c.skip)
    for a, b in ((d.norm, c.norm), (d.grad_mult, c.grad_mult)):
        assert a == b or abs(a - b) <= rel * abs(b) or (np.isnan(a) and np.isnan(b)), (a, b)
    return d
