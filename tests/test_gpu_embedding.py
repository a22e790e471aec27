"""Embedding lookup and its gradient on the GPU: whole numbers exactly, others against 64 bits."""

import numpy as np
import pytest
import torch

import sharded_zero_partition_amd as zp
from matrix_harness import DTYPES, Guarded, half_unit, held
from oracle import activations as A

pytestmark = pytest.mark.gpu


def tokens_like(rng, how, n, vocab):
    if how == "one":
        return np.full(n, vocab // 2)
    if how == "spread":
        return rng.integers(0, vocab, n)
    if how == "text":
        return np.minimum((np.exp(rng.random(n) * np.log(vocab + 1.0)) - 1).astype(np.int64), vocab - 1)
    if how == "none":
        return np.where(rng.random(n) < 0.5, -1, vocab + rng.integers(0, 3, n))
    t = np.sort(rng.integers(0, vocab, n))          # "runs": long runs, tiles that start and end with one, padding between
    t = (t // max(1, vocab // 3)) * max(1, vocab // 3)
    t[n // 3: n // 2] = -5
    return t


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("out", DTYPES)
def test_lookup(dtype, out):
    rng = np.random.default_rng(3)
    for n, vocab, cols, first, scale, off, pad, size in ((1, 1, 1, 0, 1.0, 0, 0, 8), (50, 7, 9, 0, 2.0, 1, 2, 8), (300, 1000, 129, 100, 0.3, 0, 0, 4),
                                                         (64, 40, 512, -20, 1.0, 3, 0, 8), (5, 3, 1031, 0, -1.0, 0, 8, 4)):
        table = held(rng.standard_normal((vocab, cols)), DTYPES[dtype])
        t = rng.integers(first - 3, first + vocab + 3, n)
        src, dst = Guarded(vocab, cols, DTYPES[dtype], off, pad, table), Guarded(n, cols, DTYPES[out], pad, off)
        zp.embedding_lookup(src.t, torch.from_numpy(t).to(torch.int64 if size == 8 else torch.int32).cuda(), dst.t, scale=scale, first=first)
        want = A.lookup(table, t, first, float(np.float32(scale)))
        assert (np.abs(dst.wide() - want) <= half_unit(want, DTYPES[out]) * (1 + 2.0 ** -10) + np.abs(want) * 2.0 ** -24).all()
        if scale in (1.0, 2.0, -1.0) and (dtype == out or out == "fp32"):
            assert np.array_equal(dst.wide(), want)
        assert dst.untouched() and src.untouched()


def grad(n, vocab, cols, how, dtype, out, accumulate, scale=1.0, first=0, off=0, pad=0, seed=0, size=8):
    rng = np.random.default_rng(seed + n + vocab + cols)
    t = tokens_like(rng, how, n, vocab) + first
    dy = held(rng.integers(-4, 5, (n, cols)), dtype)
    old = held(rng.integers(-9, 10, (vocab, cols)), out)
    g, w = Guarded(n, cols, dtype, off, pad, dy), Guarded(vocab, cols, out, pad, off, old)
    zp.embedding_grad(g.t, torch.from_numpy(t).to(torch.int64 if size == 8 else torch.int32).cuda(), w.t, scale=scale, first=first, accumulate=accumulate)
    want = A.embedding_grad(dy, t, vocab, first, scale)[0] + (old if accumulate else 0)
    assert w.untouched() and g.untouched()
    assert np.array_equal(w.wide(), torch.from_numpy(want).to(torch.float32).to(out).to(torch.float64).numpy())


@pytest.mark.parametrize("how", ["one", "spread", "text", "none", "runs"])
@pytest.mark.parametrize("n,vocab,cols", [(1, 1, 1), (2, 5, 3), (63, 10, 8), (64, 1000, 9), (65, 3, 513), (130, 64, 40), (700, 50, 130), (5000, 300, 24)])
def test_gradient_of_whole_numbers(how, n, vocab, cols):
    """Every sum exact, so the result is the definition's, whatever the order."""
    for i, (dtype, out, accumulate, scale, first, off, pad, size) in enumerate((
            ("bf16", "bf16", False, 1.0, 0, 0, 0, 8), ("fp16", "fp32", True, 2.0, 77, 1, 3, 4), ("fp32", "fp32", False, 0.5, -3, 0, 1, 8),
            ("fp16", "fp16", True, -1.0, 0, 8, 0, 8), ("fp32", "bf16", False, 1.0, 1 << 20, 3, 5, 4))):
        grad(n, vocab, cols, how, DTYPES[dtype], DTYPES[out], accumulate, scale, first, off, pad, i, size)


@pytest.mark.parametrize("how", ["one", "spread", "text", "runs"])
@pytest.mark.parametrize("n,vocab", [(8192, 511), (8193, 511), (8300, 2), (20000, 513), (33000, 70000), (300000, 300000), (270000, 100)])
def test_gradient_of_many_tokens(how, n, vocab):
    """Both ways of sorting, one, two and three digits, many blocks."""
    for accumulate in (False, True):
        grad(n, vocab, 5, how, DTYPES["fp16"], DTYPES["fp32"], accumulate)


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_against_64_bits(dtype):
    """A row's summands are added one by one, or in parts: as many roundings, of at most the sum of magnitudes; then the
    scale's, the addition's and the type's."""
    rng = np.random.default_rng(5)
    n, vocab, cols = 4000, 200, 70
    t = tokens_like(rng, "text", n, vocab)
    dy = held(rng.standard_normal((n, cols)), DTYPES[dtype])
    for out in DTYPES.values():
        for accumulate in (False, True):
            old = held(rng.standard_normal((vocab, cols)), out)
            w = torch.from_numpy(old).to(out).cuda()
            zp.embedding_grad(torch.from_numpy(dy).to(DTYPES[dtype]).cuda(), torch.from_numpy(t).cuda(), w, scale=0.3, accumulate=accumulate)
            want, mag, count = A.embedding_grad(dy, t, vocab, 0, float(np.float32(0.3)))
            if accumulate:
                want, mag = want + old, mag + np.abs(old)
            off = np.abs(w.to(torch.float64).cpu().numpy() - want)
            assert (off <= (count[:, None] + 3) * 2.0 ** -24 * mag + half_unit(want, out) * (1 + 2.0 ** -10)).all()


def test_gradient_is_the_lookups():
    """<dy, lookup(table)> = <lookup's gradient, table> for whole numbers."""
    g = torch.Generator(device="cuda").manual_seed(1)
    table = torch.randint(-3, 4, (40, 33), device="cuda", generator=g).float()
    dy = torch.randint(-3, 4, (500, 33), device="cuda", generator=g).float()
    t = torch.randint(-2, 43, (500,), device="cuda", generator=g)
    y, d = torch.empty_like(dy), torch.empty_like(table)
    zp.embedding_lookup(table, t, y, scale=2.0)
    zp.embedding_grad(dy, t, d, scale=2.0)
    assert (dy * y).sum().item() == (d * table).sum().item()


def test_a_table_cut_by_rows():
    """Each rank's part of a vocabulary: the lookups add up to the whole one, the gradients are its rows."""
    g = torch.Generator(device="cuda").manual_seed(2)
    table, dy = torch.randn(100, 20, device="cuda", generator=g), torch.randn(3, 70, 20, device="cuda", generator=g)
    t = torch.randint(0, 100, (3, 70), device="cuda", generator=g)
    whole, total, d = torch.empty_like(dy), torch.zeros_like(dy), torch.empty_like(table)
    zp.embedding_lookup(table, t, whole)
    zp.embedding_grad(dy, t, d)
    for lo, hi in ((0, 34), (34, 68), (68, 100)):
        part, dp = torch.empty_like(dy), torch.empty(hi - lo, 20, device="cuda")
        zp.embedding_lookup(table[lo:hi], t, part, first=lo)
        total += part
        zp.embedding_grad(dy, t, dp, first=lo)
        assert torch.equal(dp, torch.zeros_like(dp).index_add_(0, t.view(-1)[(t.view(-1) >= lo) & (t.view(-1) < hi)] - lo,
                                                               dy.view(-1, 20)[(t.view(-1) >= lo) & (t.view(-1) < hi)])) or \
            (dp - d[lo:hi]).abs().max() <= 16 * 2.0 ** -24 * dy.abs().sum()
    assert torch.equal(total, whole)


def test_special_values_stay_in_their_rows():
    dy = torch.ones(300, 40, device="cuda")
    t = torch.arange(300, device="cuda") % 30
    dy[5, 3], dy[70, 7] = float("inf"), float("nan")
    t[100] = -1
    dy[100] = float("nan")                          # padding: not read into anything
    d = torch.empty(32, 40, device="cuda")
    zp.embedding_grad(dy, t, d)
    assert d[5, 3].item() == float("inf") and bool(d[10, 7].isnan())
    d[5, 3] = d[10, 7] = 10.0
    want = torch.full((32, 40), 10.0, device="cuda")
    want[10] = 9.0                                    # token 100 would have been row 10
    want[10, 7] = 10.0
    want[30:] = 0
    assert torch.equal(d, want)


def test_empty_lists_and_tables():
    d, t = torch.ones(4, 5, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    zp.embedding_grad(torch.empty(0, 5, device="cuda"), t, d, accumulate=True)
    assert bool((d == 1).all())
    zp.embedding_grad(torch.empty(0, 5, device="cuda"), t, d)
    assert bool((d == 0).all())
    zp.embedding_lookup(d, t, torch.empty(0, 5, device="cuda"))
    y = torch.ones(3, 5, device="cuda")
    zp.embedding_lookup(d[:0], torch.tensor([0, 1, -1], device="cuda"), y)
    assert bool((y == 0).all())
    zp.embedding_grad(y, torch.tensor([0, 1, -1], device="cuda"), d[:0])


def test_broadcast_gradient():
    row = torch.randint(-3, 4, (1, 33), device="cuda").float()
    t = torch.randint(0, 9, (200,), device="cuda")
    d = torch.empty(9, 33, device="cuda")
    zp.embedding_grad(row.expand(200, 33), t, d)
    assert torch.equal(d, torch.bincount(t, minlength=9)[:, None] * row)


def test_refusals_of_the_binding():
    table, y, t = torch.zeros(4, 5, device="cuda"), torch.zeros(3, 5, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in (t.cpu(), t.short(), t[:2], torch.zeros(6, dtype=torch.int64, device="cuda")[::2]):
        with pytest.raises(ValueError):
            zp.embedding_lookup(table, bad, y)
        with pytest.raises(ValueError):
            zp.embedding_grad(y, bad, table)
    with pytest.raises(zp.ZeroError, match="overlaps"):
        zp.embedding_lookup(table, t, table[:3])


def test_tokens_and_first_rows_at_the_ends_of_their_range():
    """Tokens whose distance to the first row is beyond 64 bits name no row."""
    least, most = -2 ** 63, 2 ** 63 - 1
    table = torch.arange(1, 5, device="cuda").float()[:, None].expand(4, 9).contiguous()
    t = torch.tensor([least, least + 1, -1, 0, most - 3, most - 1, most], device="cuda")
    for first, named in ((most - 3, [0, 0, 0, 0, 1, 3, 4]), (least, [1, 2, 0, 0, 0, 0, 0]), (-1, [0, 0, 1, 2, 0, 0, 0])):
        y, d = torch.empty(7, 9, device="cuda"), torch.empty_like(table)
        zp.embedding_lookup(table, t, y, first=first)
        assert y[:, 0].tolist() == named
        zp.embedding_grad(torch.ones_like(y), t, d, first=first)
        assert d[:, 8].tolist() == [float(named.count(r + 1)) for r in range(4)]
    small = torch.tensor([-2 ** 31, 2 ** 31 - 1], device="cuda", dtype=torch.int32)
    y = torch.empty(2, 9, device="cuda")
    zp.embedding_lookup(table, small, y, first=2 ** 31 - 2)
    assert y[:, 0].tolist() == [0, 2]
    zp.embedding_lookup(table, small, y, first=most)
    assert y[:, 0].tolist() == [0, 0]
