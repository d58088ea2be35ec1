"""GPU parity of the paged serving operators (rotary positions, page plans,
cache writes of many tokens, attention over 8-bit pages) against plain 64-bit
definitions in numpy.

Tolerances count roundings: a bf16 result is off by at most 2^-8 of its value,
an E4M3 code by 2^-4 of its own (2^-10 absolute below 2^-6), plus the fp32
arithmetic before it, bounded by 2^-20 of the terms' magnitudes (fewer than 16
roundings of 2^-24, with the angle's 2^-23 and sincospi's 2^-22)."""
import ctypes
import math
import random

import numpy as np
import pytest
import torch

import mla_latent_kv_nope_b200 as mla
from oracle import mla_oracle as O

from helpers import f64

pytestmark = pytest.mark.gpu

PAGE = 64
F32 = 2.0 ** -20
BF16 = 2.0 ** -8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True, scope="module")
def _lib():
    from mla_latent_kv_nope_b200 import build
    build.build()
    mla.load_library()
    torch.cuda.set_device(0)


def randn(seed, *shape, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------ rotary positions
def frequencies(d, base=10000.0, scaling="none", factor=1.0, original=4096.0, fast=32.0, slow=1.0):
    k = np.arange(d // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (d / (d - 2))
    f = base ** (-2 * k / d)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        at = lambda n: d * math.log(original / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), d - 1)
        g = np.clip((k - lo) / max(hi - lo, 1e-3), 0, 1)
        return f * (1 - g) + g * f / factor, np.float32(0.1 * math.log(factor) + 1)
    return f, 1.0


def rope64(x, pos, freq, amp, layout, transpose=False):
    """x [T, ..., d] rotated in float64 (angles: exact products of integers and doubles)."""
    d = x.shape[-1]
    th = np.asarray(pos, dtype=np.float64).reshape(-1, *[1] * (x.ndim - 1)) * freq
    c, s = amp * np.cos(th), amp * np.sin(th) * (-1 if transpose else 1)
    i, j = (slice(0, d // 2), slice(d // 2, d)) if layout == "half" else (slice(0, d, 2), slice(1, d, 2))
    y = np.empty_like(x)
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., i] * s + x[..., j] * c
    return y


def check_rope(got, x, pos, freq, amp, layout, transpose, eps):
    ref = rope64(x, pos, freq, amp, layout, transpose)
    d = x.shape[-1]
    i, j = (slice(0, d // 2), slice(d // 2, d)) if layout == "half" else (slice(0, d, 2), slice(1, d, 2))
    mag = np.empty_like(x)
    mag[..., i] = mag[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
    # float64 angles themselves are off by 2^-53 of the angle.
    far = 2.0 ** -52 * np.abs(np.asarray(pos, dtype=np.float64)).max()
    assert np.all(np.abs(got - ref) <= eps * np.abs(ref) + (F32 + far) * amp * mag)


ROPE = [
    # T, H, d_r, dtype, layout, scaling, factor, view
    (1, 1, 64, "bf16", "half", "none", 1.0, False),
    (64, 64, 64, "bf16", "interleaved", "yarn", 32.0, True),
    (7, 5, 64, "bf16", "half", "yarn", 4.0, True),
    (33, 128, 64, "bf16", "half", "linear", 4.0, False),
    (130, 3, 128, "f32", "interleaved", "ntk", 8.0, True),
    (9, 2, 2, "f32", "half", "none", 1.0, False),          # pair kernel: narrow rows
    (9, 3, 24, "bf16", "interleaved", "linear", 2.0, False),
    (5, 7, 256, "bf16", "half", "ntk", 16.0, False),
    (3, 300, 16, "f32", "interleaved", "none", 1.0, False),   # more heads than a block holds
]


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("T,H,d,dtype,layout,scaling,factor,view", ROPE)
def test_rope(T, H, d, dtype, layout, scaling, factor, view, transpose):
    tab = mla.rope_table(d, layout=layout, scaling=scaling, factor=factor)
    full = randn(T + H, T, H, 128 + d, dtype=DT[dtype])
    x = full[..., 128:] if view else full[..., 128:].contiguous()
    rng = random.Random(d)
    pos = [rng.choice([0, 1, 4095, rng.randrange(1 << 20), 2 ** 31 - 1, -5]) for _ in range(T)]
    out = mla.rope(tab, x, i32(pos), transpose=transpose)
    freq, amp = frequencies(d, scaling=scaling, factor=factor)
    eps = BF16 if dtype == "bf16" else 0.0
    check_rope(f64(out), f64(x), pos, freq, amp, layout, transpose, eps)
    # In place, inside the wider rows: the rest of each row stays as it was.
    before = full.clone()
    part = full[..., 128:]
    assert mla.rope(tab, part, i32(pos), out=part, transpose=transpose) is part
    assert torch.equal(part, out) and torch.equal(full[..., :128], before[..., :128])
    # [T, d] rows: one head.
    one = before[:, 0, 128:]
    assert torch.equal(mla.rope(tab, one, i32(pos), transpose=transpose), out[:, 0])
    assert mla.get_device_status() == 0


@pytest.mark.parametrize("off", [1, 4, 8])
def test_rope_unaligned_rows(off):
    """Rows that start off a 16-byte boundary, odd strides, and an output among
    wider rows whose other columns stay."""
    tab = mla.rope_table(64, layout="interleaved")
    x = randn(3, 11, 3, 77, dtype=torch.bfloat16)[..., off:off + 64]
    y = torch.full((11, 3, 90), 7.0, dtype=torch.bfloat16, device="cuda")
    pos = list(range(0, 1100, 100))
    mla.rope(tab, x, i32(pos), out=y[..., off:off + 64])
    freq, amp = frequencies(64)
    check_rope(f64(y[..., off:off + 64]), f64(x), pos, freq, amp, "interleaved", False, BF16)
    assert bool((y[..., :off] == 7).all()) and bool((y[..., off + 64:] == 7).all())


def test_rope_gradient():
    """<v, dR(x)/dx u> = <R^T v, u>, and R^T v against central differences."""
    tab = mla.rope_table(64, scaling="yarn", factor=8.0)
    x, u, v = (randn(s, 6, 2, 64) for s in (1, 2, 3))
    pos = i32([0, 3, 99, 5000, 70000, 123456])
    g = f64(mla.rope(tab, v, pos, transpose=True))
    h = 0.5   # the rotation is linear: differences have no truncation error
    up = f64(mla.rope(tab, x + h * u, pos)) - f64(mla.rope(tab, x - h * u, pos))
    diff = (up / (2 * h) * f64(v)).sum((1, 2))
    mag = (np.abs(f64(x)) + np.abs(f64(u))).sum((1, 2)) * np.abs(f64(v)).max() * 2
    assert np.all(np.abs(diff - (g * f64(u)).sum((1, 2))) <= F32 * 8 * mag)


def test_rope_special_values_and_empty():
    tab = mla.rope_table(64)
    x = randn(5, 4, 1, 64, dtype=torch.bfloat16)
    x[1, 0, 3] = float("inf")
    x[2, 0, 40] = float("nan")
    out = mla.rope(tab, x, i32([5, 5, 5, 5]))
    clean = mla.rope(tab, x[3:], i32([5]))
    assert torch.equal(out[3:], clean)
    assert not torch.isfinite(out[1, 0, [3, 35]]).any() and torch.isnan(out[2, 0, [8, 40]]).all()
    keep = [i for i in range(64) if i not in (3, 35)]
    assert torch.isfinite(out[1, 0, keep]).all()
    assert mla.rope(tab, x[:0], i32([])).shape == (0, 1, 64)


# ------------------------------------------------------------------ page plans
class Pool:
    """Free list and tables of a pool in random page order, on the host and the device."""

    def __init__(self, ctx, num_pages, max_blocks, seed=0):
        rng = random.Random(seed)
        ids = list(range(num_pages))
        rng.shuffle(ids)
        self.table = [[-1] * max_blocks for _ in ctx]
        for b, L in enumerate(ctx):
            for j in range(-(-L // PAGE)):
                self.table[b][j] = ids.pop()
        self.free, self.num_pages, self.max_blocks = ids, num_pages, max_blocks
        self.d_table = i32(self.table)
        self.d_free = torch.full((num_pages,), -7, dtype=torch.int32, device="cuda")
        self.d_free[:len(ids)] = i32(ids)
        self.d_count = i32([len(ids)])
        self.d_len = i32(ctx)

    def plan(self, new, T, in_place=False, request=True):
        B = len(new)
        o = dict(query_start=torch.full((B + 1,), -9, dtype=torch.int32, device="cuda"),
                 positions=torch.full((T,), -9, dtype=torch.int32, device="cuda"),
                 slots=torch.full((T,), -9, dtype=torch.int64, device="cuda"),
                 seqlens_out=self.d_len if in_place else torch.full_like(self.d_len, -9),
                 free_count_out=self.d_count if in_place else torch.full_like(self.d_count, -9),
                 token_request=torch.full((T,), -9, dtype=torch.int32, device="cuda") if request else None)
        ws = torch.zeros(mla.plan_pages_workspace_bytes(), dtype=torch.uint8, device="cuda")
        mla.plan_pages(self.d_len, i32(new), self.d_table, self.d_free, self.d_count,
                       self.num_pages, workspace=ws, **o)
        assert not ws.any()
        return o


def plan64(ctx, new, table, free, T):
    table, free = [list(r) for r in table], list(free)
    qs, pos, slots, req = [0], [], [], []
    for b, (L, n) in enumerate(zip(ctx, new)):
        for j in range(-(-L // PAGE), -(-(L + n) // PAGE)):
            table[b][j] = free.pop()
        for p in range(L, L + n):
            pos.append(p)
            slots.append(table[b][p // PAGE] * PAGE + p % PAGE)
            req.append(b)
        qs.append(qs[-1] + n)
    pad = [-1] * (T - len(pos))
    return qs, pos + pad, slots + pad, req + pad, table, free


def random_requests(B, ctx, new, seed):
    rng = random.Random(seed)
    pick = lambda m: rng.choice([0, 1, 63, 64, 65, rng.randrange(m + 1)])  # noqa: E731
    return [min(pick(ctx), ctx) for _ in range(B)], [min(pick(new), new) for _ in range(B)]


@pytest.mark.parametrize("B,ctx,new,pad,in_place", [
    (1, 0, 1, 0, False), (1, 64, 1, 0, True), (64, 5000, 1, 0, True), (5, 200, 0, 4, False),
    (3, 100, 700, 13, True), (256, 300, 90, 1, True), (257, 300, 90, 0, False),
    (700, 130, 200, 999, True)])
def test_plan_pages(B, ctx, new, pad, in_place):
    L, n = random_requests(B, ctx, new, B)
    T = sum(n) + pad
    max_blocks = (ctx + new + PAGE - 1) // PAGE + 1
    pool = Pool(L, sum(-(-(a + b) // PAGE) for a, b in zip(L, n)) + 3, max_blocks, seed=B)
    before = pool.d_free.clone()
    o = pool.plan(n, T, in_place)
    qs, pos, slots, req, table, free = plan64(L, n, pool.table, pool.free, T)
    assert mla.get_device_status() == 0
    assert o["query_start"].tolist() == qs
    assert o["positions"].tolist() == pos and o["slots"].tolist() == slots
    assert o["token_request"].tolist() == req
    assert pool.d_table.tolist() == table and torch.equal(pool.d_free, before)
    assert o["seqlens_out"].tolist() == [a + b for a, b in zip(L, n)]
    assert o["free_count_out"].tolist() == [len(free)]


def test_plan_pages_large_batch_of_prompts():
    """Many blocks: each expands its own slice; the last one updates in place."""
    B = 600
    rng = random.Random(4)
    L, n = [rng.randrange(300) for _ in range(B)], [rng.randrange(200) for _ in range(B)]
    T = sum(n) + 5000
    pool = Pool(L, sum(-(-(a + b) // PAGE) for a, b in zip(L, n)), 9, seed=1)
    o = pool.plan(n, T, in_place=True, request=False)
    qs, pos, slots, _, table, free = plan64(L, n, pool.table, pool.free, T)
    assert not free and pool.d_count.item() == 0          # the pool is exactly used up
    assert o["slots"].tolist() == slots and o["positions"].tolist() == pos
    assert pool.d_table.tolist() == table and mla.get_device_status() == 0


@pytest.mark.parametrize("why", ["pages", "tokens", "capacity", "negative new", "negative length",
                                 "free count"])
def test_plan_pages_takes_nothing_it_cannot_serve(why):
    L, n, T, blocks = [100, 64, 0], [30, 1, 70], 101, 3
    pool = Pool(L, 3 + 3 + (0 if why == "pages" else 2), blocks)
    if why == "pages":
        pool.d_count -= 1
    if why == "tokens":
        T = 100
    if why == "capacity":
        n[1] = 3 * PAGE - 63
        T = 1000
    if why == "negative new":
        n[0] = -1
    if why == "negative length":
        pool.d_len[2] = -3
    if why == "free count":
        pool.d_count[0] = pool.num_pages + 1
    state = [t.clone() for t in (pool.d_table, pool.d_len, pool.d_count)]
    o = pool.plan(n, T, in_place=True)
    assert mla.get_device_status() == 7                    # MLA_ERR_BOUNDS
    for t, u in zip(state, (pool.d_table, pool.d_len, pool.d_count)):
        assert torch.equal(t, u)
    assert not o["query_start"].any()
    assert (o["slots"] == -1).all() and (o["positions"] == -1).all()


def test_plan_pages_bad_page_ids():
    """A page id outside the pool gives its tokens slot -1; the others are served."""
    pool = Pool([10, 10], 6, 2)
    pool.d_table[0, 0] = 6
    o = pool.plan([2, 2], 4)
    assert mla.get_device_status() == 7
    p = pool.table[1][0]
    assert o["slots"].tolist() == [-1, -1, p * PAGE + 10, p * PAGE + 11]


def test_release_pages():
    L = [0, 1, 64, 65, 500, 128]
    pool = Pool(L, 40, 9)
    release = [1, 0, 1, 1, 0, 7]
    mla.release_pages(pool.d_len, i32(release), pool.d_table, pool.d_free, pool.d_count, 40)
    back = [pool.table[b][j] for b in range(6) if release[b] for j in range(-(-L[b] // PAGE))]
    assert pool.d_count.item() == len(pool.free) + len(back)
    assert pool.d_free[:pool.d_count.item()].tolist() == pool.free + back
    assert pool.d_len.tolist() == [0, 1, 0, 0, 500, 0]
    for b in range(6):
        assert pool.d_table[b].tolist() == ([-1] * 9 if release[b] else pool.table[b])
    assert mla.get_device_status() == 0
    # A bad page id, and a free list that would overflow: nothing changes.
    pool.d_table[4, 2] = 40
    state = [t.clone() for t in (pool.d_len, pool.d_table, pool.d_free, pool.d_count)]
    mla.release_pages(pool.d_len, i32([1] * 6), pool.d_table, pool.d_free, pool.d_count, 40)
    assert mla.get_device_status() == 7
    short = pool.d_free[:pool.d_count.item()].clone()
    mla.release_pages(pool.d_len, i32([0, 1, 0, 0, 0, 0]), pool.d_table, short, pool.d_count, 40)
    assert mla.get_device_status() == 7
    for t, u in zip(state, (pool.d_len, pool.d_table, pool.d_free, pool.d_count)):
        assert torch.equal(t, u)


def test_release_many_requests():
    rng = random.Random(9)
    L = [rng.randrange(0, 200) for _ in range(2500)]
    pool = Pool(L, sum(-(-a // PAGE) for a in L) + 1, 4)
    rel = [rng.randrange(2) for _ in L]
    mla.release_pages(pool.d_len, i32(rel), pool.d_table, pool.d_free, pool.d_count, pool.num_pages)
    back = [pool.table[b][j] for b in range(len(L)) if rel[b] for j in range(-(-L[b] // PAGE))]
    assert pool.d_free[:pool.d_count.item()].tolist() == pool.free + back
    assert mla.get_device_status() == 0


# ----------------------------------------------------- cache writes, 16/32 bits
def row64(x, pos, gamma, d_c, layout, eps=1e-6, rotate=True):
    c = x[:, :d_c] / np.sqrt((x[:, :d_c] ** 2).mean(-1, keepdims=True) + eps) * gamma
    d_r = x.shape[1] - d_c
    k = x[:, d_c:]
    if rotate and d_r:
        freq, amp = frequencies(d_r)
        k = rope64(k, pos, freq, amp, layout)
    return c, k


def check_row(got, c, k, x, d_c, eps):
    # c: the norm is a sum of positive terms, its roundings average below F32.
    assert np.all(np.abs(got[:, :d_c] - c) <= (eps + F32) * np.abs(c))
    if k.shape[1]:
        mag = np.abs(x[:, d_c:]).max(-1, keepdims=True) * 2
        assert np.all(np.abs(got[:, d_c:] - k) <= eps * np.abs(k) + F32 * mag)


@pytest.mark.parametrize("T,d_c,d_r,dtype,layout,fused", [
    (1, 512, 64, "bf16", "half", False), (70, 512, 64, "bf16", "interleaved", True),
    (129, 512, 0, "bf16", "half", False), (33, 32, 16, "f32", "half", True),
    (5, 1024, 128, "f32", "interleaved", False), (6, 1024, 256, "bf16", "half", False),
    (40, 40, 8, "bf16", "interleaved", False), (300, 512, 64, "f32", "interleaved", False)])
def test_cache_write_paged(T, d_c, d_r, dtype, layout, fused):
    R, pages = d_c + d_r, T // PAGE + 2
    dims = mla.Dims(1, 1, d_c, d_r, 16, 16, 64, dtype)
    wide = randn(T, T, R + 64, dtype=DT[dtype])
    x = wide[:, 64:] if fused else wide[:, 64:].contiguous()
    gamma = 1 + 0.3 * randn(2, d_c)
    rng = random.Random(T)
    slots = rng.sample(range(pages * PAGE), T)
    if T > 4:
        slots[T // 2] = slots[-1] = -1
    pos = [rng.randrange(100000) for _ in range(T)]
    pool = torch.full((pages, PAGE, R), 3.0, dtype=DT[dtype], device="cuda")
    tab = mla.rope_table(d_r, layout=layout) if d_r else None
    mla.cache_write_paged(dims, x, gamma, i32(pos), torch.tensor(slots).cuda(), pool, tab)
    assert mla.get_device_status() == 0
    live = [t for t in range(T) if slots[t] >= 0]
    flat = pool.view(-1, R)
    c, k = row64(f64(x)[live], [pos[t] for t in live], f64(gamma), d_c, layout, rotate=d_r > 0)
    check_row(f64(flat[[slots[t] for t in live]]), c, k, f64(x)[live], d_c,
              BF16 if dtype == "bf16" else 0.0)
    rest = [s for s in range(pages * PAGE) if s not in set(slots)]
    assert bool((flat[rest] == 3.0).all())
    # No gamma, no table: the rotary part is stored as it is.
    mla.cache_write_paged(dims, x, None, None, torch.tensor(slots).cuda(), pool)
    assert torch.equal(flat[[slots[t] for t in live]][:, d_c:], x[live][:, d_c:])


def test_cache_write_paged_matches_append():
    """The same row as mla_cache_append_paged writes for the same projection."""
    dims = mla.Dims(3, 16, 512, 64, 128, 128, 128, "bf16")
    h, W = randn(1, 3, 256, dtype=torch.bfloat16), 0.05 * randn(2, 576, 256)
    W = W.to(torch.bfloat16)
    gamma = 1 + 0.1 * randn(3, 512)
    table, L = i32([[0, 1], [2, 3], [4, 5]]), [5, 64, 127]
    a = torch.zeros(6, PAGE, 576, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros_like(a)
    ws = torch.empty(mla.cache_append_workspace_bytes(dims, 256), dtype=torch.uint8, device="cuda")
    mla.cache_append_paged(dims, h, W, gamma, a, table, i32(L), ws)
    x = f64(h) @ f64(W).T      # the append keeps its projection in fp32: compare to bf16 rounding
    xb = torch.from_numpy(x).to(torch.bfloat16).cuda()
    slots = torch.tensor([table[i, L[i] // PAGE].item() * PAGE + L[i] % PAGE for i in range(3)]).cuda()
    mla.cache_write_paged(dims, xb, gamma, i32(L), slots, b, mla.rope_table(64))
    ra, rb = f64(a.view(-1, 576)[slots]), f64(b.view(-1, 576)[slots])
    # x rounded once more (2^-8), in the pair's other member too; both results rounded (2^-8).
    mag = np.abs(rb)
    mag[:, 512:] = np.sqrt(mag[:, 512:544] ** 2 + mag[:, 544:] ** 2).repeat(2, 0).reshape(3, 2, 32).reshape(3, 64)
    assert np.all(np.abs(ra - rb) <= 2 * BF16 * np.abs(rb) + 2 * BF16 * mag + 1e-6)
    assert mla.get_device_status() == 0


def test_cache_write_paged_slot_past_the_pool():
    dims = mla.Dims(1, 1, 512, 64, 128, 128, 64, "bf16")
    pool = torch.zeros(1, PAGE, 576, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([64, 3, 1 << 40], device="cuda")
    mla.cache_write_paged(dims, randn(1, 3, 576, dtype=torch.bfloat16), None, None, slots, pool)
    assert mla.get_device_status() == 7
    assert pool[0, 3].any() and not pool[0, :3].any() and not pool[0, 4:].any()


# --------------------------------------------------------- cache writes, 8 bits
def write8_64(state, x, qs, lens, table, gamma, d_r, layout):
    """The definition, page by page, in float64: `state` = (codes as values, rope, scales)."""
    codes, rope, scales = state
    for b, end in enumerate(lens):
        start = end - (qs[b + 1] - qs[b])
        if start == end:
            continue
        pos = np.arange(start, end)
        c, k = row64(x[qs[b]:qs[b + 1]], pos, gamma, 512, layout, rotate=d_r > 0)
        for j in range(start // PAGE, (end - 1) // PAGE + 1):
            p, lo, hi = table[b][j], max(start, j * PAGE), min(end, (j + 1) * PAGE)
            top = np.abs(c[lo - start:hi - start]).max()
            s = 2.0 ** max(-40, math.ceil(math.log2(top / 448))) if top > 0 else 2.0 ** -40
            r0 = lo % PAGE
            if r0:
                s = max(s, scales[p])
                codes[p, :r0] = O.e4m3_decode(O.e4m3_encode(codes[p, :r0] * (scales[p] / s)))
                rope[p, :r0] *= scales[p] / s
            codes[p, r0:r0 + hi - lo] = c[lo - start:hi - start] / s
            rope[p, r0:r0 + hi - lo] = k[lo - start:hi - start] / s
            scales[p] = s
    return codes, rope, scales


def codes64(pool):
    return O.e4m3_decode(pool[..., :512].cpu().numpy()).astype(np.float64)


def rope_part(pool):
    return f64(pool[..., 512:].contiguous().view(torch.bfloat16))


def check_pages8(pool, scales, codes, rope, ref_scales):
    assert np.array_equal(f64(scales), ref_scales)
    got = codes64(pool)
    assert np.all(np.abs(got - codes) <= np.maximum(2.0 ** -4 * np.abs(codes), 2.0 ** -10)
                  + F32 * np.abs(codes))
    if rope.size:
        g = rope_part(pool)
        # the fp32 rotation's error is relative to the pair: rope keys here are below 8.
        lim = BF16 * np.abs(rope) + F32 * 16 / ref_scales[:, None, None]
        assert np.all(np.abs(g - rope) <= lim)


@pytest.mark.parametrize("ctx,new,d_r,layout,grow", [
    ([0], [1], 64, "half", 1.0), ([0, 63, 64, 65, 127], [1, 1, 1, 1, 1], 64, "half", 1.0),
    ([5, 0, 64, 100, 7], [200, 64, 0, 28, 58], 64, "interleaved", 1.0),
    ([63, 1, 130], [2, 63, 130], 0, "half", 1.0),
    ([10, 63, 40], [1, 1, 100], 64, "half", 9.0),      # larger rows later: pages rescale
    ([33, 50], [3, 4], 64, "interleaved", 0.01),       # smaller rows keep the scale
])
def test_cache_write_fp8_paged(ctx, new, d_r, layout, grow):
    B, R = len(ctx), 512 + d_r
    lens = [a + n for a, n in zip(ctx, new)]
    pool = Pool(lens, sum(-(-n // PAGE) for n in lens) + 2, 8)
    dims = mla.Dims(B, 16, 512, d_r, 128, 128, 8 * PAGE, "bf16")
    tab = mla.rope_table(d_r, layout=layout) if d_r else None
    mem = torch.randint(0, 0x7E, (pool.num_pages, PAGE, 512 + 2 * d_r), dtype=torch.uint8).cuda()
    if d_r:
        mem[..., 512:] = randn(8, pool.num_pages, PAGE, d_r, dtype=torch.bfloat16).view(torch.uint8)
    scales = torch.exp2(torch.randint(-9, -5, (pool.num_pages,)).float()).cuda()
    gamma = grow * (1 + 0.1 * randn(3, 512))
    qs = np.concatenate([[0], np.cumsum(new)]).tolist()
    x = randn(11, qs[-1] + 3, R + 8, dtype=torch.bfloat16)[:, 8:]     # 3 padding rows
    before, old = mem.clone(), (codes64(mem), rope_part(mem) if d_r else np.zeros((0,)), f64(scales))
    if not d_r:
        old = (old[0], np.zeros((pool.num_pages, PAGE, 0)), old[2])
    ref = write8_64([a.copy() for a in old], f64(x), qs, lens, pool.table, f64(gamma), d_r, layout)
    mla.cache_write_fp8_paged(dims, x, gamma, i32(qs), i32(lens), pool.d_table, mem, scales, tab)
    assert mla.get_device_status() == 0
    check_pages8(mem, scales, *ref)
    # Rows behind a sequence's last, and pages without new tokens, bit for bit.
    for b in range(B):
        for j in range(-(-lens[b] // PAGE)):
            p, end = pool.table[b][j], min(PAGE, lens[b] - j * PAGE)
            assert torch.equal(mem[p, end:], before[p, end:])
            if (j + 1) * PAGE <= ctx[b] or new[b] == 0:
                assert torch.equal(mem[p], before[p]) and scales[p].item() == old[2][p]


@pytest.mark.parametrize("ctx,new,d_r,grow", [
    ([40], [7500], 64, 9.0), ([40, 3], [7500, 90], 0, 9.0),    # two blocks to a page
    ([40], [900], 64, 9.0), ([0, 17, 33], [3, 2, 500], 0, 9.0),   # four
])
def test_cache_write_fp8_paged_blocks_that_share_a_page(ctx, new, d_r, grow):
    """Prompts of several lengths: every block of a page uses the maximum of all its rows and
    rescales its part of the earlier ones."""
    B, R, blocks = len(ctx), 512 + d_r, 120
    lens = [a + n for a, n in zip(ctx, new)]
    pool = Pool(lens, sum(-(-n // PAGE) for n in lens) + 2, blocks)
    dims = mla.Dims(B, 16, 512, d_r, 128, 128, blocks * PAGE, "bf16")
    tab = mla.rope_table(d_r) if d_r else None
    mem = torch.randint(0, 0x7E, (pool.num_pages, PAGE, 512 + 2 * d_r), dtype=torch.uint8).cuda()
    if d_r:
        mem[..., 512:] = randn(8, pool.num_pages, PAGE, d_r, dtype=torch.bfloat16).view(torch.uint8)
    scales = torch.exp2(torch.randint(-9, -5, (pool.num_pages,)).float()).cuda()
    gamma = grow * (1 + 0.1 * randn(3, 512))
    qs = np.concatenate([[0], np.cumsum(new)]).tolist()
    x = randn(12, qs[-1], R, dtype=torch.bfloat16)
    # One row in a hundred is far from even, so that a page's maximum lies in one block.
    x[::100, 7] *= 200
    old = (codes64(mem), rope_part(mem) if d_r else np.zeros((pool.num_pages, PAGE, 0)), f64(scales))
    before = mem.clone()
    ref = write8_64([a.copy() for a in old], f64(x), qs, lens, pool.table, f64(gamma), d_r, "half")
    mla.cache_write_fp8_paged(dims, x, gamma, i32(qs), i32(lens), pool.d_table, mem, scales, tab)
    assert mla.get_device_status() == 0
    check_pages8(mem, scales, *ref)
    for b in range(B):
        j = (lens[b] - 1) // PAGE
        p, end = pool.table[b][j], lens[b] - j * PAGE
        assert torch.equal(mem[p, end:], before[p, end:])


def test_cache_write_fp8_paged_token_by_token():
    """One token at a time gives the page's scale of a whole write, codes within a
    second rounding, and a fresh page ignores what its scale was before."""
    dims = mla.Dims(1, 16, 512, 64, 128, 128, 128, "bf16")
    tab, n = mla.rope_table(64), 70
    x = randn(5, n, 576, dtype=torch.bfloat16)
    x[:, :512] *= torch.linspace(0.5, 4, n, device="cuda")[:, None].to(torch.bfloat16)
    gamma = torch.linspace(0.1, 3.0, 512, device="cuda")
    table = i32([[1, 0]])
    mems = [torch.full((2, PAGE, 640), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scs = [torch.full((2,), float("nan"), device="cuda") for _ in range(2)]
    mla.cache_write_fp8_paged(dims, x, gamma, i32([0, n]), i32([n]), table, mems[0], scs[0], tab)
    for t in range(n):
        mla.cache_write_fp8_paged(dims, x[t:t + 1], gamma, i32([0, 1]), i32([t + 1]), table,
                                  mems[1], scs[1], tab)
    assert mla.get_device_status() == 0 and torch.equal(scs[0], scs[1])
    for p, rows in ((1, 64), (0, 6)):
        a, b = codes64(mems[0][p, :rows]), codes64(mems[1][p, :rows])
        assert np.all(np.abs(a - b) <= np.maximum(2 * 2.0 ** -4 * np.abs(a), 2 * 2.0 ** -9))
        assert torch.equal(mems[0][p, :rows, 512:], mems[1][p, :rows, 512:])


def test_cache_write_fp8_paged_zero_rows_and_bad_lengths():
    dims = mla.Dims(5, 16, 512, 64, 128, 128, 128, "bf16")
    mem = torch.full((8, PAGE, 640), 0x11, dtype=torch.uint8, device="cuda")
    scales = torch.full((8,), 2.0, device="cuda")
    x = torch.zeros(6, 576, dtype=torch.bfloat16, device="cuda")
    table = i32([[0, 1], [2, 3], [4, 99], [5, -1], [7, 7]])
    # zeros; length below its count; page id past the pool; past the capacity; past T.
    mla.cache_write_fp8_paged(dims, x, None, i32([0, 1, 3, 4, 5, 7]), i32([1, 1, 70, 129, 9]), table,
                              mem, scales, mla.rope_table(64))
    assert mla.get_device_status() == 7
    assert not mem[0, 0].any() and scales[0].item() == 2.0 ** -40
    assert (mem[0, 1:] == 0x11).all() and (mem[1:] == 0x11).all() and (scales[1:] == 2.0).all()


# --------------------------------------------------- attention over 8-bit pages
def make_pages(lens, H, d_r, seed, spread=2, fill=0xFF):
    """A pool whose rows past each sequence's end, and unused pages, hold NaNs."""
    blocks = [-(-n // PAGE) for n in lens]
    num = sum(blocks) + 2
    rng = np.random.default_rng(seed)
    ids = rng.permutation(num)
    max_blocks = max(max(blocks), 1) + 1
    table = np.full((len(lens), max_blocks), -1, dtype=np.int32)
    pool = np.full((num, PAGE, 512 + 2 * d_r), fill, dtype=np.uint8)
    scales = np.full(num, np.nan, dtype=np.float32)
    rows, at = {}, 0
    for b, n in enumerate(lens):
        seq = []
        for j in range(blocks[b]):
            p = ids[at]
            at += 1
            table[b, j] = p
            m = min(PAGE, n - j * PAGE)
            s = 2.0 ** (-6 - int(rng.integers(0, spread + 1)))
            codes = O.e4m3_encode(np.clip(rng.standard_normal((m, 512)) / s, -448, 448))
            k = torch.from_numpy(rng.standard_normal((m, d_r)) / s).to(torch.bfloat16)
            pool[p, :m, :512] = codes
            if d_r:
                pool[p, :m, 512:] = k.view(torch.uint8).numpy().reshape(m, 2 * d_r)
            scales[p] = s
            seq.append(np.concatenate([O.e4m3_decode(codes), k.double().numpy()], 1) * s)
        rows[b] = np.concatenate(seq) if seq else np.zeros((0, 512 + d_r))
    return (torch.from_numpy(pool).cuda(), torch.from_numpy(scales).cuda(),
            torch.from_numpy(table).cuda(), rows)


def attend64(q, rows, scale):
    z = q @ rows.T * scale
    m = z.max(-1, keepdims=True)
    p = np.exp(z - m)
    return (p @ rows[:, :512]) / p.sum(-1, keepdims=True), (m + np.log(p.sum(-1, keepdims=True)))[:, 0], z


def run_decode8(dims, q, pool, scales, table, seq, scale, W=0):
    ws = torch.full((mla.decode_workspace_bytes(dims, W) // 4,), float("nan"), device="cuda")
    used = mla.decode_fp8_paged(dims, q, pool, scales, table, seq, scale, ws, W)
    o = torch.full((dims.B, dims.H, 512), float("nan"), device="cuda")
    lse = torch.full((dims.B, dims.H), float("nan"), device="cuda")
    mla.combine(dims, seq, ws, used, o, lse)
    return o, lse


def check_attend(o, lse, q, rows, lens, scale):
    """A probability is hi (E4M3, off by 2^-4 of itself at most) plus lo, the rest in E5M2
    (2^-3 of that), after a rounding to fp16 (2^-11): 2^-7 + 2^-11 < 2^-6.9 of itself at
    most.  The bound below takes half of that, 2^-8: the roundings of the 8 and more keys
    that a row's weight spreads over here do not all point one way, and with a single key
    p / l = 1 is exact (p is a power of two there).  Probabilities far below their
    tile's largest are rounded to 2^-13 of it at least: 128 keys' 2^-15 of the largest term.
    Scores come from exact products with fp32 sums (2^-20); the query's own two terms
    leave 2^-18 of its row's largest value per element."""
    for b, n in enumerate(lens):
        if n == 0:
            assert bool((o[b] == 0).all()) and bool(torch.isneginf(lse[b]).all())
            continue
        qb, r = f64(q[b]), rows[b]
        ref, ref_lse, z = attend64(qb, r, scale)
        dz = scale * (np.abs(qb) @ np.abs(r).T * F32
                      + 2.0 ** -18 * np.abs(qb).max(-1, keepdims=True) * np.abs(r).sum(-1)).max(-1)
        p = np.exp(z - ref_lse[:, None])
        lim = (p * (2.0 ** -8 + 2 * dz[:, None])) @ np.abs(r[:, :512])
        lim += 2.0 ** -13 * 128 * 2.0 ** -2 * p.max(-1, keepdims=True) * np.abs(r[:, :512]).max()
        assert np.all(np.abs(f64(o[b]) - ref) <= lim + 1e-6)
        assert np.all(np.abs(f64(lse[b]) - ref_lse) <= 2 * dz + 1e-5)


DECODE8 = [
    # lens, H, d_r, splits, boost
    ([1], 1, 64, 0, 1.0), ([600, 129, 1], 128, 64, 0, 1.0), ([600, 129, 1], 128, 0, 0, 1.0),
    ([1, 63, 64, 65, 127, 128, 129, 200, 0], 128, 64, 0, 1.0),
    ([900, 77], 128, 64, 7, 10.0), ([700, 1, 333, 64, 0], 64, 64, 0, 1.0),
    ([300, 65, 5, 64], 16, 64, 3, 1.0), ([2000], 8, 64, 0, 1.0), ([513, 64], 100, 64, 1, 3.0),
    ([260, 0, 31], 192, 64, 0, 1.0), ([5000], 40, 0, 5, 2.0), ([0, 0], 128, 64, 0, 1.0),
]


@pytest.mark.parametrize("lens,H,d_r,W,boost", DECODE8)
def test_decode_fp8_paged(lens, H, d_r, W, boost):
    B = len(lens)
    pool, scales, table, rows = make_pages(lens, H, d_r, seed=H + B)
    dims = mla.Dims(B, H, 512, d_r, 128, 128, table.shape[1] * PAGE, "bf16")
    q = randn(H, B, H, 512 + d_r, dtype=torch.bfloat16)
    scale = boost / math.sqrt(128 + d_r)
    o, lse = run_decode8(dims, q, pool, scales, table, i32(lens), scale, W)
    assert mla.get_device_status() == 0
    check_attend(o, lse, q, rows, lens, scale)


@pytest.mark.parametrize("kind", ["sink", "scales apart", "late maximum", "falling", "large query"])
def test_decode_fp8_paged_uneven(kind):
    """One key that outweighs thousands of small ones, pages whose scales lie far
    apart, maxima that keep growing or fall by many powers of two."""
    H, lens = 128, [4000, 1000]
    pool, scales, table, rows = make_pages(lens, H, 64, seed=77)
    dims = mla.Dims(2, H, 512, 64, 128, 128, table.shape[1] * PAGE, "bf16")
    q = randn(9, 2, H, 576, dtype=torch.bfloat16)
    scale = 1 / math.sqrt(192)
    if kind == "scales apart":
        f = torch.exp2(torch.randint(-12, 3, scales.shape, generator=torch.Generator().manual_seed(1)).float()).cuda()
        scales.mul_(f)
        for b, n in enumerate(lens):
            for j in range(-(-n // PAGE)):
                rows[b][j * PAGE:(j + 1) * PAGE] *= f[table[b, j]].item()
    elif kind == "large query":
        q *= 1000
        scale /= 1000
    else:
        # Scores set through the rotary keys: with q_r = e_0 the row's k_0 is its score.
        q[:, :, 512:] = 0
        q[:, :, 512] = 16
        q[:, :, :512] *= 0.05
        for b, n in enumerate(lens):
            j = np.arange(n)
            want = {"sink": np.where(j == 3, 12.0, 0.0),
                    "late maximum": 30.0 * j / n, "falling": -30.0 * j / n}[kind]
            for t in range(-(-n // PAGE)):
                p, m = table[b, t].item(), min(PAGE, n - t * PAGE)
                s = scales[p].item()
                v = torch.from_numpy(want[t * PAGE:t * PAGE + m] / scale / 16 / s).to(torch.bfloat16)
                k = pool[p, :m, 512:].contiguous().view(torch.bfloat16)
                k[:, 0] = v.cuda()
                pool[p, :m, 512:] = k.view(torch.uint8)
                rows[b][t * PAGE:t * PAGE + m, 512] = v.double().numpy() * s
    o, lse = run_decode8(dims, q, pool, scales, table, i32(lens), scale)
    assert mla.get_device_status() == 0
    check_attend(o, lse, q, rows, lens, scale)
    for b in range(2):
        ref = attend64(f64(q[b]), rows[b], scale)[0]
        assert np.linalg.norm(f64(o[b]) - ref) <= 5e-3 * np.linalg.norm(ref)


# lse = (log2 l + r - 6.75) ln 2 with l = n 2^39 and r = -32.25: log2 l < 48 is off by an ulp
# of 2^-18, the rest by half an ulp of numbers below 16, and the combine adds a few of 2^-21.
ZERO_LSE = 2.0 * 2.0 ** -18


def zero_pages(lens, H, d_r, zero_blocks):
    """make_pages with the rows of blocks `zero_blocks` as the writer leaves zero latents: zero
    codes and a scale of 2^-40 (rotary keys as they are)."""
    pool, scales, table, rows = make_pages(lens, H, d_r, seed=H + d_r + 5)
    for b, n in enumerate(lens):
        for j in zero_blocks:
            m = min(PAGE, n - j * PAGE)
            if m <= 0:
                continue
            p = table[b, j].item()
            pool[p, :m, :512] = 0
            k = pool[p, :m, 512:].contiguous().view(torch.bfloat16)
            pool[p, :m, 512:] = (k.float() * (scales[p] * 2.0 ** 40)).to(torch.bfloat16).view(torch.uint8)
            scales[p] = 2.0 ** -40
            rows[b][j * PAGE:j * PAGE + m, :512] = 0
    return pool, scales, table, rows


@pytest.mark.parametrize("H", [16, 64, 128])
@pytest.mark.parametrize("q_pe", [1.0, 300.0, 2.0 ** 100])
def test_decode_fp8_paged_zero_latent_query(H, q_pe):
    """Heads whose latent query is zero (all of them in the first sequence, some among
    others in the second), with rotary parts of any size: their scores are the rotary
    products alone."""
    lens = [65, 200, 1, 63]
    pool, scales, table, rows = make_pages(lens, H, 64, seed=H)
    dims = mla.Dims(4, H, 512, 64, 128, 128, table.shape[1] * PAGE, "bf16")
    q = randn(H + 1, 4, H, 576, dtype=torch.bfloat16)
    q[0, :, :512] = 0
    q[1, 3::5, :512] = 0
    q[3, ::2, :512] = 1e-30                 # next to nothing, but not zero
    zero = ~(q[:, :, :512].abs() > 1e-20).any(-1)
    q[..., 512:] *= torch.where(zero, q_pe, 1.0)[..., None].to(torch.bfloat16)
    scale = 1 / math.sqrt(192) / max(q_pe / 300, 1.0)
    o, lse = run_decode8(dims, q, pool, scales, table, i32(lens), scale)
    assert mla.get_device_status() == 0
    check_attend(o, lse, q, rows, lens, scale)
    # Where the latent part is zero the two terms leave nothing out: fp32 sums alone.
    for b, n in enumerate(lens):
        h = zero[b].cpu().numpy()
        qb = f64(q[b])[h]
        if not len(qb):
            continue
        ref, ref_lse, z = attend64(qb, rows[b], scale)
        dz = scale * F32 * (np.abs(qb) @ np.abs(rows[b]).T).max(-1)
        p = np.exp(z - ref_lse[:, None])
        lim = (p * (2.0 ** -7 + 2.0 ** -11 + 2 * dz[:, None])) @ np.abs(rows[b][:, :512])
        lim += 2.0 ** -15 * n * p.max(-1, keepdims=True) * np.abs(rows[b][:, :512]).max()
        assert np.all(np.abs(f64(o[b])[h] - ref) <= lim + 1e-6)
        assert np.all(np.abs(f64(lse[b])[h] - ref_lse) <= 2 * dz + 1e-5)


@pytest.mark.parametrize("H,d_r", [(16, 64), (64, 64), (128, 64), (64, 0), (128, 0)])
@pytest.mark.parametrize("scale", [0.07, 1e-44])
def test_decode_fp8_paged_zero_query_and_zero_pages(H, d_r, scale):
    """Zero queries over pages of zero latents with a partly filled last page (a request of
    zeros): every key weighs the same, lse = log n.  Scores of next to nothing the same."""
    lens = [1, 63, 65, 300, 64]
    pool, scales, table, rows = zero_pages(lens, H, d_r, (0, 1, 4))
    dims = mla.Dims(5, H, 512, d_r, 128, 128, table.shape[1] * PAGE, "bf16")
    q = randn(3, 5, H, 512 + d_r, dtype=torch.bfloat16)
    q[:3] = 0
    q[3, 1::3] = 0
    o, lse = run_decode8(dims, q, pool, scales, table, i32(lens), scale)
    assert mla.get_device_status() == 0
    check_attend(o, lse, q, rows, lens, scale)
    for b in range(3):
        assert bool((lse[b] - math.log(lens[b])).abs().max() <= ZERO_LSE)
        assert not o[b].any()


@pytest.mark.parametrize("H", [16, 128])
def test_paged_cache_step_of_zeros(H):
    """A request of zero rows and zero queries through PagedCache and DecodeStep (a dummy
    step before serving): zeros, and lse = log n."""
    dims = mla.Dims(2, H, 512, 64, 128, 128, 128, "bf16")
    tab = mla.rope_table(64)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    cache = mla.PagedCache(dims, num_pages=4, max_tokens=128, fp8=True, table=tab)
    step = mla.DecodeStep(dims, (0.05 * randn(1, H, 128, 512)).to(torch.bfloat16),
                          (0.05 * randn(2, H, 128, 512)).to(torch.bfloat16), rope_table=tab)
    cache.plan(i32([70, 5]), tokens=75)
    cache.write(z(75, 576))
    out = step(z(2, H, 128), z(2, H, 64), cache.last_positions(), cache.pool, cache.seqlens,
               block_table=cache.block_table, page_scales=cache.page_scales)
    assert mla.get_device_status() == 0 and not out.any()
    want = torch.tensor([math.log(70), math.log(5)], device="cuda")[:, None]
    assert bool((step.lse - want).abs().max() <= ZERO_LSE)


@pytest.mark.parametrize("H,d", [(H, d) for H in (64, 128) for d in (7.0, 9.5, 10.5, 12.0)])
def test_decode_fp8_paged_weights_far_below_their_tile(H, d):
    """The stated bound of a weight, where it is worst: tiles whose one large key lies at the
    lower edge of the reference's window (5.2 binades below the first tile's keys, which put
    the reference 7.75 above them, with a window of 13), the others d binades below that."""
    lens, per = [20 * PAGE], 2 if H > 64 else 1
    pool, scales, table, rows = make_pages(lens, H, 64, seed=H, spread=0)
    dims = mla.Dims(1, H, 512, 64, 128, 128, table.shape[1] * PAGE, "bf16")
    scale = 1 / math.sqrt(192)
    q = torch.zeros(1, H, 576, dtype=torch.bfloat16, device="cuda")
    q[:, :, 512] = 16
    j = np.arange(lens[0])
    tile = j // (per * PAGE)
    bits = np.where(tile == 0, 0.0, np.where(j % (per * PAGE) == 5, -5.2, -5.2 - d))
    want = bits * math.log(2) / scale / 16
    rows[0][:, 512:] = 0
    for t in range(20):
        pg, s = table[0, t].item(), scales[table[0, t]].item()
        k = torch.zeros(PAGE, 64, dtype=torch.bfloat16)
        k[:, 0] = torch.from_numpy(want[t * PAGE:(t + 1) * PAGE] / s).to(torch.bfloat16)
        pool[pg, :, 512:] = k.view(torch.uint8).cuda()
        rows[0][t * PAGE:(t + 1) * PAGE, 512] = k[:, 0].double().numpy() * s
    o, lse = run_decode8(dims, q, pool, scales, table, i32(lens), scale, 1)
    assert mla.get_device_status() == 0
    ref, ref_lse, z = attend64(f64(q[0]), rows[0], scale)
    p = np.exp(z - ref_lse[:, None])
    top = np.stack([p[:, tile == t].max(-1) for t in range(tile.max() + 1)], -1)[:, tile]
    # (fp16 before the two terms 2^-11, the score 2^-20 of itself.)
    c = np.abs(rows[0][:, :512])
    lim = (p * (2.0 ** -7 + 2.0 ** -11 + F32 * np.abs(z)) + 2.0 ** -10.7 * top) @ c
    assert np.all(np.abs(f64(o[0]) - ref) <= lim)
    assert np.all(np.abs(f64(lse[0]) - ref_lse) <= F32 * np.abs(z).max() + 1e-5)


def test_decode_fp8_paged_bad_page_and_long_length():
    """A page id outside the pool reads as zeros and is reported; a length past the
    capacity is cut to it."""
    pool, scales, table, rows = make_pages([200], 16, 64, seed=3)
    dims = mla.Dims(1, 16, 512, 64, 128, 128, 192, "bf16")
    q = randn(1, 1, 16, 576, dtype=torch.bfloat16)
    o, lse = run_decode8(dims, q, pool, scales, table[:, :3].contiguous(), i32([5000]), 0.05)
    mla.get_device_status()
    check_attend(o, lse, q, {0: rows[0][:192]}, [192], 0.05)
    bad = table.clone()
    bad[0, 1] = pool.shape[0]
    dims = mla.Dims(1, 16, 512, 64, 128, 128, table.shape[1] * PAGE, "bf16")
    o, lse = run_decode8(dims, q, pool, scales, bad, i32([200]), 0.05)
    assert mla.get_device_status() == 7
    r = rows[0].copy()
    r[64:128] = 0
    check_attend(o, lse, q, {0: r}, [200], 0.05)


@pytest.mark.parametrize("B,H", [(500, 16), (500, 128), (1100, 64), (900, 128)])
def test_decode_fp8_paged_many_sequences(B, H):
    """More sequences than a block has threads, many of them per worker, empty ones among
    them."""
    rng = random.Random(B + H)
    lens = [rng.choice([0, 1, 5, 64, 65, 130, 200]) for _ in range(B)]
    pool, scales, table, rows = make_pages(lens, H, 64, seed=B)
    dims = mla.Dims(B, H, 512, 64, 128, 128, table.shape[1] * PAGE, "bf16")
    q = randn(B, B, H, 576, dtype=torch.bfloat16)
    o, lse = run_decode8(dims, q, pool, scales, table, i32(lens), 0.07)
    assert mla.get_device_status() == 0
    some = rng.sample(range(B), 40)
    check_attend(o[some], lse[some], q[some], {k: rows[b] for k, b in enumerate(some)},
                 [lens[b] for b in some], 0.07)
    empty = [b for b in range(B) if lens[b] == 0]
    assert not o[empty].any() and torch.isneginf(lse[empty]).all()


@pytest.mark.parametrize("H", [64, 128])
def test_fp8_paged_offsets_past_32_bits(H):
    """Pages whose bytes lie past 2^32 of a pool of 4.6 GB, written and attended."""
    n_pages, lens = 112000, [130, 64]
    dims = mla.Dims(2, H, 512, 64, 128, 128, 256, "bf16")
    pool = torch.empty(n_pages, PAGE, 640, dtype=torch.uint8, device="cuda")
    scales = torch.empty(n_pages, device="cuda")
    ids = [n_pages - 1, 3, n_pages - 2, 111000]
    table = i32([[ids[0], ids[1], ids[2], -1], [ids[3], -1, -1, -1]])
    pool[ids] = 0xFF
    x = randn(4, sum(lens), 576, dtype=torch.bfloat16)
    mla.cache_write_fp8_paged(dims, x, None, i32([0, 130, 194]), i32(lens), table, pool, scales)
    q = randn(5, 2, H, 576, dtype=torch.bfloat16)
    o, lse = run_decode8(dims, q, pool, scales, table, i32(lens), 0.07)
    assert mla.get_device_status() == 0
    rows, at = {}, 0
    for b, n in enumerate(lens):
        p = [t for t in table[b].tolist() if t >= 0]
        sc = f64(scales[p])[:, None, None]
        c, k = codes64(pool[p]) * sc, rope_part(pool[p]) * sc
        rows[b] = np.concatenate([c, k], 2).reshape(-1, 576)[:n]
        want, _ = row64(f64(x[at:at + n]), np.arange(n), 1.0, 512, "half", rotate=False)
        assert np.linalg.norm(rows[b][:, :512] - want) < 2.0 ** -4 * np.linalg.norm(want)
        at += n
    check_attend(o, lse, q, rows, lens, 0.07)
    # The bf16 writer at a slot whose bytes lie past 2^32.
    big = torch.empty(60000, PAGE, 576, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([60000 * 64 - 1, 5], device="cuda")
    mla.cache_write_paged(dims, x[:2], None, None, slots, big)
    assert torch.equal(big.view(-1, 576)[slots][:, 512:], x[:2, 512:])


@pytest.mark.parametrize("H,d_r", [(64, 64), (128, 64), (64, 0), (128, 0)])
def test_decode_fp8_paged_gives_up(H, d_r):
    """A wait that runs out (nothing arrives on its barrier) ends the kernel with a status
    and leaves the context usable: the next decode is right."""
    lens = [700, 65, 1]
    pool, scales, table, rows = make_pages(lens, H, d_r, seed=2)
    dims = mla.Dims(3, H, 512, d_r, 128, 128, table.shape[1] * PAGE, "bf16")
    q = randn(6, 3, H, 512 + d_r, dtype=torch.bfloat16)
    assert mla.get_device_status() == 0
    try:
        mla.debug_inject_wait(200_000)      # about 0.1 ms of SM cycles
        run_decode8(dims, q, pool, scales, table, i32(lens), 0.07)
        status = mla.get_device_status()
    finally:
        mla.debug_inject_wait(0)
    assert status == 6                      # MLA_ERR_DEVICE_TIMEOUT
    o, lse = run_decode8(dims, q, pool, scales, table, i32(lens), 0.07)
    assert mla.get_device_status() == 0
    check_attend(o, lse, q, rows, lens, 0.07)


def test_two_streams_at_once():
    """Two decodes with a workspace each, on two streams, and a repeated one: the same bits."""
    cases = []
    for H, lens in ((128, [3000, 100, 77]), (64, [5000, 64])):
        pool, scales, table, rows = make_pages(lens, H, 64, seed=H)
        dims = mla.Dims(len(lens), H, 512, 64, 128, 128, table.shape[1] * PAGE, "bf16")
        q = randn(H, len(lens), H, 576, dtype=torch.bfloat16)
        cases.append((dims, q, pool, scales, table, i32(lens)))
    alone = [run_decode8(*c, 0.07) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        got = []
        for c, s in zip(cases, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(run_decode8(*c, 0.07))
        torch.cuda.synchronize()
        for (o, l), (o1, l1) in zip(alone, got):
            assert torch.equal(o, o1) and torch.equal(l, l1)
    assert mla.get_device_status() == 0


# ------------------------------------------------------------------- together
@pytest.mark.parametrize("fp8", [True, False])
def test_paged_cache_with_decode_steps(fp8):
    """PagedCache and DecodeStep: prompts, decode steps, a finished request's pages used
    again; the step's output against materialised attention over the written rows."""
    B, H = 3, 16
    dims = mla.Dims(B, H, 512, 64, 128, 128, 256, "bf16")
    tab = mla.rope_table(64, layout="interleaved", scaling="yarn", factor=4.0)
    freq, amp = frequencies(64, scaling="yarn", factor=4.0)
    W_UK = (0.05 * randn(1, H, 128, 512)).to(torch.bfloat16)
    W_UV = (0.05 * randn(2, H, 128, 512)).to(torch.bfloat16)
    cache = mla.PagedCache(dims, num_pages=8, max_tokens=256, fp8=fp8, table=tab)
    step = mla.DecodeStep(dims, W_UK, W_UV, rope_table=tab)
    xs = [np.zeros((0, 576)) for _ in range(B)]
    for it, new in enumerate([[70, 3, 0], [1, 1, 100], [1, 1, 1], "release 0", [2, 1, 1], [150, 1, 1]]):
        if new == "release 0":
            cache.release(i32([1, 0, 0]))
            xs[0] = xs[0][:0]
            continue
        cache.plan(i32(new))
        x = randn(it, sum(new), 576, dtype=torch.bfloat16)
        cache.write(x)
        at = 0
        for b in range(B):
            xs[b] = np.concatenate([xs[b], f64(x[at:at + new[b]])])
            at += new[b]
        qn = randn(20 + it, B, H, 128, dtype=torch.bfloat16)
        qp = randn(40 + it, B, H, 64, dtype=torch.bfloat16)
        out = step(qn, qp, cache.last_positions(), cache.pool, cache.seqlens,
                   block_table=cache.block_table, page_scales=cache.page_scales)
        assert mla.get_device_status() == 0
        assert cache.seqlens.tolist() == [len(v) for v in xs]
        used = sum(-(-len(v) // PAGE) for v in xs)
        assert cache.free_count.item() == 8 - used
        for b in range(B):
            n = len(xs[b])
            if n == 0:
                assert not out[b].any()
                continue
            c = xs[b][:, :512] / np.sqrt((xs[b][:, :512] ** 2).mean(-1, keepdims=True) + 1e-6)
            k = rope64(xs[b][:, 512:], np.arange(n), freq, amp, "interleaved")
            q = np.concatenate([np.einsum("hn,hnc->hc", f64(qn[b]), f64(W_UK)),
                                rope64(f64(qp[b])[None], [n - 1], freq, amp, "interleaved")[0]], 1)
            ref, _, _ = attend64(q, np.concatenate([c, k], 1), 1 / math.sqrt(192))
            ref = np.einsum("hc,hvc->hv", ref, f64(W_UV))
            # bf16 queries, probabilities and outputs; E4M3 rows where the cache is 8-bit.
            lim = 2.0 ** -4 if fp8 else 1.5e-2
            assert np.linalg.norm(f64(out[b]) - ref) < lim * np.linalg.norm(ref)
    with pytest.raises(ValueError, match="before the step"):
        step(qn, qp, cache.last_positions(), cache.pool, cache.seqlens, h=x,
             block_table=cache.block_table, page_scales=cache.page_scales)
    with pytest.raises(ValueError, match="block_table"):
        mla.DecodeStep(dims, W_UK, W_UV)(qn, qp, cache.last_positions(), cache.pool, cache.seqlens,
                                         page_scales=torch.ones(8, device="cuda"))
    with pytest.raises(ValueError, match="rope_table"):
        mla.DecodeStep(dims, W_UK, W_UV, rope_table=mla.rope_table(32))


def test_paged_serving_run():
    """Prompts in chunks, then decode steps from a captured graph: plan, write,
    rotate, attend; the 8-bit pages against attention over the same rows in 64
    bits, and the bf16 pages through mla_decode_paged."""
    B, H, T, blocks = 3, 64, 160, 4
    d8 = mla.Dims(B, H, 512, 64, 128, 128, blocks * PAGE, "bf16")
    tab = mla.rope_table(64, layout="interleaved", scaling="yarn", factor=4.0)
    freq, amp = frequencies(64, scaling="yarn", factor=4.0)
    pool = Pool([0] * B, B * blocks, blocks)
    mem8 = torch.full((pool.num_pages, PAGE, 640), 0xFF, dtype=torch.uint8, device="cuda")
    sc = torch.full((pool.num_pages,), float("nan"), device="cuda")
    mem16 = torch.full((pool.num_pages, PAGE, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    gamma = 1 + 0.1 * randn(6, 512)
    W_UV = (0.05 * randn(7, H, 128, 512)).to(torch.bfloat16)
    plan_ws = torch.zeros(mla.plan_pages_workspace_bytes(), dtype=torch.uint8, device="cuda")
    ws = torch.empty(mla.decode_workspace_bytes(d8) // 4, device="cuda")
    e = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    buf = dict(x=torch.zeros(T, 576, dtype=torch.bfloat16, device="cuda"), new=i32([0] * B),
               qs=e(B + 1, dt=torch.int32), pos=e(T, dt=torch.int32), slots=e(T, dt=torch.int64),
               q=torch.zeros(B, H, 576, dtype=torch.bfloat16, device="cuda"))
    o, lse, out = e(B, H, 512), e(B, H), e(B, H, 128, dt=torch.bfloat16)
    o16, l16 = e(B, H, 512), e(B, H)
    q_last = i32([0] * B)

    def step():
        mla.plan_pages(pool.d_len, buf["new"], pool.d_table, pool.d_free, pool.d_count,
                       pool.num_pages, buf["qs"], buf["pos"], buf["slots"], pool.d_len, pool.d_count,
                       plan_ws)
        mla.cache_write_fp8_paged(d8, buf["x"], gamma, buf["qs"], pool.d_len, pool.d_table, mem8, sc, tab)
        mla.cache_write_paged(d8, buf["x"], gamma, buf["pos"], buf["slots"], mem16, tab)
        torch.sub(pool.d_len, 1, out=q_last)
        qr = buf["q"][..., 512:]
        mla.rope(tab, qr, q_last, out=qr)
        used = mla.decode_fp8_paged(d8, buf["q"], mem8, sc, pool.d_table, pool.d_len, 0.0, ws)
        mla.combine(d8, pool.d_len, ws, used, o, lse)
        mla.out_proj(d8, o, W_UV, out)
        used = mla.decode_paged(d8, buf["q"], mem16, pool.d_table, pool.d_len, 0.0, ws)
        mla.combine(d8, pool.d_len, ws, used, o16, l16)

    xs, lens = [[] for _ in range(B)], [0] * B

    def feed(new, seed):
        n = sum(new)
        buf["x"].copy_(randn(seed, T, 576, dtype=torch.bfloat16))
        buf["new"].copy_(i32(new))
        q = randn(seed + 50, B, H, 576, dtype=torch.bfloat16)
        buf["q"].copy_(q)
        x, at = f64(buf["x"]), 0
        for b in range(B):
            xs[b].append(x[at:at + new[b]])
            at += new[b]
            lens[b] += new[b]
        assert at == n <= T
        return f64(q)

    def check(q):
        assert mla.get_device_status() == 0 and pool.d_len.tolist() == lens
        for b in range(B):
            x = np.concatenate(xs[b])
            c = x[:, :512] / np.sqrt((x[:, :512] ** 2).mean(-1, keepdims=True) + 1e-6) * f64(gamma)
            k = rope64(x[:, 512:], np.arange(len(x)), freq, amp, "interleaved")
            qq = np.concatenate([q[b, :, :512], rope64(q[b, None, :, 512:], [lens[b] - 1], freq, amp,
                                                       "interleaved")[0]], 1)
            qq = np.asarray(torch.from_numpy(qq).to(torch.bfloat16).double())
            ref, rl, _ = attend64(qq, np.concatenate([c, k], 1), 1 / math.sqrt(192))
            rel = lambda a, r: np.linalg.norm(a - r) / np.linalg.norm(r)  # noqa: E731
            assert rel(f64(o16[b]), ref) < 1e-2
            # E4M3 latents: 2^-4 at most per value, uniform below that: 2^-4 / sqrt(3) of the rms.
            assert rel(f64(o[b]), ref) < 2.0 ** -4
            assert rel(f64(out[b]), np.einsum("hc,hvc->hv", f64(o[b]), f64(W_UV))) < 1e-2

    for i, new in enumerate([[100, 0, 37], [28, 64, 1], [1, 1, 90]]):
        q = feed(new, i)
        step()
        if min(lens):
            check(q)
    g = torch.cuda.CUDAGraph()
    keep = [t.clone() for t in (pool.d_len, pool.d_table, pool.d_count, mem8, sc, mem16)]
    feed([1, 1, 1], 20)
    with torch.cuda.graph(g):
        step()
    for t, k in zip((pool.d_len, pool.d_table, pool.d_count, mem8, sc, mem16), keep):
        assert torch.equal(t.view(torch.uint8), k.view(torch.uint8))
    g.replay()
    check(f64(randn(70, B, H, 576, dtype=torch.bfloat16)))
    for i in range(3):
        q = feed([1, 1, 0 if i == 1 else 1], 30 + i)
        g.replay()
        check(q)


def test_cache_write_fp8_paged_reports_a_bad_length_behind_many_requests():
    """More requests than a block looks at together, a page for each row of x, and a
    length that does not fit behind them: reported, the others written."""
    B, n = 1100, 600
    dims = mla.Dims(B, 16, 512, 64, 128, 128, PAGE, "bf16")
    new = [1] * n + [0] * (B - n)
    qs = np.concatenate([[0], np.cumsum(new)])
    qs[B] = n + 1                       # the last request claims a row that x does not have
    lens = [v for v in new[:-1]] + [1]
    x = randn(1, n, 576, dtype=torch.bfloat16)
    pool = torch.zeros(B, PAGE, 640, dtype=torch.uint8, device="cuda")
    sc = torch.full((B,), -1.0, device="cuda")
    table = i32(np.arange(B)[:, None])
    mla.cache_write_fp8_paged(dims, x, None, i32(qs), i32(lens), table, pool, sc)
    torch.cuda.synchronize()
    assert mla.get_device_status() == 7
    assert bool((sc[:n] > 0).all()) and bool((sc[n:] == -1).all())
    assert bool(pool[:n, 0].any(-1).all()) and not pool[n:].any() and not pool[:, 1:].any()


def test_tables_that_are_none_are_refused():
    """Whatever has a rope table's size is not one; neither is an odd truth value."""
    dims = mla.Dims(1, 16, 512, 64, 128, 128, PAGE, "bf16")
    x, pool = randn(1, 1, 576, dtype=torch.bfloat16), torch.zeros(1, PAGE, 576, dtype=torch.bfloat16,
                                                                    device="cuda")
    fake = np.zeros(ctypes.sizeof(type(mla.rope_table(64))), np.uint8)
    with pytest.raises(TypeError, match="rope_table"):
        mla.cache_write_paged(dims, x, None, i32([0]), torch.zeros(1, dtype=torch.int64, device="cuda"),
                              pool, fake)
    with pytest.raises(TypeError, match="rope_table"):
        mla.cache_write_fp8_paged(dims, x, None, i32([0, 1]), i32([1]), i32([[0]]),
                                  torch.zeros(1, PAGE, 640, dtype=torch.uint8, device="cuda"),
                                  torch.ones(1, device="cuda"), fake)
    y = randn(2, 4, 64)
    with pytest.raises((RuntimeError, ValueError)):
        mla.rope(mla.rope_table(64), y, i32([0, 1, 2, 3]), out=y, transpose=torch.ones(2))
    assert mla.get_device_status() == 0


@pytest.mark.parametrize("fp8", [True, False])
def test_paged_cache_step_of_a_stated_size(fp8):
    """A step planned for fewer rows than its tokens is not begun, and nothing is written."""
    dims = mla.Dims(2, 16, 512, 64, 128, 128, 128, "bf16")
    cache = mla.PagedCache(dims, num_pages=4, max_tokens=64, fp8=fp8, table=mla.rope_table(64))
    x = randn(1, 5, 576, dtype=torch.bfloat16)
    cache.plan(i32([3, 2]), tokens=4)
    cache.write(x[:4])
    assert mla.get_device_status() == 7
    assert cache.seqlens.tolist() == [0, 0] and cache.free_count.item() == 4
    assert not cache.pool.any() and bool((cache.block_table == -1).all())
    cache.plan(i32([3, 2]), tokens=5)
    cache.write(x)
    assert mla.get_device_status() == 0 and cache.seqlens.tolist() == [3, 2]
    cache.plan(i32([1, 0]), tokens=1)
    cache.write(x[:1])
    assert mla.get_device_status() == 0 and cache.seqlens.tolist() == [4, 2]
    for b, n in enumerate((4, 2)):
        p = cache.block_table[b, 0].item()
        assert bool(cache.pool[p, :n].view(torch.uint8).any(-1).all()) and not cache.pool[p, n:].any()


@pytest.mark.parametrize("fp8", [True, False])
def test_paged_cache_reports_missing_rows(fp8):
    """A step planned without its size and written with fewer rows than its tokens is
    reported; as many or more rows are not, nor is a captured step's replay."""
    dims = mla.Dims(2, 16, 512, 64, 128, 128, 128, "bf16")
    cache = mla.PagedCache(dims, num_pages=4, max_tokens=16, fp8=fp8, table=mla.rope_table(64))
    x, new = randn(1, 16, 576, dtype=torch.bfloat16), i32([3, 2])
    for rows, want in ((4, 7), (5, 0), (1, 7), (16, 0)):
        cache.plan(new)
        cache.write(x[:rows])
        assert mla.get_device_status() == want, rows
        cache.release(i32([1, 1]))
    cache.plan(new)
    with pytest.raises(ValueError, match="tokens=0"):
        cache.write(x[:0])
    cache.release(i32([1, 1]))
    cache.plan(i32([0, 0]), tokens=0)
    cache.write(x[:0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.plan(new)
        cache.write(x[:6])
    for n, want in (([3, 3], 0), ([3, 4], 7), ([0, 0], 0), ([6, 0], 0)):
        new.copy_(i32(n))
        g.replay()
        assert mla.get_device_status() == want, n
        assert cache.seqlens.tolist() == n
        cache.release(i32([1, 1]))
    assert mla.get_device_status() == 0


def test_decode_step_refuses_an_append_before_it_forks():
    """The refusal of h is what a capture reports, and the step is usable after it."""
    dims, tab = mla.Dims(2, 16, 512, 64, 128, 128, 128, "bf16"), mla.rope_table(64)
    bf = lambda i, *s: randn(i, *s, dtype=torch.bfloat16)  # noqa: E731
    cache = mla.PagedCache(dims, num_pages=4, max_tokens=64, fp8=True, table=tab)
    step = mla.DecodeStep(dims, bf(1, 16, 128, 512), bf(2, 16, 128, 512), bf(3, 576, 256),
                          rope_table=tab)
    cache.plan(i32([3, 2]), tokens=5)
    cache.write(bf(4, 5, 576))
    args = (bf(5, 2, 16, 128), bf(6, 2, 16, 64), cache.last_positions(), cache.pool, cache.seqlens)
    kw = dict(block_table=cache.block_table, page_scales=cache.page_scales)
    want = step(*args, **kw).clone()
    for call in (step, step.capture):
        with pytest.raises(ValueError, match="before the step"):
            call(*args, h=bf(7, 2, 256), **kw)
    step.out.zero_()
    step.capture(*args, **kw).replay()
    assert torch.equal(step.out, want) and mla.get_device_status() == 0


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("capacity,H", [(100, 16), (1, 64), (1000, 128)])
def test_paged_cache_stops_at_a_capacity_inside_a_page(capacity, H, fp8):
    """A capacity that ends inside a page holds: the attention stops there, so the plan does
    too, and a step past it takes nothing."""
    dims = mla.Dims(2, H, 512, 64, 128, 128, capacity, "bf16")
    tab = mla.rope_table(64)
    cache = mla.PagedCache(dims, num_pages=40, max_tokens=2100, fp8=fp8, table=tab)
    x = randn(1, 2100, 576, dtype=torch.bfloat16)
    cache.plan(i32([capacity, capacity - 1]))
    cache.write(x)
    assert mla.get_device_status() == 0 and cache.seqlens.tolist() == [capacity, capacity - 1]
    held = [t.clone() for t in (cache.pool, cache.block_table, cache.free_count)]
    for new in ([1, 0], [0, 2], [1, 1]):
        cache.plan(i32(new), tokens=2)
        cache.write(x[:2])
        assert mla.get_device_status() == 7, new
        assert cache.seqlens.tolist() == [capacity, capacity - 1]
        assert bool((cache.slots[:2] == -1).all()) and not cache.query_start.any()
        for t, k in zip((cache.pool, cache.block_table, cache.free_count), held):
            assert torch.equal(t, k)
    cache.plan(i32([0, 1]), tokens=1)
    cache.write(x[:1])
    assert mla.get_device_status() == 0 and cache.seqlens.tolist() == [capacity, capacity]


def test_plan_pages_capacity_argument():
    pool = Pool([130, 5], 12, 4)
    args = (pool.d_len, i32([1, 60]), pool.d_table, pool.d_free, pool.d_count, pool.num_pages,
            i32([0] * 3), i32([0] * 64), torch.zeros(64, dtype=torch.int64, device="cuda"),
            i32([0] * 2), i32([0]),
            torch.zeros(mla.plan_pages_workspace_bytes(), dtype=torch.uint8, device="cuda"))
    for capacity, want in ((130, 7), (131, 0), (256, 0), (None, 0)):
        mla.plan_pages(*args, capacity=capacity)
        assert mla.get_device_status() == want, capacity
        assert args[9].tolist() == ([130, 5] if want else [131, 65])
    for capacity in (0, -1, 257):
        with pytest.raises(mla.MLAError, match="INVALID"):
            mla.plan_pages(*args, capacity=capacity)
    # The same with a stream of its own: the checks of the wrapper.
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mla.plan_pages(*args, capacity=130, stream=s)
    assert mla.get_device_status(s) == 7 and args[9].tolist() == [130, 5]


def test_errors_name_the_operator():
    """A refusal names the operator, whichever way the call took."""
    pool, dims = Pool([1], 2, 1), mla.Dims(1, 16, 512, 64, 128, 128, PAGE, "bf16")
    n, x = i32([1]), randn(1, 1, 576, dtype=torch.bfloat16)
    slots, mem = torch.zeros(1, dtype=torch.int64, device="cuda"), randn(2, 1, PAGE, 576, dtype=torch.bfloat16)
    for stream in (None, torch.cuda.current_stream()):
        with pytest.raises(mla.MLAError, match="^mla_plan_pages failed"):
            mla.plan_pages(pool.d_len, n, pool.d_table, pool.d_free, pool.d_count, 0, i32([0, 0]), n,
                           slots, pool.d_len, pool.d_count, i32([0] * 64), stream=stream)
        with pytest.raises(mla.MLAError, match="^mla_cache_write_paged failed"):
            mla.cache_write_paged(dims, x, None, n, slots, mem, eps=-1.0, stream=stream)
    assert mla.get_device_status() == 0
