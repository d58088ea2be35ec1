"""What is measured of the paged serving operators: rotary positions, page plans,
cache writes of many tokens, and attention over a paged 8-bit latent cache.

`run` computes each operator either in its plain form (elementary torch
operations in 32 bits, 64 where 32 lose what matters) or, with `own`, by the
library's calls.  Layouts are those of the library: pages of 64 rows, a latent
row of 512 values followed by 64 rotary key values.
"""
import math
import random

import torch

own = False

DEV = "cuda"
PAGE = 64
D_C, D_R = 512, 64
R = D_C + D_R
D_NOPE = D_V = 128
EPS = 1e-6
MIN_EXP = -40          # the smallest exponent of a page's scale


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # The rotary part of the queries of one decode step: a view of
        # [64, 64, 128 + 64] rotated into a buffer of its own; long contexts.
        dict(name="rope_decode_b64", op="rope", tokens=64, heads=64, d_r=64, dtype="bf16",
             layout="interleaved", scaling="yarn", factor=32.0, max_pos=131072, view=True,
             transpose=False),
        # The same of one chunk of a prompt, 128 heads.
        dict(name="rope_prompt_t4096", op="rope", tokens=4096, heads=128, d_r=64, dtype="bf16",
             layout="half", scaling="linear", factor=4.0, max_pos=32768, view=True,
             transpose=False),
        # The transposed rotation (a gradient through it), fp32, odd token count.
        dict(name="rope_grad_f32_t1023", op="rope", tokens=1023, heads=16, d_r=64, dtype="f32",
             layout="half", scaling="ntk", factor=8.0, max_pos=65536, view=False,
             transpose=True),
        # One decode step's plan: 64 ragged sequences, one token each.
        dict(name="plan_decode_b64", op="plan", B=64, ctx=32768, new=1, pad=0),
        # A step that mixes prompt chunks: 256 requests, about 66,000 tokens.
        dict(name="plan_prompts_b256", op="plan", B=256, ctx=4096, new=512, pad=100),
        # The new rows of one decode step into bf16 pages.
        dict(name="write_decode_b32", op="write", B=32, ctx=8192, new=1, dtype="bf16",
             layout="half", fused=False, pad=0),
        # Prompt chunks into bf16 pages; x is a slice of a wider projection.
        dict(name="write_prompt_t8k", op="write", B=16, ctx=1000, new=1024, dtype="bf16",
             layout="interleaved", fused=True, pad=37),
        # The new rows of one decode step into 8-bit pages.
        dict(name="write8_decode_b64", op="write8", B=64, ctx=4096, new=1, layout="half",
             fused=False, pad=0),
        # Prompt chunks into 8-bit pages.
        dict(name="write8_prompt_t8k", op="write8", B=16, ctx=1000, new=1024,
             layout="interleaved", fused=True, pad=37),
        # Attention over 8-bit pages: a small model's decode step,
        dict(name="attend8_h16_n4096", op="attend8", B=4, H=16, N=4096, ragged=False),
        # a large one's,
        dict(name="attend8_h128_n8192", op="attend8", B=32, H=128, N=8192, ragged=False),
        # and ragged sequences up to 32768 tokens.
        dict(name="attend8_h64_ragged", op="attend8", B=64, H=64, N=32768, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "plan", "write", "write8", "attend8"])
    if op == "rope":
        heads = rng.choice([1, 5, 16, 64, 128])
        return dict(op=op, tokens=_log_int(rng, 1, 4096), heads=heads,
                    d_r=rng.choice([32, 64, 64, 96, 128]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    factor=float(rng.choice([2, 4, 8, 32])), max_pos=_log_int(rng, 128, 1000000),
                    view=rng.random() < 0.5, transpose=rng.random() < 0.3)
    if op == "attend8":
        B = _log_int(rng, 1, 64)
        return dict(op=op, B=B, H=rng.choice([1, 8, 16, 40, 64, 100, 128]),
                    N=_log_int(rng, 1, 16384 if B > 8 else 65536), ragged=rng.random() < 0.6)
    B = _log_int(rng, 1, 256 if op == "plan" else 64)
    case = dict(op=op, B=B, ctx=_log_int(rng, 1, 8192),
                new=rng.choice([1, 1, _log_int(rng, 2, max(3, 16384 // B))]),
                pad=rng.choice([0, 0, 13, 64]))
    if op != "plan":
        case.update(layout=rng.choice(["half", "interleaved"]), fused=rng.random() < 0.5)
    if op == "write":
        case.update(dtype=rng.choice(["bf16", "bf16", "f32"]))
    return case


# ------------------------------------------------- sizes that the case fixes
def _spread(n, top, low=1):
    """n whole numbers spread evenly over [low, top]."""
    return [low + (top - low) * (i + 1) // n for i in range(n)]


def _lens(case):
    """(cached tokens, new tokens) of each request, before they are shuffled."""
    B, new = case["B"], case["new"]
    if new == 1:
        n = [1] * B
    else:
        n = _spread(B, new, 0)       # prompt chunks from nothing up to `new`
    return _spread(B, case["ctx"], 0), n


def _tokens(case):
    return sum(_lens(case)[1])


def _kv_lens(case):
    return _spread(case["B"], case["N"]) if case["ragged"] else [case["N"]] * case["B"]


def work(case):
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * case["heads"] * case["d_r"]
        return {"bytes": 2 * n * (2 if case["dtype"] == "bf16" else 4) + 4 * case["tokens"],
                "flops": 3 * n}
    if op == "plan":
        T, B = _tokens(case) + case["pad"], case["B"]
        return {"bytes": 12 * T + 4 * (4 * B + 1) + 8 * (T // PAGE + B), "flops": 0}
    if op == "write":
        T, e = _tokens(case), 2 if case["dtype"] == "bf16" else 4
        return {"bytes": T * (2 * R * e + 12) + 4 * D_C, "flops": T * (4 * D_C + 3 * D_R)}
    if op == "write8":
        T, B = _tokens(case), case["B"]
        return {"bytes": T * (2 * R + D_C + 2 * D_R) + 4 * D_C + 8 * (T // PAGE + B) + 8 * B,
                "flops": T * (5 * D_C + 3 * D_R)}
    L, B, H = sum(_kv_lens(case)), case["B"], case["H"]
    return {"bytes": L * (D_C + 2 * D_R) + 8 * (L // PAGE) + 2 * B * H * (R + D_V) + 4 * B * H
            + 2 * H * D_V * D_C,
            "flops": 2 * L * H * (R + D_C) + 2 * B * H * D_V * D_C}


# ------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _frequencies(case):
    """Angle per position of each pair, float64, and the amplitude of the rotation."""
    d, base, f = case.get("d_r", D_R), 10000.0, case.get("factor", 1.0)
    k = torch.arange(d // 2, dtype=torch.float64)
    kind = case.get("scaling", "none")
    if kind == "ntk":
        base = base * f ** (d / (d - 2.0))
    freq = base ** (-2.0 * k / d)
    if kind == "linear":
        freq = freq / f
    if kind == "yarn":
        at = lambda turns: d * math.log(4096.0 / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), d - 1)
        ramp = ((k - low) / max(high - low, 1e-3)).clamp(0, 1)
        freq = freq / f * ramp + freq * (1 - ramp)
        return freq, 0.1 * math.log(f) + 1.0
    return freq, 1.0


def _table(case):
    import mla_latent_kv_nope_b200 as mla
    return mla.rope_table(case.get("d_r", D_R), base=10000.0, layout=case["layout"],
                          scaling=case.get("scaling", "none"), factor=case.get("factor", 1.0),
                          original_len=4096)


def _randn(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _prepare_rope(case, g):
    T, H, d = case["tokens"], case["heads"], case["d_r"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    x = (_randn(g, T, H, 128 + d, dtype=dt)[..., 128:] if case["view"]
         else _randn(g, T, H, d, dtype=dt))
    freq, amp = _frequencies(case)
    return dict(x=x, pos=torch.randint(0, case["max_pos"], (T,), generator=g, device=DEV,
                                       dtype=torch.int32),
                freq=freq.to(DEV), amp=amp, out=torch.empty(T, H, d, dtype=dt, device=DEV))


def _requests(case, g, seed):
    """Shuffled request lengths and a page table in random page order."""
    ctx, new = _lens(case)
    rng = random.Random(seed)
    rng.shuffle(ctx)
    rng.shuffle(new)
    B, T = case["B"], sum(new) + case["pad"]
    blocks = [(c + PAGE - 1) // PAGE for c in ctx]
    after = [(c + n + PAGE - 1) // PAGE for c, n in zip(ctx, new)]
    # Sizes that do not go by how the two lists were shuffled.
    max_blocks = (max(ctx) + max(new) + PAGE - 1) // PAGE + 1
    num_pages = sum(blocks) + sum((n + PAGE - 1) // PAGE + 1 for n in new)
    order = torch.randperm(num_pages, generator=g, device=DEV, dtype=torch.int32)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return ctx, new, T, blocks, after, max_blocks, num_pages, order, i32


def _fill_table(B, max_blocks, counts, order):
    n = torch.tensor(counts, device=DEV)
    first = torch.cumsum(n, 0) - n
    j = torch.arange(max_blocks, device=DEV)
    ids = order[(first[:, None] + j).clamp(max=order.numel() - 1)]
    return torch.where(j < n[:, None], ids, -1).to(torch.int32).contiguous()


def _prepare_plan(case, g, seed):
    ctx, new, T, blocks, after, max_blocks, num_pages, order, i32 = _requests(case, g, seed)
    B, used = case["B"], sum(blocks)
    e = lambda n, dt=torch.int32: torch.empty(n, dtype=dt, device=DEV)  # noqa: E731
    return dict(seqlens=i32(ctx), new_lens=i32(new),
                block_table=_fill_table(B, max_blocks, blocks, order),
                free_pages=order[used:].contiguous(), free_count=i32([num_pages - used]),
                num_pages=num_pages, T=T, query_start=e(B + 1), positions=e(T),
                slots=e(T, torch.int64), seqlens_out=e(B), free_count_out=e(1),
                workspace=torch.zeros(64, dtype=torch.int32, device=DEV))


def _prepare_write(case, g, seed):
    eight = case["op"] == "write8"
    ctx, new, T, blocks, after, max_blocks, num_pages, order, i32 = _requests(case, g, seed)
    dt = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16
    B, n_new = case["B"], sum(new)
    x = (_randn(g, T, R + 1536, dtype=dt)[:, 1536:] if case["fused"] else _randn(g, T, R, dtype=dt))
    gamma = 1.0 + 0.1 * torch.randn(D_C, generator=g, device=DEV)
    freq, amp = _frequencies(case)
    qs = i32([0] + new).cumsum(0).to(torch.int32)
    s = dict(x=x, gamma=gamma, freq=freq.to(DEV), amp=amp, query_start=qs,
             seqlens=i32([c + n for c, n in zip(ctx, new)]),
             block_table=_fill_table(B, max_blocks, after, order))
    if eight:
        codes = _randn(g, num_pages, PAGE, D_C, dtype=torch.float32).mul_(100).clamp_(-448, 448)
        s["pool"] = torch.empty(num_pages, PAGE, D_C + 2 * D_R, dtype=torch.uint8, device=DEV)
        s["pool"][..., :D_C].view(torch.float8_e4m3fn).copy_(codes.to(torch.float8_e4m3fn))
        s["scales"] = torch.exp2(torch.randint(-9, -6, (num_pages,), generator=g, device=DEV).float())
        s["pool"][..., D_C:].view(torch.bfloat16).copy_(
            _randn(g, num_pages, PAGE, D_R, dtype=torch.float32) / s["scales"][:, None, None])
        return s
    s["pool"] = _randn(g, num_pages, PAGE, R, dtype=dt)
    # The page plan's outputs: position and slot of each token, -1 for padding.
    t = torch.arange(T, device=DEV)
    r = (torch.searchsorted(qs.long(), t, right=True) - 1).clamp(max=B - 1)
    pos = i32(ctx)[r] + t - qs[r]
    page = s["block_table"][r, (pos // PAGE).clamp(max=max_blocks - 1)]
    live = t < n_new
    s["positions"] = torch.where(live, pos, -1).to(torch.int32)
    s["slots"] = torch.where(live, page.long() * PAGE + pos % PAGE, -1)
    return s


def _prepare_attend8(case, g, seed):
    B, H, L = case["B"], case["H"], _kv_lens(case)
    random.Random(seed).shuffle(L)
    blocks = [(n + PAGE - 1) // PAGE for n in L]
    num_pages, max_blocks = sum(blocks) + 3, max(blocks)
    order = torch.randperm(num_pages, generator=g, device=DEV, dtype=torch.int32)
    # RMS-normalised latents: values near N(0, 1), codes near 2^6 N(0, 1).
    pool = torch.empty(num_pages, PAGE, D_C + 2 * D_R, dtype=torch.uint8, device=DEV)
    scales = torch.exp2(torch.randint(-7, -5, (num_pages,), generator=g, device=DEV).float())
    for a in range(0, num_pages, 1024):      # in parts: the fp32 values are not kept
        p = pool[a:a + 1024]
        inv = (1 / scales[a:a + 1024])[:, None, None]
        c = torch.randn(p.shape[0], PAGE, D_C, generator=g, device=DEV).mul_(inv).clamp_(-448, 448)
        p[..., :D_C].view(torch.float8_e4m3fn).copy_(c.to(torch.float8_e4m3fn))
        k = torch.randn(p.shape[0], PAGE, D_R, generator=g, device=DEV)
        p[..., D_C:].view(torch.bfloat16).copy_(k * inv)
    s = dict(pool=pool, scales=scales, block_table=_fill_table(B, max_blocks, blocks, order),
             seqlens=torch.tensor(L, dtype=torch.int32, device=DEV),
             q_cat=_randn(g, B, H, R, dtype=torch.bfloat16),
             W_UV=(0.02 * torch.randn(H, D_V, D_C, generator=g, device=DEV)).to(torch.bfloat16),
             scale=1 / math.sqrt(D_NOPE + D_R))
    if own:
        import mla_latent_kv_nope_b200 as mla
        d = s["dims"] = mla.Dims(B, H, D_C, D_R, D_NOPE, D_V, max_blocks * PAGE, "bf16")
        s["ws"] = torch.empty(mla.decode_workspace_bytes(d) // 4, device=DEV)
        s["o_lat"] = torch.empty(B, H, D_C, device=DEV)
        s["lse"] = torch.empty(B, H, device=DEV)
        s["out"] = torch.empty(B, H, D_V, dtype=torch.bfloat16, device=DEV)
    return s


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op == "rope":
        s = _prepare_rope(case, g)
    elif op == "plan":
        s = _prepare_plan(case, g, seed)
    elif op == "attend8":
        s = _prepare_attend8(case, g, seed)
    else:
        s = _prepare_write(case, g, seed)
    if own and op in ("rope", "write", "write8"):
        s["table"] = _table(case)
    if own and op in ("write", "write8"):
        import mla_latent_kv_nope_b200 as mla
        s["dims"] = mla.Dims(case["B"], 1, D_C, D_R, D_NOPE, D_V,
                             s["block_table"].shape[1] * PAGE, case.get("dtype", "bf16"))
    s["case"] = case
    return s


# ---------------------------------------------------------------- plain forms
def _rotate(x, pos, freq, amp, layout, transpose):
    """x [..., tokens on the first axis, d_r] rotated; fp32, angles in fp64."""
    th = pos.double()[:, None] * freq
    c, sn = (amp * th.cos()).float(), (amp * th.sin()).float()
    if transpose:
        sn = -sn
    if x.dim() == 3:
        c, sn = c[:, None], sn[:, None]
    if layout == "half":
        a, b = x.float().chunk(2, -1)
        return torch.cat([a * c - b * sn, a * sn + b * c], -1)
    a, b = x.float()[..., 0::2], x.float()[..., 1::2]
    return torch.stack([a * c - b * sn, a * sn + b * c], -1).flatten(-2)


def _plain_rope(s):
    c = s["case"]
    return _rotate(s["x"], s["pos"], s["freq"], s["amp"], c["layout"], c["transpose"]).to(s["x"].dtype)


def _plain_plan(s):
    L, n, T = s["seqlens"].long(), s["new_lens"].long(), s["T"]
    old, end = (L + PAGE - 1) // PAGE, (L + n + PAGE - 1) // PAGE
    need = end - old
    qs = torch.cat([L.new_zeros(1), n.cumsum(0)])
    first = need.cumsum(0) - need
    free = s["free_count"].long()
    j = torch.arange(s["block_table"].shape[1], device=DEV)
    p = free - 1 - (first[:, None] + j - old[:, None])
    fresh = s["free_pages"][p.clamp(0, s["free_pages"].numel() - 1)]
    table = torch.where((j >= old[:, None]) & (j < end[:, None]), fresh, s["block_table"])
    t = torch.arange(T, device=DEV)
    r = (torch.searchsorted(qs, t, right=True) - 1).clamp(max=L.numel() - 1)
    pos = L[r] + t - qs[r]
    live = t < qs[-1]
    page = table[r, (pos // PAGE).clamp(max=table.shape[1] - 1)].long()
    return dict(query_start=qs.int(), positions=torch.where(live, pos, -1).int(),
                slots=torch.where(live, page * PAGE + pos % PAGE, -1),
                seqlens=(L + n).int(), free_count=(free - need.sum()).int(), block_table=table)


def _normed(s, x, pos):
    c, k = x[:, :D_C].float(), x[:, D_C:]
    c = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS) * s["gamma"]
    return c, _rotate(k, pos, s["freq"], s["amp"], s["case"]["layout"], False)


def _plain_write(s):
    c, k = _normed(s, s["x"], s["positions"].clamp(min=0))
    live = s["slots"] >= 0
    flat = s["pool"].view(-1, R)
    flat[s["slots"][live]] = torch.cat([c, k], -1)[live].to(flat.dtype)
    return s["pool"]


def _token_pages(s):
    """Page, row and position of each new token (no padding), and its request."""
    qs, L = s["query_start"].long(), s["seqlens"].long()
    T = s["x"].shape[0] - s["case"]["pad"]
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(qs, t, right=True) - 1
    start = L - (qs[1:] - qs[:-1])
    pos = start[r] + t - qs[r]
    return s["block_table"][r, pos // PAGE].long(), pos % PAGE, pos, start, qs


def _exponent(amax):
    """Smallest k with amax <= 448 * 2^k, at least MIN_EXP."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, torch.where(m <= 0.875, e - 9, e - 8), MIN_EXP).clamp(min=MIN_EXP)


def _plain_write8(s):
    page, row, pos, start, qs = _token_pages(s)
    c, k = _normed(s, s["x"][:page.numel()], pos)
    pool, scales = s["pool"], s["scales"]
    P = pool.shape[0]
    amax = torch.full((P,), -1.0, device=DEV).scatter_reduce(0, page, c.abs().amax(-1), "amax")
    # Rows that a page held before: of the page that a request's first new token falls into.
    has = qs[1:] > qs[:-1]
    fp = s["block_table"].gather(1, (start // PAGE).clamp(max=s["block_table"].shape[1] - 1)[:, None])[:, 0]
    kept = torch.zeros(P, dtype=torch.long, device=DEV).index_add(
        0, fp.long().clamp(min=0), torch.where(has, start % PAGE, 0))
    ke_old = torch.frexp(scales)[1] - 1
    ke = torch.maximum(_exponent(amax), torch.where(kept > 0, ke_old, MIN_EXP))
    ke = torch.where(amax >= 0, ke, ke_old)
    shrink = torch.exp2((ke_old - ke).float())[:, None]
    shrink = torch.where(torch.arange(PAGE, device=DEV) < kept[:, None], shrink, 1.0)[..., None]
    codes = pool[..., :D_C].view(torch.float8_e4m3fn).float() * shrink
    rope = pool[..., D_C:].view(torch.bfloat16).float() * shrink
    inv = torch.exp2(-ke.float())[page][:, None]
    codes[page, row] = c * inv
    rope[page, row] = k.to(torch.bfloat16).float() * inv
    pool[..., :D_C].view(torch.float8_e4m3fn).copy_(codes.to(torch.float8_e4m3fn))
    pool[..., D_C:].view(torch.bfloat16).copy_(rope.to(torch.bfloat16))
    scales.copy_(torch.exp2(ke.float()))
    return _pages8(s)


def _pages8(s):
    return dict(codes=s["pool"][..., :D_C].view(torch.float8_e4m3fn),
                rope=s["pool"][..., D_C:].view(torch.bfloat16), scales=s["scales"])


def _plain_attend8(s):
    tab = s["block_table"].clamp(min=0).long()
    B, n = tab.shape[0], tab.shape[1] * PAGE
    rows = s["pool"][tab]
    sc = s["scales"][tab][:, :, None, None]
    c = (rows[..., :D_C].view(torch.float8_e4m3fn).float() * sc).view(B, n, D_C)
    k = (rows[..., D_C:].view(torch.bfloat16).float() * sc).view(B, n, D_R)
    q = s["q_cat"].float()
    x = (q[..., :D_C] @ c.transpose(1, 2) + q[..., D_C:] @ k.transpose(1, 2)) * s["scale"]
    x = x.masked_fill(torch.arange(n, device=DEV) >= s["seqlens"][:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = (x - m).exp()
    l = p.sum(-1, keepdim=True)
    o = (p @ c) / l
    out = (o[:, :, None] * s["W_UV"].float()).sum(-1) if B * s["q_cat"].shape[1] <= 64 else \
        (o.transpose(0, 1) @ s["W_UV"].float().transpose(1, 2)).transpose(0, 1)
    return out.to(torch.bfloat16), (m + l.log())[..., 0]


# ----------------------------------------------------------- the library's calls
def _own_rope(s):
    import mla_latent_kv_nope_b200 as mla
    mla.rope(s["table"], s["x"], s["pos"], s["out"], transpose=s["case"]["transpose"])
    return s["out"]


def _own_plan(s):
    import mla_latent_kv_nope_b200 as mla
    mla.plan_pages(s["seqlens"], s["new_lens"], s["block_table"], s["free_pages"], s["free_count"],
                   s["num_pages"], s["query_start"], s["positions"], s["slots"],
                   s["seqlens_out"], s["free_count_out"], s["workspace"])
    return dict(query_start=s["query_start"], positions=s["positions"], slots=s["slots"],
                seqlens=s["seqlens_out"], free_count=s["free_count_out"],
                block_table=s["block_table"])


def _own_write(s):
    import mla_latent_kv_nope_b200 as mla
    mla.cache_write_paged(s["dims"], s["x"], s["gamma"], s["positions"], s["slots"], s["pool"],
                          s["table"], eps=EPS)
    return s["pool"]


def _own_write8(s):
    import mla_latent_kv_nope_b200 as mla
    mla.cache_write_fp8_paged(s["dims"], s["x"], s["gamma"], s["query_start"], s["seqlens"],
                              s["block_table"], s["pool"], s["scales"], s["table"], eps=EPS)
    return _pages8(s)


def _own_attend8(s):
    import mla_latent_kv_nope_b200 as mla
    d = s["dims"]
    used = mla.decode_fp8_paged(d, s["q_cat"], s["pool"], s["scales"], s["block_table"],
                                s["seqlens"], s["scale"], s["ws"])
    mla.combine(d, s["seqlens"], s["ws"], used, s["o_lat"], s["lse"])
    mla.out_proj(d, s["o_lat"], s["W_UV"], s["out"])
    return s["out"], s["lse"]


_PLAIN = dict(rope=_plain_rope, plan=_plain_plan, write=_plain_write, write8=_plain_write8,
              attend8=_plain_attend8)
_OWN = dict(rope=_own_rope, plan=_own_plan, write=_own_write, write8=_own_write8,
            attend8=_own_attend8)


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------- the definitions in 64 bits
def _turned(x, pos, freq, amp, layout, transpose=False):
    """The pairs of x as complex numbers times amp * e^(+-i pos freq)."""
    x = x.double()
    d = x.shape[-1]
    z = torch.complex(x[..., :d // 2], x[..., d // 2:]) if layout == "half" else \
        torch.view_as_complex(x.reshape(*x.shape[:-1], d // 2, 2).contiguous())
    th = pos.double().reshape(-1, *[1] * (x.dim() - 1)) * freq * (-1 if transpose else 1)
    z = z * torch.polar(torch.full_like(th, amp), th)
    return torch.cat([z.real, z.imag], -1) if layout == "half" else torch.view_as_real(z).flatten(-2)


def _exact_plan(s):
    L, n = s["seqlens"].tolist(), s["new_lens"].tolist()
    free, left = s["free_pages"].tolist(), int(s["free_count"])
    table = s["block_table"].cpu().clone()
    qs, positions, slots = [0], [], []
    for b, (a, m) in enumerate(zip(L, n)):
        for j in range(-(-a // PAGE), -(-(a + m) // PAGE)):
            left -= 1
            table[b, j] = free[left]
        row = table[b].tolist()
        positions += range(a, a + m)
        slots += [row[p // PAGE] * PAGE + p % PAGE for p in range(a, a + m)]
        qs.append(qs[-1] + m)
    pad = [-1] * (s["T"] - len(slots))
    t = lambda v, dt=torch.int32: torch.tensor(v, dtype=dt)  # noqa: E731
    return dict(query_start=t(qs), positions=t(positions + pad), slots=t(slots + pad, torch.int64),
                seqlens=t([a + m for a, m in zip(L, n)]), free_count=t([left]), block_table=table)


def _exact_row(s, x, pos):
    x = x.double()
    c = x[:, :D_C] / ((x[:, :D_C] ** 2).sum(-1, keepdim=True) / D_C + EPS).sqrt() * s["gamma"].double()
    return c, _turned(x[:, D_C:], pos, s["freq"], s["amp"], s["case"]["layout"])


def _exact_write8(s):
    """Each request's pages one after the other; codes are the values before rounding."""
    qs, L, table = (s[k].tolist() for k in ("query_start", "seqlens", "block_table"))
    P = s["pool"].shape[0]
    codes = s["pool"][..., :D_C].view(torch.float8_e4m3fn).double()
    rope = s["pool"][..., D_C:].view(torch.bfloat16).double()
    scales = s["scales"].double()
    held = scales.tolist()
    for b, end in enumerate(L):
        a = end - (qs[b + 1] - qs[b])
        if a == end:
            continue
        pos = torch.arange(a, end, device=DEV)
        c, k = _exact_row(s, s["x"][qs[b]:qs[b + 1]], pos)
        top = c.abs().amax(-1).tolist()
        for j in range(a // PAGE, (end - 1) // PAGE + 1):
            p, lo, hi = table[b][j], max(a, j * PAGE), min(end, (j + 1) * PAGE)
            e = max(MIN_EXP, math.ceil(math.log2(max(max(top[lo - a:hi - a]), 1e-30) / 448)))
            if lo % PAGE:
                e0 = round(math.log2(held[p]))
                e = max(e, e0)
                codes[p, :lo % PAGE] *= 2.0 ** (e0 - e)
                rope[p, :lo % PAGE] *= 2.0 ** (e0 - e)
            r = slice(lo % PAGE, lo % PAGE + hi - lo)
            codes[p, r] = c[lo - a:hi - a] / 2.0 ** e
            rope[p, r] = k[lo - a:hi - a] / 2.0 ** e
            scales[p] = 2.0 ** e
    assert P == scales.numel()
    return dict(codes=codes, rope=rope, scales=scales)


def _exact_attend8(s):
    B, H = s["q_cat"].shape[:2]
    out = torch.empty(B, H, D_V, dtype=torch.float64, device=DEV)
    lse = torch.empty(B, H, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["seqlens"].tolist()):
        ids = s["block_table"][b, :-(-n // PAGE)].long()
        sc = s["scales"][ids].double()[:, None, None]
        c = (s["pool"][ids][..., :D_C].view(torch.float8_e4m3fn).double() * sc).reshape(-1, D_C)[:n]
        k = (s["pool"][ids][..., D_C:].view(torch.bfloat16).double() * sc).reshape(-1, D_R)[:n]
        z = s["q_cat"][b].double() @ torch.cat([c, k], 1).T * s["scale"]
        lse[b] = z.logsumexp(-1)
        v = torch.softmax(z, -1) @ c
        out[b] = torch.einsum("hc,hvc->hv", v, s["W_UV"].double())
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _turned(s["x"], s["pos"], s["freq"], s["amp"], case["layout"], case["transpose"])
    if op == "plan":
        return _exact_plan(s)
    if op == "write":
        c, k = _exact_row(s, s["x"], s["positions"].clamp(min=0))
        pool = s["pool"].double().reshape(-1, R)
        for a, t in enumerate(s["slots"].tolist()):
            if t >= 0:
                pool[t, :D_C], pool[t, D_C:] = c[a], k[a]
        return pool.reshape(s["pool"].shape)
    if op == "write8":
        return _exact_write8(s)
    return _exact_attend8(s)
