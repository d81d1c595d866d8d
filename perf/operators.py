"""Operators of the 4-bit paged latent cache, in their plain form and as the library's calls.

The set is what a serving step over a 4-bit latent cache needs around the attention that
reads it:

  rope_table   RoPE rows built on the GPU, plain or scaled for long contexts
  rope_apply   rotation of part of each head's vector by given positions, and its gradient
  page_plan    block tables and slot maps from request lengths and a list of free pages
  q4_store     latents rounded to 4 bits into paged rows, and read back from them
  q4_decode    latent-store decode attention over the 4-bit paged cache

``run`` computes the plain form with elementary torch operations in 32 bits (angles in 64)
while ``own`` is false, and calls the library while it is true.

A 4-bit row holds one token of one head: r_k/2 bytes of K codes, r_v/2 bytes of V codes,
one bf16 scale per 32 columns of K, then of V, padded to a multiple of 16 bytes.  Eight
columns make a 32-bit word: column c sits in bits 4(c/2) (c even) or 16 + 4(c/2) (c odd),
as code + 8 with code in [-7, 7]; the value is code * scale.
"""
import math

import torch

own = False

D = 128            # head width
GROUP = 32         # columns that share a scale
BETA_FAST, BETA_SLOW = 32.0, 1.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # RoPE rows of a long-context model (by-parts scaling) and of the 64-wide rotary branch
        {"name": "table_by_parts_131072", "op": "rope_table", "d": 128, "n_pos": 131072, "pos0": 0,
         "scaling": "by_parts", "factor": 8.0, "original": 16384, "base": 10000.0},
        {"name": "table_linear_5000", "op": "rope_table", "d": 64, "n_pos": 5000, "pos0": 0,
         "scaling": "linear", "factor": 4.0, "original": 4096, "base": 10000.0},
        # a decode step's queries
        {"name": "apply_step_64", "op": "rope_apply", "n": 64, "heads": 16, "d_x": 128, "offset": 0, "d_rope": 128,
         "style": 0, "dtype": "bf16", "inverse": False, "scale": 1.0, "rope_len": 16384},
        # the gradient of a prefill's [content ; rotary] vectors: the last 64 of 192, interleaved pairs
        {"name": "apply_grad_32768", "op": "rope_apply", "n": 32768, "heads": 16, "d_x": 192, "offset": 128,
         "d_rope": 64, "style": 1, "dtype": "bf16", "inverse": True, "scale": 1.0, "rope_len": 32768},
        # every sequence of a serving batch gets its next token
        {"name": "plan_step_768", "op": "page_plan", "B": 768, "page": 16, "ctx_hi": 4095, "new_hi": 1,
         "max_pages": 256, "short": False},
        # prompts of a prefill, ragged; the free list runs out before the last ones
        {"name": "plan_prefill_64", "op": "page_plan", "B": 64, "page": 64, "ctx_hi": 0, "new_hi": 16384,
         "max_pages": 256, "short": True},
        # one new token of every sequence at the extreme compression
        {"name": "store_step_768", "op": "q4_store", "n": 768, "H": 16, "r_k": 16, "r_v": 32, "page": 64,
         "dtype": "bf16"},
        # a prefill's tokens at the mild compression
        {"name": "store_prefill_65536", "op": "q4_store", "n": 65536, "H": 16, "r_k": 96, "r_v": 160, "page": 64,
         "dtype": "bf16"},
        # fp32 storage, few short sequences, odd sizes
        {"name": "decode_f32_3x333", "op": "q4_decode", "B": 3, "H": 2, "len_lo": 1, "len_hi": 333, "r_k": 96,
         "r_v": 160, "page": 24, "T": 4, "t": 2, "style": 0, "dtype": "f32"},
        # one layer of a 1.4B looped decoder at 4x compression, ragged lengths
        {"name": "decode_32x4096", "op": "q4_decode", "B": 32, "H": 16, "len_lo": 3584, "len_hi": 4096, "r_k": 96,
         "r_v": 160, "page": 64, "T": 4, "t": 1, "style": 0, "dtype": "bf16"},
        # the same layer at 21.3x compression and a serving batch
        {"name": "decode_128x4096_small", "op": "q4_decode", "B": 128, "H": 16, "len_lo": 2048, "len_hi": 4096,
         "r_k": 16, "r_v": 32, "page": 64, "T": 4, "t": 3, "style": 0, "dtype": "bf16"},
        # two long sequences: the work has to be split along them
        {"name": "decode_2x65001", "op": "q4_decode", "B": 2, "H": 16, "len_lo": 65001, "len_hi": 65001, "r_k": 96,
         "r_v": 160, "page": 128, "T": 4, "t": 0, "style": 1, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_table", "rope_apply", "page_plan", "q4_store", "q4_decode", "q4_decode"])
    if op == "rope_table":
        return {"op": op, "d": 2 * rng.randint(8, 64), "n_pos": _log(rng, 100, 131072),
                "pos0": rng.choice([0, rng.randint(0, 1 << 20)]),
                "scaling": rng.choice(["plain", "linear", "base", "by_parts"]), "factor": rng.uniform(1.0, 32.0),
                "original": rng.choice([2048, 4096, 8192, 16384]), "base": rng.choice([10000.0, 500000.0])}
    if op == "rope_apply":
        d_x = rng.choice([64, 96, 128, 192, 100])
        d_rope = rng.choice([d_x, 2 * rng.randint(1, d_x // 2)])
        return {"op": op, "n": _log(rng, 1, 32768), "heads": rng.randint(1, 16), "d_x": d_x,
                "offset": rng.choice([0, d_x - d_rope]), "d_rope": d_rope, "style": rng.randint(0, 1),
                "dtype": rng.choice(["bf16", "f32"]), "inverse": rng.random() < 0.5,
                "scale": rng.choice([1.0, 1.2079]), "rope_len": _log(rng, 256, 65536)}
    if op == "page_plan":
        page = rng.choice([1, 16, 24, 64, 128])
        B = _log(rng, 1, 1500)
        new_hi = rng.choice([1, 7, 500])
        ctx_hi = _log(rng, 1, 8000)
        return {"op": op, "B": B, "page": page, "ctx_hi": ctx_hi, "new_hi": new_hi,
                "max_pages": (ctx_hi + new_hi) // page + 1, "short": rng.random() < 0.4}
    if op == "q4_store":
        return {"op": op, "n": _log(rng, 1, 30000), "H": rng.randint(1, 16), "r_k": 16 * rng.randint(1, 16),
                "r_v": 16 * rng.randint(1, 16), "page": rng.choice([1, 16, 24, 64, 128]),
                "dtype": rng.choice(["bf16", "f32"])}
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    hi = _log(rng, 1, 2000 if dtype == "f32" else 20000)
    H = rng.randint(1, 16)
    most = (40000 if dtype == "f32" else 1500000) // (hi * H)
    return {"op": "q4_decode", "B": _log(rng, 1, max(1, min(64, most))), "H": H, "len_lo": rng.randint(0, hi),
            "len_hi": hi, "r_k": 16 * rng.randint(1, 12), "r_v": 16 * rng.randint(1, 12),
            "page": rng.choice([1, 8, 16, 24, 64, 100, 128, 256]), "T": 4, "t": rng.randint(0, 3),
            "style": rng.randint(0, 1), "dtype": dtype}


# ------------------------------------------------------------------ inputs

def _token_slots(case):
    """Token entries of a plan's maps: the step's budget, not the sum of this step's lengths."""
    return case["B"] * case["new_hi"] * (3 if case["short"] else 4) // 4 + 3


def _groups(r):
    return (r + GROUP - 1) // GROUP


def _row_bytes(r_k, r_v):
    return (r_k // 2 + r_v // 2 + 2 * (_groups(r_k) + _groups(r_v)) + 15) // 16 * 16


def _storage(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _thetas(case):
    """The fp64 frequencies of a table case."""
    d, base, f, o = case["d"], case["base"], case["factor"], case["original"]
    i = torch.arange(d // 2, dtype=torch.float64)
    if case["scaling"] == "base":
        base = base * f ** (d / (d - 2))
    theta = base ** (-2.0 * i / d)
    if case["scaling"] == "linear":
        theta = theta / f
    if case["scaling"] == "by_parts":
        g = ((o * theta / (2 * math.pi) - BETA_SLOW) / (BETA_FAST - BETA_SLOW)).clamp(0, 1)
        theta = (1 - g) * theta / f + g * theta
    return theta


def _dims(case):
    from looped_transformer_cross_gb300 import lla
    return lla.dims(case.get("T", 1), case.get("H", 1), case["r_k"], case["r_v"],
                    dtype=lla.LLA_BF16 if case["dtype"] == "bf16" else lla.LLA_F32, rope_style=case.get("style", 0))


def _shifts(r, device):
    """The bit of its word at which the code of column c < r begins."""
    c = torch.arange(r, device=device)
    return 4 * ((c % 8) // 2) + 16 * (c % 2)


def _pack(codes, scales):
    """The bytes of `codes` [..., r] and of their bf16 scales [..., groups]."""
    r = codes.shape[-1]
    w = ((codes + 8).to(torch.int64) << _shifts(r, codes.device)).reshape(*codes.shape[:-1], r // 8, 8).sum(-1)
    w = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)
    return w.contiguous().view(torch.uint8), scales.to(torch.bfloat16).contiguous().view(torch.uint8)


def _random_rows(shape, r_k, r_v, gen, device):
    """4-bit rows of N(0, 1) latents, for a pool that a program has filled before."""
    parts, scales = [], []
    for r in (r_k, r_v):
        x = torch.randn(*shape, r, generator=gen, device=device, dtype=torch.float32)
        s = torch.nn.functional.pad(x.abs(), (0, _groups(r) * GROUP - r)).reshape(*shape, _groups(r), GROUP).amax(-1)
        s = (s / torch.full_like(s, 7.0)).to(torch.bfloat16)
        q = torch.round(x / s.float().repeat_interleave(GROUP, -1)[..., :r]).clamp_(-7, 7)
        words, sb = _pack(q, s)
        del x, q
        parts.append(words)
        scales.append(sb)
    rows = torch.cat(parts + scales, -1)
    pad = _row_bytes(r_k, r_v) - rows.shape[-1]
    return torch.nn.functional.pad(rows, (0, pad)).contiguous()


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(1000003 * (seed + 1) + 17)
    host = torch.Generator().manual_seed(7919 * (seed + 1) + 3)
    state = {"case": case}
    if own:
        from looped_transformer_cross_gb300 import lla
        state["lla"] = lla
    op = case["op"]
    if op == "rope_table":
        # a table's only inputs are its parameters: another seed moves its first position
        state["pos0"] = case["pos0"] + seed % 1024
        state["theta"] = _thetas(case).to(dev)
        if own:
            state["dm"] = lla.dims(1, 1, 16, 16, d_head=case["d"], rope_base=case["base"])
            state["scaling"] = lla.rope_scaling(case["scaling"], case["factor"], case["original"], BETA_FAST, BETA_SLOW)
            state["cos"] = torch.empty((case["n_pos"], case["d"] // 2), dtype=torch.float32, device=dev)
            state["sin"] = torch.empty_like(state["cos"])
    elif op == "rope_apply":
        n, half = case["n"], case["d_rope"] // 2
        state["x"] = torch.randn(n, case["heads"], case["d_x"], generator=gen, device=dev).to(_storage(case))
        state["pos"] = torch.randint(0, case["rope_len"], (n,), generator=gen, device=dev, dtype=torch.int32)
        theta = 10000.0 ** (-2.0 * torch.arange(half, dtype=torch.float64, device=dev) / case["d_rope"])
        ang = torch.arange(case["rope_len"], dtype=torch.float64, device=dev)[:, None] * theta
        state["cos"], state["sin"] = ang.cos().float(), ang.sin().float()
        if own:
            state["dm"] = lla.dims(1, case["heads"], 16, 16, dtype=lla.LLA_BF16 if case["dtype"] == "bf16" else lla.LLA_F32,
                                   rope_style=case["style"])
            state["out"] = torch.empty_like(state["x"])
            state["ws"] = torch.zeros(256, dtype=torch.uint8, device=dev)
    elif op == "page_plan":
        B, P, mp = case["B"], case["page"], case["max_pages"]
        ctx = torch.randint(0, case["ctx_hi"] + 1, (B,), generator=host)
        new = torch.randint(1 if case["new_hi"] == 1 else 0, case["new_hi"] + 1, (B,), generator=host)
        held = (ctx + P - 1) // P
        need = int(((ctx + new + P - 1) // P - held).sum())
        n_free = max(1, need * 3 // 4 if case["short"] else need + 5)
        num = int(held.sum()) + n_free
        perm = torch.randperm(num, generator=host).to(torch.int32)
        table = torch.full((B, mp), -1, dtype=torch.int32)
        used = torch.arange(mp)[None, :] < held[:, None]
        table[used] = perm[: int(held.sum())]
        state.update(P=P, num_pages=num, n_tok=_token_slots(case), ctx=ctx.to(torch.int32).to(dev),
                     new=new.to(torch.int32).to(dev), free=perm[int(held.sum()):].contiguous().to(dev), table=table.to(dev))
        if own:
            state["plan"] = lla.PagePlan(B, state["n_tok"], device=dev)
    elif op == "q4_store":
        n, H, sd = case["n"], case["H"], _storage(case)
        state["k"] = torch.randn(n, H, case["r_k"], generator=gen, device=dev).to(sd)
        state["v"] = torch.randn(n, H, case["r_v"], generator=gen, device=dev).to(sd)
        P = case["page"]
        pages = n // P + 2
        state["slots"] = torch.randperm(pages * P, generator=gen, device=dev)[:n].contiguous()
        if own:
            state["dm"] = _dims(case)
            state["pool"] = torch.zeros((pages, H, P, _row_bytes(case["r_k"], case["r_v"])), dtype=torch.uint8, device=dev)
            state["ws"] = torch.zeros(256, dtype=torch.uint8, device=dev)
            state["out_k"], state["out_v"] = torch.empty_like(state["k"]), torch.empty_like(state["v"])
    else:
        B, H, T, rk, rv, P = (case[x] for x in ("B", "H", "T", "r_k", "r_v", "page"))
        sd = _storage(case)
        lens = torch.randint(case["len_lo"], case["len_hi"] + 1, (B,), generator=host)
        mp = (case["len_hi"] + P - 1) // P
        held = (lens + P - 1) // P
        num = int(held.sum()) + 1
        state["pool"] = _random_rows((num, H, P), rk, rv, gen, dev)
        table = torch.full((B, mp), -1, dtype=torch.int32)
        table[torch.arange(mp)[None, :] < held[:, None]] = torch.randperm(num, generator=host)[: int(held.sum())].to(torch.int32)
        state["table"] = table.to(dev)
        state["lens"] = lens.to(torch.int32).to(dev)
        state["q_pos"] = (lens - 1).clamp(min=0).to(torch.int32).to(dev)
        rnd = lambda std, *s: torch.randn(*s, generator=gen, device=dev) * std  # noqa: E731
        state["q"] = rnd(1.0, B, H, D).to(sd)
        state["wk"] = rnd(rk ** -0.5, T, H, D, rk).to(sd)
        state["wv"] = rnd(rv ** -0.5, T, H, D, rv).to(sd)
        state["mk"], state["mv"] = rnd(0.1 ** 0.5, H, T * D), rnd(0.1 ** 0.5, H, T * D)
        n_pos = max(128, mp * P)
        theta = 10000.0 ** (-2.0 * torch.arange(D // 2, dtype=torch.float64, device=dev) / D)
        ang = torch.arange(n_pos, dtype=torch.float64, device=dev)[:, None] * theta
        state["cos"], state["sin"] = ang.cos().float(), ang.sin().float()
        if own:
            state["dm"] = _dims(case)
            state["out"] = torch.empty((B, H, D), dtype=sd, device=dev)
            state["ws"] = lla.q4_workspace(state["dm"], B, mp * P, device=dev)
    return state


# ------------------------------------------------------------------ plain forms

def _plain_rope_table(st):
    n = st["case"]["n_pos"]
    p = torch.arange(n, dtype=torch.float64, device=st["theta"].device) + st["pos0"]
    ang = p[:, None] * st["theta"]
    return ang.cos().float(), ang.sin().float()


def _pairs(x, style):
    """The first and second members of the rotation pairs of [..., d]."""
    h = x.shape[-1] // 2
    return (x[..., :h], x[..., h:]) if style == 0 else (x[..., 0::2], x[..., 1::2])


def _join(a, b, style):
    return torch.cat((a, b), -1) if style == 0 else torch.stack((a, b), -1).flatten(-2)


def _plain_rope_apply(st):
    c = st["case"]
    cos = st["cos"][st["pos"].long()][:, None, :]
    sin = st["sin"][st["pos"].long()][:, None, :]
    if c["inverse"]:
        sin = -sin
    o, d = c["offset"], c["d_rope"]
    x = st["x"].float()
    a, b = _pairs(x[..., o:o + d], c["style"])
    y = _join((a * cos - b * sin) * c["scale"], (a * sin + b * cos) * c["scale"], c["style"])
    return torch.cat((x[..., :o], y, x[..., o + d:]), -1).to(st["x"].dtype)


def _plain_page_plan(st):
    P, mp, n_tok = st["P"], st["table"].shape[1], st["n_tok"]
    ctx, new, table = st["ctx"].long(), st["new"].long(), st["table"]
    n_free, dev = st["free"].shape[0], table.device
    end = torch.cumsum(new, 0)
    tok_start = torch.cat((torch.zeros(1, dtype=torch.int64, device=dev), end))
    held = (ctx + P - 1) // P
    fits = (ctx + new <= mp * P) & (end <= n_tok)
    need = torch.where(fits, (ctx + new + P - 1) // P - held, 0)
    page_end = torch.cumsum(need, 0)
    granted = fits & ((need == 0) | (page_end <= n_free))
    take = torch.where(granted, need, 0)
    # block table: the pages past the held ones come off the free list in order
    lp = torch.arange(mp, device=dev)[None, :]
    grown = (lp >= held[:, None]) & (lp < (held + take)[:, None])
    src = (page_end - need)[:, None] + lp - held[:, None]
    new_table = torch.where(grown, st["free"][src.clamp(0, n_free - 1)], table)
    # slot map: the request of token n is the last one that starts at or before it
    n = torch.arange(n_tok, device=dev)
    b = torch.searchsorted(end, n, right=True).clamp(max=ctx.shape[0] - 1)
    live = (n < tok_start[-1]) & granted[b]
    pos = ctx[b] + n - tok_start[b]
    page = new_table[b, (pos // P).clamp(0, mp - 1)].long()
    i32 = lambda x: x.to(torch.int32)  # noqa: E731
    counts = torch.stack((take.sum(), torch.where(granted, new, 0).sum()))
    return (new_table, i32(ctx + torch.where(granted, new, 0)), i32(tok_start), i32(granted),
            i32(torch.where(live, b, -1)), i32(torch.where(live, pos, -1)), torch.where(live, page * P + pos % P, -1),
            i32(counts))


def _plain_q4_store(st):
    """The values that the stored rows stand for, in the storage type."""
    def rounded(x):
        r = x.shape[-1]
        f = x.float()
        s = torch.nn.functional.pad(f.abs(), (0, _groups(r) * GROUP - r)).reshape(*f.shape[:-1], _groups(r), GROUP).amax(-1)
        s = (s / torch.full_like(s, 7.0)).to(torch.bfloat16).float().repeat_interleave(GROUP, -1)[..., :r]
        return (torch.round(f / s).clamp(-7, 7) * s).to(x.dtype)
    return rounded(st["k"]), rounded(st["v"])


def _unpack(rows, r, at, scale_at):
    """Values [..., r] of the codes at byte `at` of 4-bit rows, fp32."""
    w = rows[..., at:at + r // 2].contiguous().view(torch.int32)
    code = ((w.repeat_interleave(8, -1) >> _shifts(r, rows.device).to(torch.int32)) & 15) - 8
    g = _groups(r)
    s = rows[..., scale_at:scale_at + 2 * g].contiguous().view(torch.bfloat16).float()
    return code.float() * s.repeat_interleave(GROUP, -1)[..., :r]


def _plain_q4_decode(st):
    c = st["case"]
    rk, rv, t, style = c["r_k"], c["r_v"], c["t"], c["style"]
    B, H = c["B"], c["H"]
    pages = st["pool"][st["table"].long().clamp(min=0)]                      # [B, pages, H, P, bytes]
    rows = pages.permute(0, 2, 1, 3, 4).reshape(B, H, -1, pages.shape[-1])     # [B, H, L, bytes]
    L = rows.shape[2]
    scale_at = rk // 2 + rv // 2
    ck = _unpack(rows, rk, 0, scale_at)
    q0, q1 = _pairs(st["q"].float(), style)
    at = st["q_pos"].long()
    cos, sin = st["cos"][at][:, None], st["sin"][at][:, None]
    q = _join(q0 * cos - q1 * sin, q0 * sin + q1 * cos, style)
    k = torch.matmul(ck, st["wk"][t].float().transpose(-1, -2)) + st["mk"][:, None, t * D:(t + 1) * D]
    k0, k1 = _pairs(k, style)
    cos, sin = st["cos"][:L], st["sin"][:L]
    k = _join(k0 * cos - k1 * sin, k0 * sin + k1 * cos, style)
    s = torch.matmul(k, q[..., None])[..., 0] * D ** -0.5                      # [B, H, L]
    live = torch.arange(L, device=s.device) < st["lens"][:, None, None]
    s = torch.where(live, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.where(live, torch.exp(s - m), 0.0)
    cv = _unpack(rows, rv, rk // 2, scale_at + 2 * _groups(rk))
    a = torch.matmul(p[..., None, :], cv)[..., 0, :] / p.sum(-1, keepdim=True)
    o = torch.matmul(st["wv"][t].float(), a[..., None])[..., 0] + st["mv"][:, t * D:(t + 1) * D]
    return torch.where(st["lens"][:, None, None] > 0, o, 0.0).to(st["q"].dtype)


# ------------------------------------------------------------------ the library's calls

def _own_rope_table(st):
    return st["lla"].rope_table_scaled(st["dm"], st["case"]["n_pos"], st["scaling"], pos0=st["pos0"],
                                       cos=st["cos"], sin=st["sin"])


def _own_rope_apply(st):
    c = st["case"]
    return st["lla"].rope_apply(st["dm"], st["x"], st["pos"], st["cos"], st["sin"], out=st["out"], offset=c["offset"],
                                scale=c["scale"], inverse=c["inverse"], workspace=st["ws"])


def _own_page_plan(st):
    p = st["plan"]
    p(st["P"], st["num_pages"], st["ctx"], st["new"], st["free"], st["table"])
    return (st["table"], p.seq_lens, p.tok_start, p.granted, p.seq_idx, p.pos, p.slots, p.counts)


def _own_q4_store(st):
    lla = st["lla"]
    lla.q4_store(st["dm"], st["k"], st["v"], st["slots"], st["pool"], st["ws"])
    lla.q4_load(st["dm"], st["slots"], st["pool"], st["out_k"], st["out_v"], st["ws"])
    return st["out_k"], st["out_v"]


def _own_q4_decode(st):
    st["lla"].decode_attn_q4(st["dm"], st["case"]["t"], st["q"], st["pool"], st["table"], st["lens"], st["q_pos"],
                             st["wk"], st["wv"], st["mk"], st["mv"], st["cos"], st["sin"], st["out"], None, st["ws"])
    return st["out"]


_PLAIN = {"rope_table": _plain_rope_table, "rope_apply": _plain_rope_apply, "page_plan": _plain_page_plan,
          "q4_store": _plain_q4_store, "q4_decode": _plain_q4_decode}
_OWN = {"rope_table": _own_rope_table, "rope_apply": _own_rope_apply, "page_plan": _own_page_plan,
        "q4_store": _own_q4_store, "q4_decode": _own_q4_decode}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op == "rope_table":
        # two fp32 values written per position and frequency; a product and two functions each
        n = case["n_pos"] * (case["d"] // 2)
        return {"bytes": 8 * n, "flops": 3 * n}
    if op == "rope_apply":
        # every element read and written once, each position's row of the table once
        e = 2 if case["dtype"] == "bf16" else 4
        x = case["n"] * case["heads"] * case["d_x"]
        rows = min(case["n"], case["rope_len"]) * case["d_rope"] * 4
        return {"bytes": 2 * x * e + rows + 4 * case["n"], "flops": 4 * case["n"] * case["heads"] * case["d_rope"]}
    if op == "page_plan":
        # lengths in; per request its length, start, grant; per token entry 16 bytes of maps, per page a table entry
        tok = _token_slots(case)
        return {"bytes": int(case["B"] * 20 + tok * 16 + 8 * tok / case["page"]), "flops": int(4 * case["B"] + 4 * tok)}
    if op == "q4_store":
        # latents read, rows written and read back, the values written
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["n"] * case["H"]
        r = case["r_k"] + case["r_v"]
        return {"bytes": 2 * n * r * e + 2 * n * _row_bytes(case["r_k"], case["r_v"]) + 16 * case["n"], "flops": 5 * n * r}
    # every live row once, the loop's weights, queries and outputs; the score contracts a token's K latent with
    # the folded query (128 x r_k), the value path adds the V latent up
    rk, rv, e = case["r_k"], case["r_v"], 2 if case["dtype"] == "bf16" else 4
    tok = case["B"] * (case["len_lo"] + case["len_hi"]) / 2
    rows = tok * case["H"] * _row_bytes(rk, rv)
    weights = case["H"] * D * (rk + rv) * e + 2 * case["H"] * D * 4
    table = case["len_hi"] * D * 4
    io = 2 * case["B"] * case["H"] * D * e + 4 * tok / case["page"]
    flops = tok * case["H"] * (2 * D * rk + 2 * D * 2 + 2 * rv) + case["B"] * case["H"] * 2 * D * (rk + rv)
    return {"bytes": int(rows + weights + table + io), "flops": int(flops)}


# ------------------------------------------------------------------ in 64 bits

def _exact_rows(rows, r_k, r_v):
    """K and V latents of 4-bit rows, byte by byte, in 64 bits."""
    out, at, sc = [], 0, r_k // 2 + r_v // 2
    for r in (r_k, r_v):
        cols = []
        for c in range(r):
            bit = 4 * ((c % 8) // 2) + 16 * (c % 2)
            byte = rows[..., at + 4 * (c // 8) + bit // 8].to(torch.int16)
            code = ((byte >> (bit % 8)) & 15) - 8
            g = sc + 2 * (c // GROUP)
            bits = (rows[..., g].to(torch.int32) << 16) | (rows[..., g + 1].to(torch.int32) << 24)
            cols.append(code.double() * bits.view(torch.float32).double())
        out.append(torch.stack(cols, -1))
        at += r // 2
        sc += 2 * _groups(r)
    return out


def exact(case, seed):
    op = case["op"]
    if op == "page_plan":
        return None        # whole numbers only
    st = prepare(case, seed)
    if op == "rope_table":
        rows = torch.arange(st["pos0"], st["pos0"] + case["n_pos"], dtype=torch.float64, device="cuda")
        f = torch.outer(rows, _thetas(case).cuda())
        return torch.cos(f), torch.sin(f)
    if op == "rope_apply":
        x = st["x"].double().clone()
        o, d, at = case["offset"], case["d_rope"], st["pos"].long()
        for f in range(d // 2):
            i, j = (o + f, o + f + d // 2) if case["style"] == 0 else (o + 2 * f, o + 2 * f + 1)
            z = torch.polar(torch.ones_like(at, dtype=torch.float64), torch.atan2(st["sin"][at, f].double(), st["cos"][at, f].double()))
            z = z * torch.hypot(st["sin"][at, f].double(), st["cos"][at, f].double()) * case["scale"]
            z = z.conj() if case["inverse"] else z
            w = torch.complex(x[..., i], x[..., j]) * z[:, None]
            x[..., i], x[..., j] = w.real, w.imag
        return x
    if op == "q4_store":
        # the scale is the bf16 of the fp32 quotient, a code the nearest integer to an fp32 quotient
        def grid(x):
            y = x.double()
            for g in range(0, y.shape[-1], GROUP):
                s = (y[..., g:g + GROUP].abs().amax(-1, keepdim=True) / 7).float().bfloat16().double()
                y[..., g:g + GROUP] = torch.clamp(torch.round((y[..., g:g + GROUP] / s).float()), -7, 7).double() * s
            return y
        return grid(st["k"].clone()), grid(st["v"].clone())
    B, H, t, P = case["B"], case["H"], case["t"], case["page"]
    out = torch.zeros(B, H, D, dtype=torch.float64, device="cuda")
    f = torch.arange(D // 2, device="cuda")
    i, j = (f, f + D // 2) if case["style"] == 0 else (2 * f, 2 * f + 1)
    wk, wv = st["wk"][t].double(), st["wv"][t].double()
    mk, mv = (st[n][:, t * D:(t + 1) * D].double() for n in ("mk", "mv"))
    for b in range(B):
        L = int(st["lens"][b])
        if L == 0:
            continue
        pages = st["pool"][st["table"][b, :(L + P - 1) // P].long()]           # [pages, H, P, bytes]
        ck, cv = _exact_rows(pages.transpose(0, 1).flatten(1, 2)[:, :L], case["r_k"], case["r_v"])
        k = torch.einsum("hlr,hdr->hld", ck, wk) + mk[:, None]
        q, at = st["q"][b].double(), int(st["q_pos"][b])
        key = torch.complex(k[..., i], k[..., j]) * torch.complex(st["cos"][:L].double(), st["sin"][:L].double())
        qry = torch.complex(q[:, i], q[:, j]) * torch.complex(st["cos"][at].double(), st["sin"][at].double())
        p = torch.softmax(torch.einsum("hlf,hf->hl", key, qry.conj()).real / math.sqrt(D), -1)
        out[b] = torch.einsum("hl,hlr,hdr->hd", p, cv, wv) + mv
    return out
