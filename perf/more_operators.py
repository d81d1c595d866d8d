"""Operators of a step that verifies drafted tokens, in their plain form and as the library's calls.

A server that drafts a tree of tokens for every sequence and checks all of them in one step
needs, around the model's own layers:

  tree_attn      attention of every drafted token over the sequence's latent cache and over the
                 drafted tokens on its path, whose keys and values are exact
  logits_adjust  repetition, presence and frequency penalties, biases and grammar masks on the
                 logits of every drafted token, with each row's best token and log-sum-exp
  tree_accept    the walk down the drafted tree along the tokens that the model chose

``run`` computes the plain form with elementary torch operations in 32 bits while ``own`` is
false, and calls the library while it is true.

A tree is ``tok_start`` [B + 1] (the nodes of sequence b are the token entries
tok_start[b] .. tok_start[b + 1] - 1; entries behind the last sequence are padding and are
left as they were), ``parent`` (index among the sequence's nodes, -1 for a root) and ``pos``.
"""
import math

import torch

own = False

D = 128            # head width


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one sequence of a chat, a short chain of drafted tokens: latency
        {"name": "tree_1x500_chain4", "op": "tree_attn", "B": 1, "H": 16, "len_lo": 500, "len_hi": 500, "r_k": 96,
         "r_v": 160, "page": 0, "T": 4, "t": 1, "style": 0, "dtype": "bf16", "nodes_lo": 4, "nodes_hi": 4, "branch": 1},
        # one layer of a 1.4B looped decoder at 4x compression, ragged lengths, small trees
        {"name": "tree_32x4096_n16", "op": "tree_attn", "B": 32, "H": 16, "len_lo": 3584, "len_hi": 4096, "r_k": 96,
         "r_v": 160, "page": 0, "T": 4, "t": 1, "style": 0, "dtype": "bf16", "nodes_lo": 9, "nodes_hi": 16, "branch": 3},
        # the same layer over pages, long contexts, the largest usual trees
        {"name": "tree_8x16384_n64_paged", "op": "tree_attn", "B": 8, "H": 16, "len_lo": 15000, "len_hi": 16384,
         "r_k": 96, "r_v": 160, "page": 64, "T": 4, "t": 3, "style": 1, "dtype": "bf16", "nodes_lo": 40, "nodes_hi": 64,
         "branch": 4},
        # a serving batch at 21.3x compression
        {"name": "tree_128x4096_small_n8", "op": "tree_attn", "B": 128, "H": 16, "len_lo": 2048, "len_hi": 4096, "r_k": 16,
         "r_v": 32, "page": 64, "T": 4, "t": 3, "style": 0, "dtype": "bf16", "nodes_lo": 1, "nodes_hi": 8, "branch": 2},
        # a chunk of a prompt (a chain) behind cached turns of a conversation
        {"name": "tree_16x2001_chunk128", "op": "tree_attn", "B": 16, "H": 16, "len_lo": 1000, "len_hi": 2001, "r_k": 64,
         "r_v": 128, "page": 0, "T": 4, "t": 0, "style": 0, "dtype": "bf16", "nodes_lo": 128, "nodes_hi": 128, "branch": 1},
        # fp32 storage, few short sequences, odd sizes, pages that end inside a tile
        {"name": "tree_f32_3x333_n7", "op": "tree_attn", "B": 3, "H": 2, "len_lo": 0, "len_hi": 333, "r_k": 96, "r_v": 160,
         "page": 24, "T": 4, "t": 2, "style": 0, "dtype": "f32", "nodes_lo": 1, "nodes_hi": 7, "branch": 3},
        # the logits of one request's tree
        {"name": "logits_1x4_32000", "op": "logits_adjust", "B": 1, "nodes_lo": 4, "nodes_hi": 4, "branch": 1,
         "vocab": 32000, "dtype": "bf16", "hist_lo": 500, "hist_hi": 500, "max_bias": 16, "masks": 0},
        # a serving batch with trees, a large vocabulary, long histories and grammars
        {"name": "logits_32x16_131072", "op": "logits_adjust", "B": 32, "nodes_lo": 9, "nodes_hi": 16, "branch": 3,
         "vocab": 131072, "dtype": "bf16", "hist_lo": 1000, "hist_hi": 4096, "max_bias": 64, "masks": 40},
        # plain steps (one node a request) of a large batch, fp32 logits, an odd vocabulary
        {"name": "logits_300x1_49999_f32", "op": "logits_adjust", "B": 300, "nodes_lo": 1, "nodes_hi": 1, "branch": 1,
         "vocab": 49999, "dtype": "f32", "hist_lo": 1, "hist_hi": 3000, "max_bias": 8, "masks": 7},
        # the walk down one tree, and down a serving batch's
        {"name": "accept_1_n8", "op": "tree_accept", "B": 1, "nodes_lo": 8, "nodes_hi": 8, "branch": 2},
        {"name": "accept_768_n64", "op": "tree_accept", "B": 768, "nodes_lo": 1, "nodes_hi": 64, "branch": 4},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree_attn", "tree_attn", "tree_attn", "logits_adjust", "logits_adjust", "tree_accept"])
    nodes = _log(rng, 1, 128)
    tree = {"nodes_lo": rng.randint(min(nodes, rng.choice([0, 1, 1])), nodes), "nodes_hi": nodes,
            "branch": rng.choice([1, 2, 3, 4, 8])}
    if op == "tree_attn":
        dtype = "f32" if rng.random() < 0.2 else "bf16"
        hi = _log(rng, 1, 2000 if dtype == "f32" else 20000)
        H = rng.randint(1, 16)
        most = (40000 if dtype == "f32" else 1500000) // (hi * H)
        return {"op": op, "B": _log(rng, 1, max(1, min(64, most))), "H": H, "len_lo": rng.randint(0, hi), "len_hi": hi,
                "r_k": 16 * rng.randint(1, 12), "r_v": 16 * rng.randint(1, 12),
                "page": rng.choice([0, 0, 1, 8, 16, 24, 64, 100, 128, 256]), "T": 4, "t": rng.randint(0, 3),
                "style": rng.randint(0, 1), "dtype": dtype, **tree}
    if op == "logits_adjust":
        vocab = _log(rng, 100, 200000)
        hi = _log(rng, 1, 8000)
        return {"op": op, "B": _log(rng, 1, max(1, min(300, 60000000 // (vocab * nodes)))), "vocab": vocab,
                "dtype": rng.choice(["bf16", "f32"]), "hist_lo": rng.randint(0, hi), "hist_hi": hi,
                "max_bias": rng.choice([0, 1, 16, 300]), "masks": rng.choice([0, 1, 20]), **tree}
    return {"op": op, "B": _log(rng, 1, 1500), **tree}


# ------------------------------------------------------------------ inputs

def _storage(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _tree(case, host):
    """tok_start, parent and depth of a random forest of one root a sequence, and the padding's parents.
    A node hangs under one of the `branch` nodes before it, so 1 gives chains."""
    B, lo, hi = case["B"], case["nodes_lo"], case["nodes_hi"]
    n = torch.randint(lo, hi + 1, (B,), generator=host)
    n[B - B // 2:] = (lo + hi - n[:B // 2]).flip(0)      # the same sum for every seed: a step's shapes are fixed
    if B % 2:
        n[B // 2] = (lo + hi) // 2
    i = torch.arange(hi)
    back = 1 + torch.randint(0, case["branch"], (B, hi), generator=host)
    parent = torch.clamp(i - back, min=0)
    parent[:, 0] = -1
    depth = torch.zeros((B, hi), dtype=torch.int64)
    for k in range(1, hi):
        depth[:, k] = torch.gather(depth, 1, parent[:, k:k + 1])[:, 0] + 1
    live = i[None, :] < n[:, None]
    tok_start = torch.cat((torch.zeros(1, dtype=torch.int64), torch.cumsum(n, 0)))
    pad = 3                                              # entries behind the last sequence
    flat = lambda x, fill: torch.cat((x[live], torch.full((pad,), fill, dtype=x.dtype)))  # noqa: E731
    return n, tok_start, flat(parent, -1), flat(depth, 0)


def _dims(case):
    from looped_transformer_cross_gb300 import lla
    return lla.dims(case["T"], case["H"], case["r_k"], case["r_v"],
                    dtype=lla.LLA_BF16 if case["dtype"] == "bf16" else lla.LLA_F32, rope_style=case["style"])


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(1000003 * (seed + 1) + 29)
    host = torch.Generator().manual_seed(7919 * (seed + 1) + 11)
    state = {"case": case}
    if own:
        from looped_transformer_cross_gb300 import lla
        state["lla"] = lla
    n, tok_start, parent, depth = _tree(case, host)
    B, N, n_tok = case["B"], max(1, case["nodes_hi"]), parent.shape[0]
    i32 = lambda x: x.to(torch.int32).to(dev)  # noqa: E731
    state.update(N=N, n_tok=n_tok, tok_start=i32(tok_start), parent=i32(parent))
    owner = torch.cat((torch.repeat_interleave(torch.arange(B), n), torch.zeros(3, dtype=torch.int64)))
    if case["op"] == "tree_attn":
        H, T, rk, rv, P = (case[x] for x in ("H", "T", "r_k", "r_v", "page"))
        sd = _storage(case)
        lens = torch.randint(case["len_lo"], case["len_hi"] + 1, (B,), generator=host)
        state["lens"] = i32(lens)
        state["pos"] = i32(lens[owner] + depth)
        rnd = lambda std, *s: torch.randn(*s, generator=gen, device=dev) * std  # noqa: E731
        cap = max(1, case["len_hi"])
        if P == 0:
            state["ck"], state["cv"] = rnd(1.0, B, H, cap, rk).to(sd), rnd(1.0, B, H, cap, rv).to(sd)
        else:
            mp = (cap + P - 1) // P
            held = (lens + P - 1) // P
            num = int(held.sum()) + 1
            state["ck"], state["cv"] = rnd(1.0, num, H, P, rk).to(sd), rnd(1.0, num, H, P, rv).to(sd)
            table = torch.full((B, mp), -1, dtype=torch.int32)
            table[torch.arange(mp)[None, :] < held[:, None]] = torch.randperm(num, generator=host)[: int(held.sum())].to(torch.int32)
            state["table"] = table.to(dev)
            cap = mp * P
        # queries, keys and values are slices of the step's fused projection
        state["qkv"] = rnd(1.0, n_tok, 3 * H, D).to(sd)
        state["wk"] = rnd(rk ** -0.5, T, H, D, rk).to(sd)
        state["wv"] = rnd(rv ** -0.5, T, H, D, rv).to(sd)
        state["mk"], state["mv"] = rnd(0.1 ** 0.5, H, T * D), rnd(0.1 ** 0.5, H, T * D)
        n_pos = max(128, cap + N)
        theta = 10000.0 ** (-2.0 * torch.arange(D // 2, dtype=torch.float64, device=dev) / D)
        ang = torch.arange(n_pos, dtype=torch.float64, device=dev)[:, None] * theta
        state["cos"], state["sin"] = ang.cos().float(), ang.sin().float()
        if own:
            state["dm"] = _dims(case)
            state["tree"] = lla.DraftTree(state["tok_start"], state["parent"], N, pos=state["pos"])
            state["out"] = torch.zeros((n_tok, H, D), dtype=sd, device=dev)
            state["lse"] = torch.zeros((n_tok, H), dtype=torch.float32, device=dev)
            state["ws"] = lla.tree_workspace(state["dm"], state["tree"], cap)
        return state
    if case["op"] == "logits_adjust":
        V, mb, nm, cap = case["vocab"], case["max_bias"], case["masks"], max(1, case["hist_hi"])
        state["logits"] = (3.0 * torch.randn(n_tok, V, generator=gen, device=dev)).to(_storage(case))
        # tokens as a text has them: few of them often
        skew = lambda *s: (V * torch.rand(*s, generator=gen, device=dev) ** 4).to(torch.int32).clamp_(max=V - 1)  # noqa: E731
        state["hist"], state["token"] = skew(B, cap), skew(n_tok)
        hl = torch.randint(case["hist_lo"], case["hist_hi"] + 1, (B,), generator=host)
        state["hist_len"] = i32(hl)
        state["prompt_len"] = i32((hl * torch.rand(B, generator=host)).to(torch.int64))
        unif = lambda lo, hi: lo + (hi - lo) * torch.rand(B, generator=gen, device=dev)  # noqa: E731
        state["rep"], state["pres"], state["freq"] = unif(1.0, 1.5), unif(0.0, 1.0), unif(0.0, 0.5)
        if mb:
            # a list of different tokens for each request, some of its entries unused
            step = max(1, V // mb)
            bt = (torch.arange(mb, device=dev) * step + torch.randint(0, step, (B, mb), generator=gen, device=dev)).to(torch.int32)
            bt[:, max(1, mb // 2):] = torch.where(torch.rand(B, mb - max(1, mb // 2), generator=gen, device=dev) < 0.5, -1, bt[:, max(1, mb // 2):])
            state["bias_token"] = torch.where(bt < V, bt, -1)
            state["bias"] = 4.0 * torch.randn(B, mb, generator=gen, device=dev)
        if nm:
            words = (V + 31) // 32
            dense = torch.randint(-2 ** 31, 2 ** 31, (nm, words), generator=gen, device=dev)
            for _ in range(2):                           # an eighth of the tokens allowed
                dense &= torch.randint(-2 ** 31, 2 ** 31, (nm, words), generator=gen, device=dev)
            dense[:, 0] |= 4                             # and the end of the text always
            state["allowed"] = torch.where(dense >= 2 ** 31, dense - 2 ** 32, dense).to(torch.int32)
            row = torch.randint(-nm // 2, nm, (n_tok,), generator=host).clamp(min=-1)
            state["allowed_row"] = i32(row)
        if own:
            state["tree"] = lla.DraftTree(state["tok_start"], state["parent"], N)
            state["rules"] = lla.LogitRules(state["hist"], state["hist_len"], state["prompt_len"], repetition=state["rep"],
                                            presence=state["pres"], frequency=state["freq"],
                                            bias_token=state.get("bias_token"), bias=state.get("bias"),
                                            allowed=state.get("allowed"), allowed_row=state.get("allowed_row"))
            state["out"] = torch.zeros_like(state["logits"])
            state["best"] = torch.zeros(n_tok, dtype=torch.int32, device=dev)
            state["lse"] = torch.zeros(n_tok, dtype=torch.float32, device=dev)
            state["ws"] = lla.logits_workspace(state["tree"], V)
        return state
    # tokens of which one child in two is the one that the model chose after its parent
    state["token"] = torch.randint(0, 4, (n_tok,), generator=host).to(torch.int32).to(dev)
    state["chosen"] = torch.randint(0, 4, (n_tok,), generator=host).to(torch.int32).to(dev)
    state["ctx"] = torch.randint(0, 8000, (B,), generator=host).to(torch.int32).to(dev)
    if own:
        state["tree"] = lla.DraftTree(state["tok_start"], state["parent"], N)
        state["walk"] = lla.TreeAccept(state["tree"])
        state["walk"].path.zero_(), state["walk"].seq_idx.zero_(), state["walk"].pos.zero_()
    return state


# ------------------------------------------------------------------ plain forms

def _padded(st):
    """Token entry [B, N] of each sequence's nodes (clamped), and which of them there are."""
    at = st["tok_start"][:-1, None].long() + torch.arange(st["N"], device=st["parent"].device)
    live = at < st["tok_start"][1:, None]
    return torch.where(live, at, 0), live


def _paths(parent, live):
    """[B, N, N]: node j is i or one of i's ancestors; by repeated squaring of the parent relation."""
    N = parent.shape[1]
    j = torch.arange(N, device=parent.device)
    m = ((parent[:, :, None] == j) | (j[:, None] == j)).float() * live[:, :, None]
    for _ in range(max(1, (N - 1).bit_length())):
        m = (torch.matmul(m, m) > 0).float()
    return m > 0


def _turn(x, cos, sin, style):
    h = x.shape[-1] // 2
    a, b = (x[..., :h], x[..., h:]) if style == 0 else (x[..., 0::2], x[..., 1::2])
    a, b = a * cos - b * sin, a * sin + b * cos
    return torch.cat((a, b), -1) if style == 0 else torch.stack((a, b), -1).flatten(-2)


def _latents(st, name):
    """The cache [B, H, L, r], fp32, through the block table where there is one."""
    if "table" not in st:
        return st[name].float()
    pages = st[name][st["table"].long().clamp(min=0)].float()               # [B, pages, H, P, r]
    return pages.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_tree_attn(st):
    c = st["case"]
    t, style, H = c["t"], c["style"], c["H"]
    at, live = _padded(st)
    path = _paths(st["parent"][at], live)
    pos = st["pos"][at].long()
    qkv = st["qkv"][at].float()                                              # [B, N, 3H, D]
    q, kd, vd = (qkv[:, :, i * H:(i + 1) * H].transpose(1, 2) for i in range(3))
    cos, sin = st["cos"][pos][:, None], st["sin"][pos][:, None]
    q, kd = _turn(q, cos, sin, style), _turn(kd, cos, sin, style)
    ck = _latents(st, "ck")
    L = ck.shape[2]
    k = torch.matmul(ck, st["wk"][t].float().transpose(-1, -2)) + st["mk"][:, None, t * D:(t + 1) * D]
    k = _turn(k, st["cos"][:L], st["sin"][:L], style)
    s = torch.matmul(q, k.transpose(-1, -2)) * D ** -0.5                       # [B, H, N, L]
    del k, ck
    held = torch.arange(L, device=s.device) < st["lens"][:, None, None, None]
    s = torch.where(held, s, -math.inf)
    sd = torch.where(path[:, None], torch.matmul(q, kd.transpose(-1, -2)) * D ** -0.5, -math.inf)
    m = torch.maximum(s.amax(-1, keepdim=True), sd.amax(-1, keepdim=True))
    m = torch.where(live[:, None, :, None], m, 0.0)
    p, pd = torch.exp(s - m), torch.exp(sd - m)
    del s
    cv = torch.where(held.transpose(-1, -2), _latents(st, "cv"), 0.0)
    a, held_sum = torch.matmul(p, cv), p.sum(-1, keepdim=True)
    o = torch.matmul(a, st["wv"][t].float().transpose(-1, -2)) + held_sum * st["mv"][:, None, t * D:(t + 1) * D]
    o = o + torch.matmul(pd, vd)
    z = held_sum + pd.sum(-1, keepdim=True)
    o, lse = o / z, (m + torch.log(z))[..., 0]
    out = torch.zeros((st["n_tok"], H, D), dtype=st["qkv"].dtype, device=o.device)
    res = torch.zeros((st["n_tok"], H), dtype=torch.float32, device=o.device)
    out[at[live]] = o.transpose(1, 2)[live].to(out.dtype)
    res[at[live]] = lse.transpose(1, 2)[live]
    return out, res


def _plain_logits_adjust(st):
    c = st["case"]
    V, n_tok, dev = c["vocab"], st["n_tok"], st["logits"].device
    at, live = _padded(st)
    path = _paths(st["parent"][at], live)
    n_live = st["tok_start"][-1]
    row = torch.arange(n_tok, device=dev)
    b = torch.searchsorted(st["tok_start"][1:].contiguous(), row.to(torch.int32), right=True).clamp(max=c["B"] - 1)
    # occurrences in the output part of the history and in its prompt part
    j = torch.arange(st["hist"].shape[1], device=dev)
    inside, prompt = j < st["hist_len"][:, None], j < st["prompt_len"][:, None]
    hist = st["hist"].long()
    out_part = torch.zeros((c["B"], V), device=dev).scatter_add_(1, hist, (inside & ~prompt).float())
    in_prompt = torch.zeros((c["B"], V), device=dev).scatter_add_(1, hist, (inside & prompt).float())
    count = out_part[b]
    which = path.nonzero()                                                   # (sequence, node, its ancestor)
    count.index_put_((at[which[:, 0], which[:, 1]], st["token"][at[which[:, 0], which[:, 2]]].long()),
                     torch.ones(which.shape[0], device=dev), accumulate=True)
    x = st["logits"].float()
    r = st["rep"][b][:, None]
    x = torch.where((count > 0) | (in_prompt[b] > 0), torch.where(x > 0, x / r, x * r), x)
    x = x - st["freq"][b][:, None] * count
    x = x - torch.where(count > 0, st["pres"][b][:, None], 0.0)
    if "bias" in st:
        used = st["bias_token"] >= 0
        bias = torch.zeros((c["B"], V), device=dev).scatter_add_(1, st["bias_token"].clamp(min=0).long(), torch.where(used, st["bias"], 0.0))
        x = x + bias[b]
    if "allowed" in st:
        v = torch.arange(V, device=dev)
        rows = st["allowed"][st["allowed_row"].clamp(min=0).long()]
        bit = (rows[:, v // 32] >> (v % 32).to(torch.int32)) & 1
        x = torch.where((bit == 1) | (st["allowed_row"] < 0)[:, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    best = torch.where(x == m, torch.arange(V, device=dev), V).amin(-1)
    lse = m[:, 0] + torch.log(torch.exp(x - m).sum(-1))
    keep = row < n_live
    return (torch.where(keep[:, None], x, 0.0).to(st["logits"].dtype), torch.where(keep, best, 0).to(torch.int32),
            torch.where(keep, lse, 0.0))


def _plain_tree_accept(st):
    B, N, dev = st["case"]["B"], st["N"], st["parent"].device
    at, live = _padded(st)
    parent, token, chosen = st["parent"][at], st["token"][at], st["chosen"][at]
    i = torch.arange(N, device=dev)
    cur = torch.zeros(B, dtype=torch.int64, device=dev)
    going = live[:, 0]
    rank = torch.where(live & (i == 0), 0, -1)                               # place on the accepted path
    for step in range(1, N):
        want = torch.gather(chosen, 1, cur[:, None])
        child = live & (parent == cur[:, None]) & (token == want) & going[:, None]
        first = torch.where(child, i, N).amin(-1)
        going = first < N
        cur = torch.where(going, first, cur)
        rank = torch.where((i == cur[:, None]) & going[:, None], step, rank)
    taken = rank >= 0
    count = taken.sum(-1)
    some = live[:, 0]
    nxt = torch.where(some, torch.gather(chosen, 1, cur[:, None])[:, 0], -1)
    # accepted nodes take the positions behind the cached tokens, the others the ones after them
    behind = count[:, None] + torch.cumsum((live & ~taken).long(), -1) - 1
    pos = st["ctx"][:, None] + torch.where(taken, rank, behind)
    # the accepted entries of each sequence, in path order from its first entry on
    order = torch.full((B, N + 1), -1, dtype=torch.int64, device=dev).scatter_(1, torch.where(taken, rank, N), at)[:, :N]
    flat = lambda x: torch.zeros(st["n_tok"], dtype=torch.int32, device=dev).index_put_((at[live],), x[live].to(torch.int32))  # noqa: E731
    order = torch.where(i < count[:, None], order, -1)
    seq = torch.arange(B, device=dev)[:, None].expand(B, N)
    w = lambda x: x.to(torch.int32)  # noqa: E731
    return w(count), w(nxt), w(st["ctx"] + count), flat(order), flat(seq), flat(pos)


# ------------------------------------------------------------------ the library's calls

def _own_tree_attn(st):
    lla, c, H = st["lla"], st["case"], st["case"]["H"]
    q, k, v = (st["qkv"][:, i * H:(i + 1) * H] for i in range(3))
    rest = (st["lens"], st["wk"], st["wv"], st["mk"], st["mv"], st["cos"], st["sin"], st["out"], st["lse"], st["ws"])
    if "table" in st:
        lla.tree_attn_paged(st["dm"], c["t"], st["tree"], q, k, v, st["ck"], st["cv"], st["table"], c["page"], *rest)
    else:
        lla.tree_attn(st["dm"], c["t"], st["tree"], q, k, v, st["ck"], st["cv"], *rest)
    return st["out"], st["lse"]


def _own_logits_adjust(st):
    st["lla"].logits_adjust(st["tree"], st["token"], st["logits"], st["rules"], out=st["out"], best=st["best"],
                            lse=st["lse"], workspace=st["ws"])
    return st["out"], st["best"], st["lse"]


def _own_tree_accept(st):
    w = st["walk"](st["token"], st["chosen"], st["ctx"])
    return w.count, w.next_token, w.seq_lens, w.path, w.seq_idx, w.pos


_PLAIN = {"tree_attn": _plain_tree_attn, "logits_adjust": _plain_logits_adjust, "tree_accept": _plain_tree_accept}
_OWN = {"tree_attn": _own_tree_attn, "logits_adjust": _own_logits_adjust, "tree_accept": _own_tree_accept}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    nodes = case["B"] * (case["nodes_lo"] + case["nodes_hi"]) / 2
    if op == "tree_accept":
        # three words a node in, three out; three words a request in, three out
        return {"bytes": int(24 * nodes + 20 * case["B"]), "flops": int(2 * nodes)}
    if op == "logits_adjust":
        # logits read and written, a mask bit per logit, histories; a comparison, an exponential and a sum a logit
        e = 2 if case["dtype"] == "bf16" else 4
        n = nodes * case["vocab"]
        masks = min(case["masks"], nodes) * case["vocab"] / 8
        hist = 4 * case["B"] * (case["hist_lo"] + case["hist_hi"]) / 2 + 8 * case["B"] * case["max_bias"]
        return {"bytes": int(2 * n * e + masks + hist + 12 * nodes), "flops": int(4 * n)}
    # every cached token's latents once, the loop's weights, the nodes' vectors in and out; a key is
    # reconstructed and turned once for all nodes, and meets each of them
    rk, rv, e, H = case["r_k"], case["r_v"], 2 if case["dtype"] == "bf16" else 4, case["H"]
    per = (case["nodes_lo"] + case["nodes_hi"]) / 2
    tok = case["B"] * (case["len_lo"] + case["len_hi"]) / 2
    latents = tok * H * (rk + rv) * e
    weights = H * D * (rk + rv) * e + 2 * H * D * 4
    table = case["len_hi"] * D * 4
    io = nodes * H * (4 * D * e + 4)
    flops = tok * H * (2 * D * rk + 3 * D + per * (2 * D + 2 * rv)) + nodes * H * 2 * D * rv
    return {"bytes": int(latents + weights + table + io), "flops": int(flops)}


# ------------------------------------------------------------------ in 64 bits

def _chain(parent, i):
    """Node i and its ancestors."""
    got = []
    while i >= 0:
        got.append(i)
        i = parent[i]
    return got


def _exact_tree_attn(case, st):
    H, t, P = case["H"], case["t"], case["page"]
    out = torch.zeros((st["n_tok"], H, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((st["n_tok"], H), dtype=torch.float64, device="cuda")
    start, parent, lens = st["tok_start"].tolist(), st["parent"].tolist(), st["lens"].tolist()
    f = torch.arange(D // 2, device="cuda")
    i0, i1 = (f, f + D // 2) if case["style"] == 0 else (2 * f, 2 * f + 1)
    wk, wv = st["wk"][t].double(), st["wv"][t].double()
    mk, mv = (st[n][:, t * D:(t + 1) * D].double() for n in ("mk", "mv"))

    def pairs(x, at):                                    # [..., len(at), D] turned, as complex numbers
        z = torch.complex(x[..., i0], x[..., i1])
        return z * torch.complex(st["cos"][at].double(), st["sin"][at].double())

    for b in range(case["B"]):
        s0, n, L = start[b], start[b + 1] - start[b], lens[b]
        if n == 0:
            continue
        if P:
            pages = st["table"][b, :(L + P - 1) // P].long()
            ck, cv = (st[x][pages].transpose(0, 1).flatten(1, 2)[:, :L].double() for x in ("ck", "cv"))
        else:
            ck, cv = (st[x][b, :, :L].double() for x in ("ck", "cv"))
        qkv = st["qkv"][s0:s0 + n].double().transpose(0, 1)                     # [3H, n, D]
        at = st["pos"][s0:s0 + n].long()
        q, kd, vd = pairs(qkv[:H], at), pairs(qkv[H:2 * H], at), qkv[2 * H:]
        k = pairs(torch.einsum("hlr,hdr->hld", ck, wk) + mk[:, None], torch.arange(L, device="cuda"))
        own_path = torch.zeros((n, n), dtype=torch.bool)
        for i in range(n):
            own_path[i, _chain(parent[s0:s0 + n], i)] = True
        s = torch.einsum("hnf,hlf->hnl", q, torch.cat((k, kd), 1).conj()).real / math.sqrt(D)
        s[:, :, L:][:, ~own_path.cuda()] = -math.inf
        p = torch.softmax(s, -1)
        o = torch.einsum("hnr,hdr->hnd", torch.einsum("hnl,hlr->hnr", p[..., :L], cv), wv)
        o = o + p[..., :L].sum(-1, keepdim=True) * mv[:, None] + torch.einsum("hnm,hmd->hnd", p[..., L:], vd)
        out[s0:s0 + n], lse[s0:s0 + n] = o.transpose(0, 1), torch.logsumexp(s, -1).T
    return out, lse


def _exact_logits_adjust(case, st):
    V = case["vocab"]
    out = torch.zeros((st["n_tok"], V), dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["n_tok"], dtype=torch.float64, device="cuda")
    start, parent, token = st["tok_start"].tolist(), st["parent"].tolist(), st["token"].tolist()
    hl, pl = st["hist_len"].tolist(), st["prompt_len"].tolist()
    which = st["allowed_row"].tolist() if "allowed" in st else [-1] * st["n_tok"]
    shift = torch.arange(32, device="cuda")
    for b in range(case["B"]):
        said = torch.bincount(st["hist"][b, pl[b]:hl[b]], minlength=V)
        asked = torch.bincount(st["hist"][b, :pl[b]], minlength=V) > 0
        extra = torch.zeros(V, dtype=torch.float64, device="cuda")
        if "bias" in st:
            u = st["bias_token"][b] >= 0
            extra[st["bias_token"][b][u].long()] = st["bias"][b][u].double()
        r, p, f = (st[x][b].double() for x in ("rep", "pres", "freq"))
        for i in range(start[b + 1] - start[b]):
            at = start[b] + i
            words = [token[start[b] + a] for a in _chain(parent[start[b]:start[b + 1]], i)]
            n = said + torch.bincount(torch.tensor(words, device="cuda"), minlength=V)
            x = st["logits"][at].double()
            seen = (n > 0) | asked
            x = torch.where(seen & (x > 0), x / r, torch.where(seen, x * r, x))
            x = x - f * n - p * (n > 0) + extra
            if which[at] >= 0:
                bits = (st["allowed"][which[at]].long()[:, None] >> shift) & 1
                x = x.masked_fill(bits.flatten()[:V] == 0, -math.inf)
            out[at], lse[at] = x, torch.logsumexp(x, 0)
    return out, None, lse


def exact(case, seed):
    if case["op"] == "tree_accept":
        return None        # whole numbers only
    st = prepare(case, seed)
    return (_exact_tree_attn if case["op"] == "tree_attn" else _exact_logits_adjust)(case, st)
