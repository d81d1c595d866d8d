"""lla_logits_adjust and lla_tree_accept against the 64-bit oracle, and a whole verification step.

Tolerance of a logit: five fp32 operations, each off by half a step (2^-24) of the largest value
on the way, and half a step of the storage type where that is bf16 (2^-8).  Log-sum-exp: 2^-24 for
each of its value's roundings and of the sum's, 1e-5 in all.  Best tokens, and everything about
acceptance, are equal."""
import math

import numpy as np
import pytest
import torch

from lla_cases import widen
from looped_transformer_cross_gb300 import lla
from oracle import tree as otree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from looped_transformer_cross_gb300 import build
    build.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def forest(nodes, branch, g, pad=2):
    parent = []
    for m in nodes:
        parent += [-1 if i == 0 else max(0, i - 1 - int(torch.randint(0, branch, (1,), generator=g))) for i in range(m)]
    return [0] + [int(x) for x in np.cumsum(nodes)], parent + [-1] * pad


def make(nodes, V, dtype="f32", hist=50, max_bias=5, masks=3, branch=2, seed=0, stride=None, pad=2):
    g = torch.Generator().manual_seed(seed + V + sum(nodes))
    rint = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g)  # noqa: E731
    B = len(nodes)
    start, parent = forest(nodes, branch, g, pad)
    n_tok = len(parent)
    sd = torch.bfloat16 if dtype == "bf16" else torch.float32
    few = min(V, 40)                                  # tokens that repeat
    c = dict(nodes=nodes, V=V, B=B, n_tok=n_tok, dtype=dtype)
    c["tree"] = lla.DraftTree(i32(start), i32(parent), max([1, *nodes]))
    c["start"], c["parent"] = start, parent
    stride = V if stride is None else stride
    buf = torch.full((n_tok, stride), float("nan"), dtype=sd)
    buf[:, :V] = (3 * torch.randn(n_tok, V, generator=g)).to(sd)
    buf[start[-1]:] = float("nan")
    c["buf"] = buf.cuda()
    c["logits"] = c["buf"][:, :V]
    tok = rint(0, few, n_tok)
    tok[tok == 3] = V - 1
    c["token"] = tok.to(torch.int32).cuda()
    c["history"] = torch.where(torch.rand(B, hist, generator=g) < 0.7, rint(0, few, B, hist), rint(0, V, B, hist)).to(torch.int32)
    c["hist_len"] = rint(0, hist + 1, B)
    c["hist_len"][0] = hist
    c["prompt_len"] = (c["hist_len"] * torch.rand(B, generator=g)).long()
    c["rep"], c["pres"], c["freq"] = 1 + torch.rand(B, generator=g), torch.rand(B, generator=g), torch.rand(B, generator=g)
    if max_bias:
        c["bias_token"] = rint(0, V, B, max_bias).to(torch.int32)
        c["bias_token"][:, 0] = V - 1
        if max_bias > 2:
            c["bias_token"][:, 1], c["bias_token"][:, 2] = -1, V - 1          # an unused entry, a token twice
        c["bias"] = 2 * torch.randn(B, max_bias, generator=g)
    if masks:
        words = (V + 31) // 32
        bits = torch.rand(masks, words * 32, generator=g) < 0.3
        bits[0] = False                                                        # nothing allowed
        if masks > 1:
            bits[1] = False
            bits[1, V - 1] = True                                              # one token
        c["bits"] = bits[:, :V]
        packed = (bits.view(masks, words, 32).long() << torch.arange(32)).sum(-1)
        c["allowed"] = torch.where(packed >= 1 << 31, packed - (1 << 32), packed).to(torch.int32).cuda()
        c["allowed_row"] = rint(-1, masks, n_tok).to(torch.int32).cuda()
    c["best"], c["lse"] = torch.full((n_tok,), 99, dtype=torch.int32, device="cuda"), torch.full((n_tok,), 99.0, device="cuda")
    return c


def rules_of(c):
    up = lambda k: c[k].to(torch.int32).cuda() if k in c else None  # noqa: E731
    return lla.LogitRules(up("history"), up("hist_len"), up("prompt_len"), repetition=c["rep"].cuda(), presence=c["pres"].cuda(),
                          frequency=c["freq"].cuda(), bias_token=up("bias_token"), bias=c["bias"].cuda() if "bias" in c else None,
                          allowed=c.get("allowed"), allowed_row=c.get("allowed_row"))


def expected(c):
    hist = [c["history"][b, : int(c["hist_len"][b])].tolist() for b in range(c["B"])]
    bias = [[(t, v) for t, v in zip(c["bias_token"][b].tolist(), c["bias"][b].tolist()) if t >= 0] if "bias" in c else [] for b in range(c["B"])]
    rows = c["allowed_row"].tolist() if "allowed" in c else [-1] * c["n_tok"]
    allowed = [None if r < 0 or r >= len(c["bits"]) else set(np.flatnonzero(c["bits"][r].numpy()).tolist()) for r in rows]
    return otree.logits_adjust(widen(c["logits"]), c["start"], c["parent"], c["token"].tolist(), hist, c["prompt_len"].tolist(),
                               c["rep"].tolist(), c["pres"].tolist(), c["freq"].tolist(), bias, allowed)


def compare(c, x, best, lse, out):
    n = c["start"][-1]
    got = widen(out)[:n]
    fin = np.isfinite(x[:n])
    assert np.array_equal(np.isneginf(got), np.isneginf(x[:n])) and np.array_equal(np.isfinite(got), fin)
    size = np.abs(widen(c["logits"]))[:n] * 2.0 + c["history"].shape[1] + 130.0       # repetition, counts, biases
    tol = 5 * 2.0 ** -24 * size + (2.0 ** -8 * np.abs(np.where(fin, x[:n], 0)) if c["dtype"] == "bf16" else 0)
    assert (np.abs(np.where(fin, got - x[:n], 0)) <= tol).all()
    assert np.array_equal(c["best"].cpu().numpy()[:n], best[:n])
    gl = widen(c["lse"])[:n]
    assert np.array_equal(np.isneginf(gl), np.isneginf(lse[:n]))
    f = np.isfinite(lse[:n])
    assert (np.abs(gl[f] - lse[:n][f]) <= 1e-5).all()
    assert (c["best"][n:] == 99).all() and (c["lse"][n:] == 99.0).all()


def run(c, out=None, rules=None):
    ws = lla.logits_workspace(c["tree"], c["V"])
    lla.logits_adjust(c["tree"], c["token"], c["logits"], rules_of(c) if rules is None else rules, out=out, best=c["best"], lse=c["lse"], workspace=ws)
    return ws


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nodes,V,branch", [
    ([1], 1, 1), ([1], 2, 1), ([3], 33, 1), ([1, 0, 2], 4096, 1), ([5, 1], 4097, 2), ([16, 9, 1], 12001, 3), ([128], 5000, 1),
    ([64, 33], 8191, 4), ([2] * 40, 64, 1), ([1] * 300, 999, 1), ([3, 3], 70000, 2)])
def test_logits(nodes, V, branch, dtype):
    """Penalties, biases (a token twice, the vocabulary's last), masks (none, one token, nothing): against
    the oracle, the padding's rows untouched."""
    c = make(nodes, V, dtype, branch=branch)
    out = torch.full_like(c["logits"], 55.0)
    x, best, lse = expected(c)
    ws = run(c, out)
    assert lla.device_status(ws) == lla.LLA_OK
    compare(c, x, best, lse, out)
    assert (out[c["start"][-1]:] == 55.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("stride", [5001, 5002, 6000])
def test_in_place_and_strides(dtype, stride):
    c = make([4, 7], 5000, dtype, stride=stride)
    x, best, lse = expected(c)
    before = c["buf"].clone()
    c0 = dict(c, logits=c["logits"].clone())
    run(c, c["logits"])
    compare(c0 | {"best": c["best"], "lse": c["lse"]}, x, best, lse, c["logits"])
    assert torch.equal(c["buf"][:, 5000:].isnan(), before[:, 5000:].isnan())
    c = make([4, 7], 4999, dtype)                     # rows that start within a pair, into an aligned buffer
    x, best, lse = expected(c)
    out = torch.full((c["n_tok"], stride), 55.0, dtype=c["logits"].dtype, device="cuda")
    run(c, out[:, :4999])
    compare(c, x, best, lse, out[:, :4999])
    assert (out[:, 4999:] == 55.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_histories_and_many_biases(dtype):
    """Counts past 14 bits, and more biases of one stretch of the vocabulary than shared memory holds."""
    c = make([3, 2], 6000, dtype, hist=20000, max_bias=400)
    c["history"][0, :17000] = 5                       # one token 17,000 times
    c["prompt_len"][0] = 100
    c["bias_token"][0] = torch.arange(400) % 390      # some of them twice, all below 4096
    c["freq"] *= 1e-3
    x, best, lse = expected(c)
    out = torch.full_like(c["logits"], 55.0)
    ws = run(c, out)
    assert lla.device_status(ws) == lla.LLA_OK
    compare(c, x, best, lse, out)


def test_parts_on_their_own():
    """No rule at all, one rule at a time, and outputs one at a time."""
    c = make([6, 2], 3000, "f32", hist=20, max_bias=0, masks=0)
    full = rules_of(c)
    ws = lla.logits_workspace(c["tree"], 3000)
    c["best"].fill_(99)
    lla.logits_adjust(c["tree"], c["token"], c["logits"], lla.LogitRules(), best=c["best"], workspace=ws)
    n = c["start"][-1]
    assert torch.equal(c["best"][:n].long(), c["logits"][:n].argmax(-1))
    out = torch.empty_like(c["logits"])
    lla.logits_adjust(c["tree"], c["token"], c["logits"], lla.LogitRules(), out=out, workspace=ws)
    assert torch.equal(out[:n], c["logits"][:n])
    lla.logits_adjust(c["tree"], c["token"], c["logits"], full, lse=c["lse"], workspace=ws)
    x, _, lse = expected(c)
    assert np.abs(widen(c["lse"])[:n] - lse[:n]).max() <= 1e-5
    # only the path counts where there is no history
    c2 = dict(c, history=torch.zeros(2, 1, dtype=torch.int32), hist_len=torch.zeros(2, dtype=torch.long), prompt_len=torch.zeros(2, dtype=torch.long))
    x, best, lse = expected(c2)
    up = lambda k: c[k].cuda()  # noqa: E731
    lla.logits_adjust(c["tree"], c["token"], c["logits"], lla.LogitRules(repetition=up("rep"), presence=up("pres"), frequency=up("freq")), out=out,
                      best=c["best"], lse=c["lse"], workspace=ws)
    compare(c2, x, best, lse, out)


def test_values_that_are_not_finite():
    """Infinities and NaN: masked ones leave nothing behind, others go into the log-sum-exp and, but for
    NaN, can be best; ties go to the lowest index."""
    V = 9000
    c = make([8], V, "f32", hist=1, max_bias=0, masks=0, branch=1, pad=0)
    inf, nan = math.inf, math.nan
    x = c["logits"]
    x[0, 5], x[0, 8500] = nan, inf
    x[1, 7], x[1, 8000] = inf, inf
    x[2, :] = -inf
    x[3, :] = -inf
    x[3, 8999] = -1e30
    x[4, 100] = nan
    x[5, 4000], x[5, 8000], x[5, 17] = 50.0, 50.0, 49.0
    x[6, :] = nan
    bits = torch.full((1, (V + 31) // 32), -1, dtype=torch.int32, device="cuda")
    bits[0, 5 // 32] &= ~(1 << 5)
    bits[0, 100 // 32] &= ~(1 << (100 % 32))
    bits[0, 8500 // 32] &= ~(1 << (8500 % 32))
    rows = i32([0, -1, -1, -1, -1, -1, -1, 0])
    out = torch.empty_like(x)
    ws = lla.logits_workspace(c["tree"], V)
    lla.logits_adjust(c["tree"], c["token"], x, lla.LogitRules(allowed=bits, allowed_row=rows), out=out, best=c["best"], lse=c["lse"], workspace=ws)
    best, lse = c["best"].tolist(), c["lse"].tolist()
    assert out[0, 5] == -inf and out[0, 8500] == -inf and math.isfinite(lse[0])
    assert best[1] == 7 and lse[1] == inf
    assert best[2] == -1 and lse[2] == -inf
    assert best[3] == 8999 and abs(lse[3] + 1e30) < 1e23
    assert math.isnan(lse[4]) and best[4] != 100 and best[4] >= 0
    assert best[5] == 4000
    assert best[6] == -1 and math.isnan(lse[6])
    assert lla.device_status(ws) == lla.LLA_OK


def test_bad_device_values():
    def base():
        return make([3, 2], 500, "f32", masks=2)

    def flagged(c, **over):
        ws = run(dict(c, **over))
        assert lla.device_status(ws) == lla.LLA_ERR_DEVICE_ARG
        return c

    c = base()
    c["history"][0, 3], c["history"][1, 0] = 500, -1                # tokens outside the vocabulary count nowhere
    out = torch.empty_like(c["logits"])
    x, best, lse = expected(c)
    ws = run(c, out)
    assert lla.device_status(ws) == lla.LLA_ERR_DEVICE_ARG
    compare(c, x, best, lse, out)
    c = base()
    c["token"][1] = 1 << 30
    flagged(c)
    c = base()
    c["hist_len"][0] = 10000
    flagged(c)
    c = base()
    c["prompt_len"][1] = c["hist_len"][1] + 1
    flagged(c)
    c = base()
    c["bias_token"][0, 0] = 500
    flagged(c)
    c = base()
    c["allowed_row"][0] = 2
    x, best, lse = expected(c)
    flagged(c)
    assert int(c["best"][0]) == int(best[0])
    c = base()
    c["tree"].parent[2] = 7
    flagged(c)


def test_logits_replay():
    c = make([9, 4], 20000, "bf16")
    rules, out, ws = rules_of(c), torch.empty_like(c["logits"]), lla.logits_workspace(c["tree"], 20000)
    args = dict(out=out, best=c["best"], lse=c["lse"], workspace=ws)
    lla.logits_adjust(c["tree"], c["token"], c["logits"], rules, **args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lla.logits_adjust(c["tree"], c["token"], c["logits"], rules, **args)
    c["logits"].neg_()
    x, best, lse = expected(c)
    graph.replay()
    torch.cuda.synchronize()
    compare(c, x, best, lse, out)


def test_binding_refusals():
    c = make([3, 2], 500, "f32")
    rules, ws = rules_of(c), lla.logits_workspace(c["tree"], 500)
    x, out = c["logits"], torch.empty_like(c["logits"])
    for bad in (dict(token=c["token"].long()), dict(logits=x.half()), dict(logits=x[:3]), dict(out=out.bfloat16()), dict(out=out[:, :400]),
                dict(logits=x.repeat(1, 2)[:, ::2]), dict(best=c["lse"]), dict(lse=c["best"]), dict(rules=lla.LogitRules(repetition=torch.ones(3).cuda())),
                dict(rules=lla.LogitRules(allowed=torch.zeros(1, 3, dtype=torch.int32).cuda(), allowed_row=c["allowed_row"])),
                dict(rules=lla.LogitRules(allowed=c["allowed"], allowed_row=c["allowed_row"][:2].contiguous())), dict(workspace=None)):
        a = dict(dict(token=c["token"], logits=x, rules=rules, out=out, best=c["best"], lse=c["lse"], workspace=ws), **bad)
        with pytest.raises(ValueError):
            lla.logits_adjust(c["tree"], a.pop("token"), a.pop("logits"), a.pop("rules"), **a)
    for bad in (dict(workspace=ws[:256]), dict(out=None, best=None, lse=None)):
        a = dict(dict(out=out, best=c["best"], lse=c["lse"], workspace=ws), **bad)
        with pytest.raises(lla.LLAError):
            lla.logits_adjust(c["tree"], c["token"], x, rules, **a)


# ------------------------------------------------------------------ acceptance

def accept_case(nodes, branch, tokens, seed=0, pad=2):
    g = torch.Generator().manual_seed(seed + sum(nodes))
    start, parent = forest(nodes, branch, g, pad)
    n = len(parent)
    tree = lla.DraftTree(i32(start), i32(parent), max([1, *nodes]))
    token, chosen = (torch.randint(0, tokens, (n,), generator=g).to(torch.int32).cuda() for _ in range(2))
    ctx = torch.randint(0, 1000, (len(nodes),), generator=g).to(torch.int32).cuda()
    return tree, token, chosen, ctx


def check_accept(tree, token, chosen, ctx, w):
    start, n = tree.tok_start.tolist(), tree.n_tok
    for a in (w.path, w.seq_idx, w.pos):
        assert (a[start[-1]:] == 42).all()
    res = otree.tree_accept(start, tree.parent.tolist(), token.tolist(), chosen.tolist(), ctx.tolist())
    count, nxt, lens = w.count.tolist(), w.next_token.tolist(), w.seq_lens.tolist()
    path, seq, pos = w.path.tolist(), w.seq_idx.tolist(), w.pos.tolist()
    for b, (k, t, L, entries, slots) in enumerate(res):
        s0, s1 = start[b], start[b + 1]
        assert (count[b], nxt[b], lens[b]) == (k, t, L)
        assert path[s0:s1] == entries + [-1] * (s1 - s0 - k) and pos[s0:s1] == slots and seq[s0:s1] == [b] * (s1 - s0)
    assert n == len(path)


@pytest.mark.parametrize("nodes,branch,tokens", [
    ([1], 1, 1), ([8], 1, 1), ([128], 1, 1), ([128, 0, 1, 127], 8, 2), ([0], 1, 1), ([64, 33, 32, 31, 65], 3, 2), ([5] * 700, 2, 2),
    ([16, 9, 3], 16, 3)])
def test_accept(nodes, branch, tokens):
    tree, token, chosen, ctx = accept_case(nodes, branch, tokens)
    w = lla.TreeAccept(tree)
    for a in (w.path, w.seq_idx, w.pos):
        a.fill_(42)
    assert w(token, chosen, ctx) is w
    check_accept(tree, token, chosen, ctx, w)
    assert lla.device_status(w.workspace) == lla.LLA_OK


def test_accept_bad_device_values():
    tree, token, chosen, ctx = accept_case([6, 5], 2, 1)
    tree.parent[3], tree.parent[8], ctx[0] = 3, -4, -7          # roots that are not node 0 are never accepted
    w = lla.TreeAccept(tree)
    for a in (w.path, w.seq_idx, w.pos):
        a.fill_(42)
    w(token, chosen, ctx)
    check_accept(tree, token, chosen, ctx, w)
    assert lla.device_status(w.workspace) == lla.LLA_ERR_DEVICE_ARG
    tree.tok_start[1] = 1 << 20
    w.count.fill_(-9)
    w(token, chosen, ctx)
    assert w.count.tolist() == [0, 0] and w.next_token.tolist() == [-1, -1]


# ------------------------------------------------------------------ the calls together

@pytest.mark.parametrize("page", [0, 16])
def test_a_verification_step(page):
    """Drafted trees through attention, logits, acceptance and encode: what the accepted tokens leave in
    the cache is what a step without drafting would have written, and the next step's attention over
    it agrees with the oracle."""
    import test_tree_gpu as tg
    c = tg.make([50, 17], [7, 5], 2, 96, 160, page, 0, "bf16", T=2, t=1, cap=80)
    if page:        # pages for the new tokens too
        num = c["ck"].shape[0]
        extra = c["table"].shape[0] * c["table"].shape[1]
        grow = lambda x: torch.cat((x, torch.zeros((extra, *x.shape[1:]), dtype=x.dtype, device="cuda")))  # noqa: E731
        c["ck"], c["cv"] = grow(c["ck"]), grow(c["cv"])
        fresh = torch.arange(num, num + extra, dtype=torch.int32, device="cuda").view_as(c["table"])
        c["table"] = torch.where(c["table"] < 0, fresh, c["table"])
    tree = tg.tree_of(c)
    tg.check(c, tg.call(c))
    n, V = sum(c["nodes"]), 700
    g = torch.Generator().manual_seed(5)
    head = torch.randn(2 * 128, V, generator=g).cuda()
    logits = (c["out"][:, :2].float().flatten(1) @ head).nan_to_num()
    token = torch.randint(0, V, (tree.n_tok,), generator=g).to(torch.int32).cuda()
    best = torch.zeros(tree.n_tok, dtype=torch.int32, device="cuda")
    rules = lla.LogitRules(repetition=torch.full((2,), 1.3, device="cuda"))
    lws = lla.logits_workspace(tree, V)
    lla.logits_adjust(tree, token, logits, rules, best=best, workspace=lws)
    # the draft guessed right along the last node's path of the first sequence, once in the second
    par = c["parent"].tolist()
    for i in reversed(otree.path_of(par[:7], 6)[:-1]):
        token[i] = best[par[i]]
        lla.logits_adjust(tree, token, logits, rules, best=best, workspace=lws)
    token[7 + 1] = best[7]
    lla.logits_adjust(tree, token, logits, rules, best=best, workspace=lws)
    walk = lla.TreeAccept(tree)(token, best, c["seq_lens"])
    res = otree.tree_accept(c["tok_start"].tolist(), par, token.tolist(), best.tolist(), c["lens"])
    assert walk.count.tolist() == [r[0] for r in res] and walk.count.tolist()[0] >= len(otree.path_of(par[:7], 6))
    # encode all nodes at the slots that the walk gave them
    dm, H, T = c["dm"], 2, 2
    x_k, x_v = (torch.randn(n, H, T * 128, generator=g).bfloat16().cuda() for _ in range(2))
    wd_k, wd_v = (torch.randn(H, T * 128, r, generator=g).div(16).bfloat16().cuda() for r in (96, 160))
    seq, pos = walk.seq_idx[:n].contiguous(), walk.pos[:n].contiguous()
    if page:
        ws = lla.make_workspace(dm, 2, c["cap"], n)
        lla.encode_paged(dm, x_k, x_v, seq, pos, wd_k, wd_v, c["mk"], c["mv"], c["ck"], c["cv"], c["table"], page, ws)
    else:
        ws = lla.make_workspace(dm, 2, c["cap"], n)
        lla.encode(dm, x_k, x_v, seq, pos, wd_k, wd_v, c["mk"], c["mv"], c["ck"], c["cv"], ws)
    assert lla.device_status(ws) == lla.LLA_OK
    lat = (x_k.double() - c["mk"].double()).transpose(0, 1) @ wd_k.double()          # [H][n][r_k]
    for b in range(2):
        for r, e in enumerate(res[b][3]):
            j = c["lens"][b] + r
            row = c["ck"][b, :, j] if not page else c["ck"][int(c["table"][b, j // page]), :, j % page]
            assert (row.double() - lat[:, e]).abs().max() <= 2.0 ** -8 * lat[:, e].abs().max() + 1e-3
    # the next step: one new node a sequence behind the accepted ones
    c["lens"], c["nodes"], c["max_nodes"] = walk.seq_lens.tolist(), [1, 1], 1
    c["seq_lens"] = walk.seq_lens.clone()
    c["tok_start"], c["parent"], c["pos"] = i32([0, 1, 2]), i32([-1, -1]), walk.seq_lens.clone()
    c["qkv"], c["out"], c["lse"] = c["qkv"][:2].contiguous(), c["out"][:2].contiguous(), c["lse"][:2].contiguous()
    tg.check(c, tg.call(c))


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("own_stream", [False, True])
def test_all_entries_of_a_step_go_to_encode(captured, own_stream):
    """Steps of fewer and fewer nodes over the same arrays, all entries handed on to lla_encode: only the slots of the
    step's own nodes are written, though the host never knows how many there are."""
    import test_tree_gpu as tg
    c = tg.make([20, 9], [6, 5], 2, 16, 16, 0, 0, "bf16", cap=60, pad=4)
    tree, n_tok, T = tg.tree_of(c), c["parent"].shape[0], 2
    dirty = [torch.zeros(n_tok, dtype=torch.int32, device="cuda") for _ in range(8)]
    del dirty                                        # (memory that new tensors take over holds zeros, a slot)
    walk = lla.TreeAccept(tree, clear=True)
    assert (walk.seq_idx == -1).all() and (lla.TreeAccept(tree).seq_idx == -1).all()
    g = torch.Generator().manual_seed(3)
    x = [torch.randn(n_tok, 2, T * 128, generator=g).bfloat16().cuda() for _ in range(2)]
    wd = [torch.randn(2, T * 128, 16, generator=g).div(16).bfloat16().cuda() for _ in range(2)]
    token, chosen = (torch.zeros(n_tok, dtype=torch.int32, device="cuda") for _ in range(2))
    ctx, ws = c["seq_lens"].clone(), lla.make_workspace(c["dm"], 2, 60, n_tok)
    stream = torch.cuda.Stream() if own_stream else None
    torch.cuda.synchronize()

    def step(s):
        walk(token, chosen, ctx, stream=s)
        lla.encode(c["dm"], *x, walk.seq_idx, walk.pos, *wd, c["mk"], c["mv"], c["ck"], c["cv"], ws, stream=s)

    graph = None
    if captured:
        step(stream)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step(None)
    for sizes in ([6, 5], [2, 3], [0, 1], [0, 0], [1, 0]):
        tree.tok_start.copy_(i32([0, sizes[0], sum(sizes)]))
        c["ck"].fill_(float("nan")), c["cv"].fill_(float("nan"))
        torch.cuda.synchronize()
        if graph is not None:
            graph.replay()
        else:
            step(stream)
        torch.cuda.synchronize()
        for b, L in enumerate(ctx.tolist()):
            there = torch.isfinite(c["ck"][b, 0, :, 0].float()).nonzero().flatten().tolist()
            assert there == list(range(L, L + sizes[b]))
    for part in (walk.path, walk.seq_idx, walk.pos):
        assert (part[1:] == -1).all()
