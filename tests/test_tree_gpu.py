"""lla_tree_attn and lla_tree_attn_paged against the 64-bit oracle.

Cache rows that hold no token of a call, and entries that belong to no sequence, are NaN: a result
that touched one shows it.  Tolerances: fp32 storage 1e-5 of the largest value of an output
vector, as everywhere; bf16 storage the oracle's bound of the roundings to bf16 (six standard
deviations) and half a step of the result, 2^-8 of its value."""
import numpy as np
import pytest
import torch

from lla_cases import widen
from looped_transformer_cross_gb300 import lla
from oracle import tree as otree

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from looped_transformer_cross_gb300 import build
    build.build()


def make(lens, nodes, H, rk, rv, page=0, style=0, dtype="bf16", branch=2, T=2, t=1, seed=0, pad=3, device="cuda", scale=1.0,
         fused=True, roots=False, cap=None):
    """A call's tensors: sequences of the given cached lengths and node counts."""
    g = torch.Generator().manual_seed(1000 * seed + 7 * rk + rv + sum(lens) + 31 * sum(nodes))
    sd = torch.bfloat16 if dtype == "bf16" else torch.float32
    rnd = lambda std, *s: torch.randn(*s, generator=g) * std  # noqa: E731
    B, n = len(lens), sum(nodes)
    parent, pos = [], []
    for L, m in zip(lens, nodes):
        depth = []
        for i in range(m):
            p = -1 if i == 0 or (roots and i % 5 == 4) else max(0, i - 1 - int(torch.randint(0, branch, (1,), generator=g)))
            depth.append(0 if p < 0 else depth[p] + 1)
            parent.append(p)
            pos.append(L + depth[-1])
    c = dict(H=H, T=T, t=t, style=style, page=page, lens=list(lens), nodes=list(nodes), dtype=dtype)
    c["dm"] = lla.dims(T, H, rk, rv, dtype=lla.LLA_BF16 if dtype == "bf16" else lla.LLA_F32, rope_style=style)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=device)  # noqa: E731
    c["tok_start"] = i32([0] + list(np.cumsum(nodes)))
    c["parent"], c["pos"] = i32(parent + [-1] * pad), i32(pos + [0] * pad)
    c["seq_lens"] = i32(list(lens))
    qkv = rnd(scale, n + pad, 3 * H, D).to(sd)
    qkv[n:] = float("nan")
    c["qkv"] = qkv.to(device)
    cap = max([1, *lens]) if cap is None else cap
    if page == 0:
        ck, cv = rnd(1.0, B, H, cap, rk).to(sd), rnd(1.0, B, H, cap, rv).to(sd)
        for b, L in enumerate(lens):
            ck[b, :, L:], cv[b, :, L:] = float("nan"), float("nan")
    else:
        mp = (cap + page - 1) // page
        held = [(L + page - 1) // page for L in lens]
        num = sum(held) + 2
        ck, cv = rnd(1.0, num, H, page, rk).to(sd), rnd(1.0, num, H, page, rv).to(sd)
        perm, used = torch.randperm(num, generator=g).tolist(), 0
        table = np.full((B, mp), -7, np.int32)
        for b, L in enumerate(lens):
            table[b, :held[b]] = perm[used:used + held[b]]
            used += held[b]
            if L % page:
                ck[table[b, held[b] - 1], :, L % page:] = float("nan")
                cv[table[b, held[b] - 1], :, L % page:] = float("nan")
        for p in perm[used:]:
            ck[p], cv[p] = float("nan"), float("nan")
        c["table"] = torch.from_numpy(table).to(device)
        cap = mp * page
    c["cap"], c["ck"], c["cv"] = cap, ck.to(device), cv.to(device)
    c["wk"], c["wv"] = rnd(rk ** -0.5, T, H, D, rk).to(sd).to(device), rnd(rv ** -0.5, T, H, D, rv).to(sd).to(device)
    c["mk"], c["mv"] = rnd(0.3, H, T * D).to(device), rnd(0.3, H, T * D).to(device)
    ang = torch.arange(max(128, cap + 130), dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * torch.arange(64, dtype=torch.float64) / D)
    c["cos"], c["sin"] = ang.cos().float().to(device), ang.sin().float().to(device)
    c["max_nodes"] = max([1, *nodes])
    c["out"] = torch.full((n + pad, H, D), 77.0, dtype=sd, device=device)
    c["lse"] = torch.full((n + pad, H), 77.0, device=device)
    return c


def tree_of(c, max_nodes=None):
    return lla.DraftTree(c["tok_start"], c["parent"], c["max_nodes"] if max_nodes is None else max_nodes, pos=c["pos"])


def call(c, ws=None, tree=None, out="out", lse="lse", stream=None):
    tree = tree_of(c) if tree is None else tree
    ws = lla.tree_workspace(c["dm"], tree, c["cap"]) if ws is None else ws
    H = c["H"]
    q, k, v = (c["qkv"][:, i * H:(i + 1) * H] for i in range(3))
    rest = (c["seq_lens"], c["wk"], c["wv"], c["mk"], c["mv"], c["cos"], c["sin"], c[out], None if lse is None else c[lse], ws)
    if c["page"]:
        lla.tree_attn_paged(c["dm"], c["t"], tree, q, k, v, c["ck"], c["cv"], c["table"], c["page"], *rest, stream=stream)
    else:
        lla.tree_attn(c["dm"], c["t"], tree, q, k, v, c["ck"], c["cv"], *rest, stream=stream)
    return ws


def want(c):
    ck, cv = widen(c["ck"]), widen(c["cv"])

    def latents(b, h):
        L, P = c["lens"][b], c["page"]
        if not P:
            return ck[b, h, :L], cv[b, h, :L]
        pages = c["table"][b, :(L + P - 1) // P].tolist()
        return tuple(np.concatenate([x[p, h] for p in pages] + [np.zeros((0, x.shape[3]))])[:L] for x in (ck, cv))

    H, t = c["H"], c["t"]
    qkv = widen(c["qkv"])
    sl = slice(t * D, (t + 1) * D)
    return otree.tree_attn(qkv[:, :H], qkv[:, H:2 * H], qkv[:, 2 * H:], c["tok_start"].tolist(), c["parent"].tolist(), c["pos"].tolist(),
                           latents, widen(c["wk"])[t], widen(c["wv"])[t], widen(c["mk"])[:, sl], widen(c["mv"])[:, sl],
                           widen(c["cos"]), widen(c["sin"]), c["style"])


def check(c, ws, lse=True):
    assert lla.device_status(ws) == lla.LLA_OK
    o, s, tol, tol_s = want(c)
    n = sum(c["nodes"])
    got, got_s = widen(c["out"]), widen(c["lse"])
    top = np.abs(o[:n]).max(-1, keepdims=True) if n else np.zeros((0, c["H"], 1))
    if c["dtype"] == "f32":
        tol, tol_s = 1e-5 * top, np.full_like(s[:n], 1e-5)
    else:
        # (fp32 sums, and what a bound to first order leaves out: 1e-4 of the largest value)
        tol, tol_s = tol[:n] + 2.0 ** -8 * np.abs(o[:n]) + 1e-4 * top, tol_s[:n] + 1e-4
    err = np.abs(got[:n] - o[:n])
    assert np.isfinite(got[:n]).all() and (err <= tol).all(), float((err / tol).max())
    if lse:
        assert (np.abs(got_s[:n] - s[:n]) <= tol_s).all(), float((np.abs(got_s[:n] - s[:n]) / tol_s).max())
    assert (got[n:] == 77.0).all() and (got_s[n:] == 77.0).all()


CASES = [
    # lens, nodes, H, r_k, r_v, page
    ([1], [1], 1, 16, 16, 0),
    ([0], [1], 2, 96, 160, 0),
    ([0, 130, 0], [3, 0, 0], 1, 96, 160, 0),
    ([127, 128, 129], [1, 2, 3], 2, 96, 160, 0),
    ([300, 7, 0, 256], [9, 16, 5, 0], 3, 96, 160, 0),
    ([513], [33], 2, 64, 128, 0),
    ([260, 90], [64, 31], 2, 96, 160, 64),
    ([385], [128], 1, 96, 160, 0),
    ([200, 70], [65, 127], 1, 32, 64, 16),
    ([700, 3, 511], [4, 8, 2], 4, 16, 32, 0),
    ([700, 3, 511], [4, 8, 2], 4, 16, 32, 8),
    ([257, 100], [7, 5], 2, 16, 32, 32),
    ([150, 49], [5, 6], 2, 96, 160, 24),
    ([150, 49], [5, 6], 2, 96, 160, 1),
    ([301, 64], [5, 6], 2, 96, 160, 100),
    ([301, 600], [17, 6], 2, 96, 160, 128),
    ([301, 600], [17, 6], 2, 80, 48, 256),
    ([500, 131], [9, 40], 2, 96, 160, 48),
    ([500, 131], [9, 40], 2, 80, 112, 40),
    ([333, 260], [70, 3], 3, 64, 80, 192),
    ([333, 260], [70, 3], 3, 48, 128, 6),
    ([700, 20], [5, 31], 2, 192, 192, 2),
    ([513, 256], [100, 64], 2, 16, 240, 20),
    ([301], [40], 2, 112, 112, 0),
    ([140], [6], 2, 256, 256, 0),
    ([140], [6], 1, 240, 16, 64),
    ([129], [12], 2, 16, 256, 0),
    ([2100], [10], 3, 128, 208, 0),
    ([1300, 1, 40], [3, 20, 50], 5, 48, 80, 0),
]


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("lens,nodes,H,rk,rv,page", CASES)
def test_tree_attn_bf16(lens, nodes, H, rk, rv, page, style):
    c = make(lens, nodes, H, rk, rv, page, style, "bf16")
    check(c, call(c))


@pytest.mark.parametrize("lens,nodes,H,rk,rv,page", CASES)
def test_tree_attn_f32(lens, nodes, H, rk, rv, page):
    c = make(lens, nodes, H, rk, rv, page, len(lens) % 2, "f32")
    check(c, call(c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("branch,roots", [(1, False), (8, False), (2, True)])
def test_tree_shapes(dtype, branch, roots):
    """Chains, bushy trees and forests."""
    c = make([130, 20, 0], [20, 33, 64], 2, 96, 160, 0, 0, dtype, branch=branch, roots=roots)
    check(c, call(c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences_and_long_ones(dtype):
    """More units than multiprocessors, lengths far apart, none of a unit's tiles in one block only."""
    lens = [5000, 1, 0, 127, 640, 130] + [100] * 30
    c = make(lens, [3, 1, 2, 4, 1, 0] + [2] * 30, 6, 32, 64, 0, 0, dtype)
    check(c, call(c))


def test_large_scores():
    """Queries and keys of 4 standard deviations: weights far apart, a running maximum that rises."""
    c = make([900], [12], 2, 96, 160, 0, 0, "f32", scale=4.0)
    check(c, call(c))
    c = make([900], [12], 2, 96, 160, 0, 0, "bf16", scale=4.0)
    check(c, call(c))


@pytest.mark.parametrize("n", [3, 20, 50, 100])
def test_scores_that_rise(n):
    """Latents that grow along the cache: scores 2^30 and more above the first tile's, twice, and
    falling again (a reference taken early has to move, and the sums with it)."""
    c = make([700, 380, 129], [n, 1, 2], 2, 96, 160, 0, 0, "bf16", scale=12.0)
    c["ck"][:, :, :128] *= 0.05
    c["ck"][:, :, 128:256] *= 0.5
    c["ck"][:, :, 400:] *= 0.1
    check(c, call(c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_lse_and_on_another_stream(dtype):
    c = make([300, 40], [4, 9], 2, 96, 160, 64, 0, dtype)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = lla.tree_workspace(c["dm"], tree_of(c), c["cap"])
    torch.cuda.synchronize()
    call(c, ws, lse=None, stream=s)
    s.synchronize()
    check(c, ws, lse=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_separate_tensors_and_room_for_more_nodes(dtype):
    """q, k, v as tensors of their own; max_nodes above what any sequence has."""
    c = make([300, 40], [4, 9], 2, 96, 160, 0, 0, dtype)
    tree = tree_of(c, 100)
    ws = lla.tree_workspace(c["dm"], tree, c["cap"])
    q, k, v = (c["qkv"][:, 2 * i:2 * i + 2].contiguous() for i in range(3))
    lla.tree_attn(c["dm"], c["t"], tree, q, k, v, c["ck"], c["cv"], c["seq_lens"], c["wk"], c["wv"], c["mk"], c["mv"], c["cos"], c["sin"],
                  c["out"], c["lse"], ws)
    check(c, ws)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_repeats_bit_for_bit_and_replays(dtype):
    """The same call gives the same bits, and so does a captured graph after its inputs changed."""
    c = make([700, 333], [20, 5], 3, 96, 160, 64, 0, dtype)
    ws = call(c)
    first = c["out"].clone()
    call(c, ws)
    assert torch.equal(first, c["out"])
    tree = tree_of(c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(c, ws, tree)
    c["qkv"].neg_()
    c["seq_lens"] -= 1
    c["pos"] -= 1
    c["lens"] = [x - 1 for x in c["lens"]]
    c["out"].fill_(77.0)
    c["lse"].fill_(77.0)
    graph.replay()
    torch.cuda.synchronize()
    check(c, ws)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_device_values(dtype):
    """Values that the host cannot see: recorded, and read as the documentation says."""
    base = lambda: make([200, 100], [5, 4], 2, 96, 160, 64, 0, dtype)  # noqa: E731

    def flagged(c, ws):
        assert lla.device_status(ws) == lla.LLA_ERR_DEVICE_ARG
        return ws

    c = base()                                       # a parent that does not come before its node: a root
    c["parent"][2] = 2
    c["parent"][7] = -3
    check(c, flagged(c, call(c)))
    c = base()                                       # a sequence with more nodes than there is room for: none
    n0 = c["nodes"][0]
    ws = flagged(c, call(c, tree=tree_of(c, 4)))
    assert (c["out"][:n0] == 77.0).all() and torch.isfinite(c["out"][n0:9].float()).all()
    c = base()                                       # starts that descend, or leave the array
    c["tok_start"][1] = 50
    ws = flagged(c, call(c))
    assert (c["out"] == 77.0).all()
    c = base()                                       # lengths and positions out of range: clamped
    c["seq_lens"][0], c["pos"][6] = -1, 1 << 30
    ws = call(c)
    flagged(c, ws)
    c["lens"][0] = 0
    c["pos"][6] = c["cos"].shape[0] - 1
    check(c, ws)
    c = base()                                       # a page outside the pool: read as one inside, flagged
    c["table"][1, 0] = 1 << 20
    flagged(c, call(c))
    assert torch.isfinite(c["out"][:5].float()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_pages(dtype):
    """Two sequences whose tables name the same pages (a shared prefix)."""
    c = make([128, 128], [3, 4], 2, 96, 160, 64, 0, dtype)
    c["table"][1] = c["table"][0]
    check(c, call(c))


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("lens,nodes,rk,rv,page", [([300, 7, 0, 129], [9, 3, 4, 1], 96, 160, 0), ([200, 140], [40, 128], 64, 128, 24),
                                                   ([130, 33], [20, 2], 16, 240, 64)])
def test_keys_beyond_half_precision(lens, nodes, rk, rv, page, style):
    """Cached keys with components up to 1e6 (and some tokens' far below), queries small enough that the scores
    are ordinary ones."""
    c = make(lens, nodes, 2, rk, rv, page, style, "bf16")
    c["ck"].mul_(2.0 ** 18)
    c["wk"][:, :, :64].mul_(2.0 ** -3)
    c["mk"].mul_(2.0 ** 10)
    c["qkv"][:, :2].mul_(2.0 ** -18)
    ws = call(c)
    check(c, ws)
    assert np.abs(widen(c["ck"])[np.isfinite(widen(c["ck"]))]).max() > 65504


@pytest.mark.parametrize("scale", [2.0 ** -20, 2.0 ** -6, 2.0 ** 12])
def test_log_sum_exp_is_as_exact_as_fp32(scale):
    """bf16 storage, the log-sum-exp of fp32 arithmetic: keys and queries of 22 bits (scores up to 6 with an
    error of 6 * 2^-20), weights of 16 (2^-17 of a sum each, independent); key sizes far from 1, the queries'
    the other way."""
    for lens, nodes in (([1, 2, 5, 0], [1, 3, 2, 4]), ([130, 700], [16, 2]), ([260], [33]), ([140, 90], [128, 65])):
        c = make(lens, nodes, 2, 96, 160, 0, 0, "bf16")
        if scale != 1.0:
            c["wk"].mul_(scale), c["mk"].mul_(scale)
            c["qkv"][:, :2].div_(scale)
            c["qkv"][:, 2:4].mul_(scale)
        ws = call(c)
        check(c, ws)
        o, s, _, _ = want(c)
        n = sum(nodes)
        assert np.abs(widen(c["lse"])[:n] - s[:n]).max() <= 2e-5


@pytest.mark.parametrize("nodes", [3, 20, 64])
def test_keys_that_grow(nodes):
    """Cached keys that grow 2^18-fold after the first 128 tokens."""
    c = make([400, 129, 128], [nodes, 2, 1], 2, 96, 160, 0, 0, "bf16")
    c["ck"][:, :, :128].mul_(2.0 ** -18)
    c["mk"].mul_(2.0 ** -18)
    check(c, call(c))


@pytest.mark.parametrize("nodes,page,style", [(3, 0, 0), (40, 24, 1), (128, 64, 0)])
def test_latents_far_above_their_weights(nodes, page, style):
    """Latents of 2^26 in one of three sequences: its keys leave the range that their weights suggest."""
    c = make([300, 150, 77], [5, nodes, 2], 2, 96, 160, page, style, "bf16")
    if page:
        used = c["table"][1, :(150 + page - 1) // page].long()
        c["ck"][used] *= 2.0 ** 26
    else:
        c["ck"][1] *= 2.0 ** 26
    c["qkv"][5:5 + nodes, :2] *= 2.0 ** -26
    check(c, call(c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_in_one_sequence(dtype):
    """A NaN among a sequence's cached latents makes its own results NaN and no other's."""
    c = make([300, 150, 77], [5, 20, 2], 2, 96, 160, 0, 0, dtype)
    c["ck"][1, :, 70, 3] = float("nan")
    ws = call(c)
    assert lla.device_status(ws) == lla.LLA_OK
    assert torch.isnan(c["out"][5:25].float()).all() and torch.isnan(c["lse"][5:25]).all()
    o, s, tol, tol_s = want(c)
    keep = [*range(5), 25, 26]
    err = np.abs(widen(c["out"])[keep] - o[keep])
    assert (err <= tol[keep] + 2.0 ** -8 * np.abs(o[keep]) + 1e-4 * np.abs(o[keep]).max()).all()
    assert (np.abs(widen(c["lse"])[keep] - s[keep]) <= 2e-5).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("L", [0, 200])
def test_nan_and_infinity_off_the_path(dtype, what, L):
    """A node's key and value that are not finite reach the nodes below it and no others, and a query its own node."""
    c = make([L, L], [40, 9], 2, 96, 160, 0, 0, dtype)
    parent = c["parent"].tolist()
    for node, part in ((7, 1), (30, 2), (12, 0)):
        c["qkv"][node, 2 * part:2 * part + 2, 5] = what
    below = set()
    for i in range(40):
        if any(a in (7, 30) for a in otree.path_of(parent[:40], i)) or i == 12:
            below.add(i)
    ws = call(c)
    assert lla.device_status(ws) == lla.LLA_OK
    c["qkv"] = torch.nan_to_num(c["qkv"], 0.0, 0.0, 0.0)
    o, s, tol, tol_s = want(c)
    keep = [i for i in range(49) if i not in below]
    assert len(keep) >= 10
    err = np.abs(widen(c["out"])[keep] - o[keep])
    assert (err <= (0 if dtype == "f32" else tol[keep] + 2.0 ** -8 * np.abs(o[keep])) + 1e-4 * np.abs(o[keep]).max()).all()
    assert (np.abs(widen(c["lse"])[keep] - s[keep]) <= 2e-5).all()
    got = c["out"].float()
    if what == what:
        # an infinite value: infinite in its component where the weights are above 0, finite in the others
        chain = [i for i in range(40) if 30 in otree.path_of(parent[:40], i) and 7 not in otree.path_of(parent[:40], i) and i != 12]
        assert (got[chain][:, :, 5] == what).all() and torch.isfinite(got[chain][:, :, 6:]).all() if chain else True
    else:
        assert torch.isnan(got[30, :, 5]).all() and torch.isnan(got[12]).all()


@pytest.mark.parametrize("lens,nodes,rk,rv,page", [([300, 7, 0, 129], [9, 3, 4, 1], 96, 160, 0), ([700, 140], [40, 128], 64, 128, 24),
                                                   ([130, 1300], [20, 30], 16, 240, 64), ([2, 1, 5], [1, 2, 16], 192, 192, 1)])
def test_out_is_rounded_once(lens, nodes, rk, rv, page):
    """bf16 storage: an output is off by half a step of its own, 2^-8 of its value, and by what parts of 16
    bits leave out: weights and latent sums 2^-17 each, weights by scores of up to 8 with 22 bits 2^-18 more:
    2^-15 of a sum of |p v| of up to twice the largest value, taken as 2^-14 of that value."""
    c = make(lens, nodes, 2, rk, rv, page, 0, "bf16")
    ws = call(c)
    assert lla.device_status(ws) == lla.LLA_OK
    o = want(c)[0]
    n = sum(nodes)
    err = np.abs(widen(c["out"])[:n] - o[:n])
    tol = 2.0 ** -8 * np.abs(o[:n]) + 2.0 ** -14 * np.abs(o[:n]).max(-1, keepdims=True)
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_streams_at_once(dtype):
    """Calls on two streams with a workspace each, under way together."""
    cases = [make([900, 333], [20, 5], 3, 96, 160, 64, 0, dtype), make([500, 40, 77], [64, 1, 9], 2, 32, 64, 0, 1, dtype)]
    streams = [torch.cuda.Stream() for _ in cases]
    spaces = [lla.tree_workspace(c["dm"], tree_of(c), c["cap"]) for c in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, ws in zip(cases, streams, spaces):
            call(c, ws, stream=s)
    torch.cuda.synchronize()
    for c, ws in zip(cases, spaces):
        check(c, ws)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_graphs_that_share_a_workspace(dtype):
    """Two captured calls of different shapes over one workspace, whose contents are whatever was there before."""
    cases = [make([900, 333], [20, 5], 3, 96, 160, 64, 0, dtype), make([500, 40, 77], [64, 1, 9], 2, 32, 64, 0, 1, dtype)]
    trees = [tree_of(c) for c in cases]
    size = max(lla.tree_workspace(c["dm"], t, c["cap"]).numel() for c, t in zip(cases, trees))
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    ws[:256] = 0
    graphs = []
    for c, t in zip(cases, trees):
        call(c, ws, t)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(c, ws, t)
    for _ in range(3):
        for c, g in zip(cases, graphs):
            c["out"].fill_(77.0), c["lse"].fill_(77.0)
            g.replay()
    torch.cuda.synchronize()
    for c in cases:
        check(c, ws)


@pytest.mark.parametrize("dtype,page", [("bf16", 64), ("bf16", 12), ("f32", 64)])
def test_pages_far_into_a_pool(dtype, page):
    """Pages whose elements lie beyond 2^32 in their pools."""
    c = make([150, 70], [3, 6], 16, 96, 160, page, 0, dtype)
    num = (1 << 32) // (16 * page * 96) + 50
    if torch.cuda.mem_get_info()[0] < 2 * num * 16 * page * 256 * c["ck"].element_size():
        pytest.skip("not enough memory")
    for name in ("ck", "cv"):
        small = c[name]
        c[name] = torch.empty((num, *small.shape[1:]), dtype=small.dtype, device="cuda")
        c[name][num - small.shape[0]:] = small
    small = {k: c[k][num - len(small):].clone() for k in ("ck", "cv")}
    table = c["table"].clone()
    c["table"] = torch.where(table >= 0, table + (num - len(small["ck"])), table)
    ws = call(c)
    c.update(small, table=table)
    check(c, ws)


def test_tree_binding_refusals():
    c = make([40, 20], [4, 3], 2, 96, 160, 0, 0, "bf16")
    ws = lla.tree_workspace(c["dm"], tree_of(c), c["cap"])
    good = dict(c)

    def refused(error, **over):
        bad = dict(good, **over)
        with pytest.raises(error):
            call(bad, over.get("ws", ws), over.get("tree"))

    refused(ValueError, qkv=good["qkv"].float())
    refused(ValueError, qkv=good["qkv"][:-1])
    refused(ValueError, qkv=good["qkv"].cpu())
    refused(ValueError, ck=good["ck"][:1])
    refused(ValueError, ck=good["ck"].transpose(1, 2))
    refused(ValueError, seq_lens=good["seq_lens"].long())
    refused(ValueError, wk=good["wk"][:1])
    refused(ValueError, mk=good["mk"].bfloat16())
    refused(ValueError, cos=good["cos"][:, :32].contiguous())
    refused(ValueError, sin=good["sin"][:-1])
    refused(ValueError, out=good["out"].float())
    refused(ValueError, lse=good["lse"][:-1])
    refused(ValueError, tree=lla.DraftTree(good["tok_start"], good["parent"], 4))              # no positions
    refused(ValueError, tree=lla.DraftTree(good["tok_start"][:2].contiguous(), good["parent"], 4, pos=good["pos"]))
    refused(lla.LLAError, ws=ws[:-4096].contiguous())
    refused(lla.LLAError, out=good["qkv"].view(-1)[:good["out"].numel()].view(good["out"].shape))     # over its inputs
    with pytest.raises(ValueError):
        lla.DraftTree(good["tok_start"], good["parent"], lla.LLA_TREE_MAX_NODES + 1, pos=good["pos"])
    call(c, ws)
    check(c, ws)


def test_many_sequences_without_work():
    """Long runs of sequences without nodes or without cached tokens between others."""
    lens, nodes = [0] * 200, [0] * 200
    for b, L, n in ((3, 300, 2), (4, 90, 0), (70, 129, 3), (140, 0, 4), (199, 260, 1)):
        lens[b], nodes[b] = L, n
    c = make(lens, nodes, 2, 32, 64, 0, 0, "bf16")
    check(c, call(c))


def _half_step(o):
    """Half a step of bf16 at values o."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(o), 1e-30))) - 8)


def test_drafted_weights_are_not_rounded():
    """bf16 storage, two nodes and no cached tokens, scores that keys and queries of 22 bits give exactly but for
    2^-22 of at most 0.4: an output is off by half a step and, relative to the sum of |p v|, by the exponential's two units
    (2^-22), the score (2^-24), three products' sums (2^-23 each), sum, division and scaling (2^-24 each): below 2^-20."""
    B, H = 256, 16
    c = make([0] * B, [2] * B, H, 16, 16, dtype="bf16", pad=0, branch=1)
    c["pos"].zero_()
    c["qkv"][:, :2 * H, 1:] = 0.0
    c["qkv"][:, :H, 0] = 1.0
    ws = call(c)
    assert lla.device_status(ws) == lla.LLA_OK
    x = widen(c["qkv"]).reshape(B, 2, 3, H, D)
    s = x[:, :, 1, :, 0] / np.sqrt(D)
    p = np.exp(s - s.max(1, keepdims=True))[..., None]
    o, mass = (p * x[:, :, 2]).sum(1) / p.sum(1), (p * np.abs(x[:, :, 2])).sum(1) / p.sum(1)
    err = np.abs(widen(c["out"]).reshape(B, 2, H, D)[:, 1] - o)
    assert (err <= _half_step(o) + 2.0 ** -20 * mass).all(), int((err > _half_step(o) + 2.0 ** -20 * mass).sum())


@pytest.mark.parametrize("nodes,page", [(1, 0), (20, 24), (40, 0)])
def test_latent_sums_are_not_rounded(nodes, page):
    """bf16 storage, equal weights (queries of 0) and latents of one component: out = W sum(c) / l, where the sum, in
    24 bits, is off by 2^-24 a cached token, and three products' sums (2^-23 each), division and scaling (2^-24 each) follow:
    below 2^-20 of the value, beside half a step."""
    B, H, L = 64, 16, 5
    c = make([L] * B, [nodes] * B, H, 16, 32, page, dtype="bf16", pad=0, branch=1)
    c["qkv"][:, :H] = 0.0
    c["qkv"][:, 2 * H:] = 0.0
    c["mv"].zero_()
    c["cv"].nan_to_num_(0.0)
    c["cv"][..., :3] = 0.0
    c["cv"][..., 4:] = 0.0
    c["cv"] *= (2.0 ** (-3.0 * torch.arange(c["cv"].shape[2], device="cuda")))[:, None].bfloat16()     # (sums of 20 bits)
    ws = call(c)
    assert lla.device_status(ws) == lla.LLA_OK
    cv = widen(c["cv"])[..., 3]
    total = cv[:, :, :L].sum(-1) if not page else cv[c["table"][:, 0].cpu().numpy()][:, :, :L].sum(-1)      # [B][H]
    got = widen(c["out"]).reshape(B, nodes, H, D)
    depth = np.arange(1, nodes + 1)[None, :, None, None]                                               # (chains)
    o = total[:, None, :, None] * widen(c["wv"])[c["t"]][None, None, :, :, 3] / (L + depth)
    err, tol = np.abs(got - o), _half_step(o) + 2.0 ** -20 * np.abs(o)
    assert (err <= tol).all(), int((err > tol).sum())


@pytest.mark.parametrize("nodes,B,std", [(64, 10, 1.0), (64, 10, 3.0), (128, 5, 1.0), (24, 10, 1.0), (10, 10, 3.0)])
def test_long_sums(nodes, B, std):
    """65536 cached tokens, a unit's in one block's sums, values that do not cancel.  The log-sum-exp as exact as fp32 makes
    it (2e-5: scores of up to 15 with 22 bits, 2^-18, and sums cut off for 64 steps, 2^-17); outputs off by half a step
    and by sums cut off for 512 steps of 2^-23 (2^-14 of the sum, all its terms being positive), parts of 16 bits and those scores."""
    H, L, rk, rv = 16, 65536, 16, 32
    g = torch.Generator(device="cuda").manual_seed(nodes)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    dm, n = lla.dims(1, H, rk, rv), B * nodes
    qkv = rnd(n, 3 * H, D).bfloat16()
    qkv[:, :H] *= std
    ck, cv = rnd(B, H, L, rk).bfloat16(), (1 + 0.1 * rnd(B, H, L, rv)).bfloat16()
    wk, wv = (rnd(1, H, D, rk) / 4).bfloat16(), (rnd(1, H, D, rv).abs() / 6).bfloat16()
    zero = torch.zeros(H, D, device="cuda")
    ang = torch.arange(L + 1, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-2.0 * torch.arange(64, dtype=torch.float64, device="cuda") / D)
    cos, sin = ang.cos().float(), ang.sin().float()
    tree = lla.DraftTree(i32([nodes * b for b in range(B + 1)]), i32([-1] * n), nodes, pos=i32([L] * n))
    out, lse = torch.zeros(n, H, D, device="cuda", dtype=torch.bfloat16), torch.zeros(n, H, device="cuda")
    ws = lla.tree_workspace(dm, tree, L)
    lla.tree_attn(dm, 0, tree, qkv[:, :H], qkv[:, H:2 * H], qkv[:, 2 * H:], ck, cv, i32([L] * B), wk, wv, zero, zero, cos, sin, out, lse, ws)
    assert lla.device_status(ws) == lla.LLA_OK
    turn = lambda x, at: torch.cat((x[..., :64] * cos[at].double() - x[..., 64:] * sin[at].double(),  # noqa: E731
                                    x[..., :64] * sin[at].double() + x[..., 64:] * cos[at].double()), -1)
    for b, h in ((0, 0), (B // 2, 7), (B - 1, 15)):
        own = slice(b * nodes, (b + 1) * nodes)
        q, kd = turn(qkv[own, h].double(), L), turn(qkv[own, H + h].double(), L)
        k = turn(ck[b, h].double() @ wk[0, h].double().T, slice(0, L))
        s = torch.cat((q @ k.T, (q * kd).sum(-1, keepdim=True)), -1) / D ** 0.5
        assert (lse[own, h].double() - torch.logsumexp(s, -1)).abs().max() <= 2e-5
        p = torch.softmax(s, -1)
        cached = (p[:, :L] @ cv[b, h].double()) @ wv[0, h].double().T
        o = (cached + p[:, L:] * qkv[own, 2 * H + h].double()).cpu().numpy()
        err = np.abs(widen(out[own, h]) - o)
        assert (err <= _half_step(o) + 2.0 ** -13 * np.abs(cached.cpu().numpy())).all()


@pytest.mark.parametrize("e", [8, 12, 16, 24, -20])
@pytest.mark.parametrize("lens,nodes,page", [([1, 2, 5, 0], [1, 3, 2, 4], 0), ([130, 700], [16, 2], 24), ([260, 1], [33, 40], 0), ([140, 90], [128, 65], 64)])
def test_scale_between_latents_and_weights(lens, nodes, page, e):
    """The same keys from latents 2^-e as large and weights 2^e as large: the same log-sum-exp."""
    c = make(lens, nodes, 2, 96, 160, page, 0, "bf16")
    c["ck"].mul_(2.0 ** -e), c["wk"].mul_(2.0 ** e)
    check(c, call(c))
    n = sum(nodes)
    assert np.abs(widen(c["lse"])[:n] - want(c)[1][:n]).max() <= 2e-5


@pytest.mark.parametrize("nodes", [2, 40])
@pytest.mark.parametrize("which,by", [(slice(0, 250), 2.0 ** -14), (slice(0, 12), 0.0), (slice(0, 250), 0.0), (slice(0, 1), 2.0 ** 10),
                                      (slice(10, 14), 2.0 ** 14)])
def test_sizes_of_latents_that_differ(which, by, nodes):
    """Tokens whose latents are far smaller or far larger than the others', or zero."""
    c = make([400, 300], [nodes, 3], 2, 96, 160, 0, 0, "bf16")
    c["ck"][:, :, which] *= by
    if by > 1:      # (their keys small enough in the end that others keep some weight)
        c["qkv"][:, :2] *= 1.0 / by
    check(c, call(c))
    n = nodes + 3
    assert np.abs(widen(c["lse"])[:n] - want(c)[1][:n]).max() <= 2e-5


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("factor", [1.25, 0.1 * np.log(32.0) + 1.0, 0.5])
@pytest.mark.parametrize("lens,nodes,page,style", [([300, 40], [4, 9], 0, 0), ([520], [50], 64, 1), ([130, 7], [20, 1], 24, 0)])
def test_tables_with_an_attention_factor(lens, nodes, page, style, factor, dtype):
    """A factor on the table's rows multiplies queries and keys, cached and drafted, once each."""
    c = make(lens, nodes, 2, 96, 160, page, style, dtype)
    c["cos"].mul_(factor), c["sin"].mul_(factor)
    check(c, call(c))
    n = sum(nodes)
    assert np.abs(widen(c["lse"])[:n] - want(c)[1][:n]).max() <= 2e-5


@pytest.mark.parametrize("nodes,page", [(3, 0), (20, 24), (70, 64)])
def test_keys_beyond_half_precision_in_a_long_cache(nodes, page):
    """A few of 16389 tokens with keys 2^20 times the others', in one of two sequences; weights that make up the sums
    from all of them.  A score is off by a share of |q| |k| / sqrt d (22 bits of queries, fp32 keys), which is 2^20 2^-18 = 4
    times that of ordinary queries and keys, for which 2e-5 stands: 8e-5."""
    c = make([16389, 300], [nodes, 2], 1, 96, 160, page, 0, "bf16")
    for t in (5, 4000, 16388):
        if page:
            c["ck"][int(c["table"][0, t // page]), :, t % page] *= 2.0 ** 20
        else:
            c["ck"][0, :, t] *= 2.0 ** 20
    c["qkv"][:nodes, 0] *= 2.0 ** -18
    check(c, call(c))
    n = nodes + 2
    assert np.abs(widen(c["lse"])[:n] - want(c)[1][:n]).max() <= 8e-5


def test_a_nan_does_not_hold_up_the_step():
    """A NaN query, or a NaN early in a cache, beside long sequences: its own results are NaN and the call takes about as
    long as any other (ten times as long would be a walk over the cache)."""
    c = make([16384, 16384], [20, 9], 2, 96, 160, 0, 0, "bf16")
    tree = tree_of(c)
    ws = call(c, tree=tree)

    def took():
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        a.record()
        for _ in range(5):
            call(c, ws, tree)
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b)

    took()
    ordinary = took()
    first = c["out"].clone()
    c["qkv"][3, 0, 7] = float("nan")
    assert took() < 10 * ordinary
    assert torch.isnan(c["out"][3, 0].float()).all()
    rest = torch.ones(29, 2, dtype=torch.bool)
    rest[3, 0] = False
    assert torch.equal(c["out"][:29][rest], first[:29][rest])
    c["qkv"][3, 0, 7] = 0.0
    c["ck"][1, 1, 100, 5] = float("nan")
    assert took() < 10 * ordinary
    assert torch.isnan(c["out"][20:29, 1].float()).all() and torch.isfinite(c["out"][:20].float()).all()


def test_calls_without_nodes_between_others():
    """Steps in which no sequence has nodes, and ordinary ones, in turn over one workspace and without a wait."""
    c = make([900, 333], [20, 5], 3, 96, 160, 64, 0, "bf16")
    tree, ws = tree_of(c), None
    none = lla.DraftTree(torch.zeros(3, dtype=torch.int32, device="cuda"), c["parent"], c["max_nodes"], pos=c["pos"])
    for _ in range(50):
        ws = call(c, ws, none)
        ws = call(c, ws, tree)
        ws = call(c, ws, none)
    check(c, ws)
    c["out"].fill_(77.0), c["lse"].fill_(77.0)
    call(c, ws, none)
    assert lla.device_status(ws) == lla.LLA_OK
    assert (c["out"] == 77.0).all() and (c["lse"] == 77.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_caches_of_sequences_without_nodes_are_left_alone(dtype):
    """A sequence without nodes may have a table that names no pages: nothing of it is read, and nothing recorded."""
    c = make([200, 300, 0], [5, 0, 2], 2, 96, 160, 64, 0, dtype)
    c["table"][1].fill_(-1)
    check(c, call(c))


@pytest.mark.parametrize("nodes", [3, 24, 64, 100])
def test_scores_that_rise_in_long_sums(nodes):
    """20000 cached tokens whose keys grow along the cache, a unit's in one block: references move after sums have left
    the accumulators.  Queries 12 times as large: the log-sum-exp to 12 x 2e-5; a weight is then off by 2^-11 at most, and an
    output by that share of its values beside half a step."""
    H, L, rk, rv, B = 16, 20000, 16, 32, 10
    g = torch.Generator(device="cuda").manual_seed(nodes)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    dm, n = lla.dims(1, H, rk, rv), B * nodes
    qkv = rnd(n, 3 * H, D).bfloat16()
    qkv[:, :H] *= 12.0
    qkv[:, H:2 * H] *= 0.1
    size = torch.full((L, 1), 1.0, device="cuda")
    size[:8192], size[8192:9000], size[9000:16384] = 0.02, 0.3, 0.1
    ck, cv = (rnd(B, H, L, rk) * size).bfloat16(), (1 + 0.1 * rnd(B, H, L, rv)).bfloat16()
    wk, wv = (rnd(1, H, D, rk) / 4).bfloat16(), (rnd(1, H, D, rv).abs() / 6).bfloat16()
    zero = torch.zeros(H, D, device="cuda")
    ang = torch.arange(L + 1, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-2.0 * torch.arange(64, dtype=torch.float64, device="cuda") / D)
    cos, sin = ang.cos().float(), ang.sin().float()
    lens = [L, 9000, 8192, 8193, 16384, 12000, L, L, L, L]
    tree = lla.DraftTree(i32([nodes * b for b in range(B + 1)]), i32([-1] * n), nodes, pos=i32([x for x in lens for _ in range(nodes)]))
    out, lse = torch.zeros(n, H, D, device="cuda", dtype=torch.bfloat16), torch.zeros(n, H, device="cuda")
    ws = lla.tree_workspace(dm, tree, L)
    lla.tree_attn(dm, 0, tree, qkv[:, :H], qkv[:, H:2 * H], qkv[:, 2 * H:], ck, cv, i32(lens), wk, wv, zero, zero, cos, sin, out, lse, ws)
    assert lla.device_status(ws) == lla.LLA_OK
    turn = lambda x, at: torch.cat((x[..., :64] * cos[at].double() - x[..., 64:] * sin[at].double(),  # noqa: E731
                                    x[..., :64] * sin[at].double() + x[..., 64:] * cos[at].double()), -1)
    for b, h in ((0, 0), (1, 3), (2, 5), (3, 9), (4, 2), (5, 7), (9, 15)):
        own, m = slice(b * nodes, (b + 1) * nodes), lens[b]
        q, kd = turn(qkv[own, h].double(), m), turn(qkv[own, H + h].double(), m)
        k = turn(ck[b, h, :m].double() @ wk[0, h].double().T, slice(0, m))
        s = torch.cat((q @ k.T, (q * kd).sum(-1, keepdim=True)), -1) / D ** 0.5
        assert (lse[own, h].double() - torch.logsumexp(s, -1)).abs().max() <= 12 * 2e-5
        p = torch.softmax(s, -1)
        o = ((p[:, :m] @ cv[b, h, :m].double()) @ wv[0, h].double().T + p[:, m:] * qkv[own, 2 * H + h].double()).cpu().numpy()
        err = np.abs(widen(out[own, h]) - o)
        assert (err <= _half_step(o) + 2.0 ** -11 * np.abs(o).max() + 2.0 ** -13 * np.abs(o)).all()
