"""Host-side checks (no GPU) of the calls that verify drafted tokens: what they refuse before any
launch, sizes, the binding's structures and argument checks, and pins of their oracle."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import oracle
from looped_transformer_cross_gb300 import build, lla
from oracle import tree as otree

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, UNS, OK = lla.LLA_ERR_INVALID_ARG, lla.LLA_ERR_UNSUPPORTED, lla.LLA_OK


@pytest.fixture(scope="module")
def L():
    build.build()
    return lla.lib()


@pytest.fixture(scope="module")
def mem():
    """A host buffer whose addresses stand in for device pointers: every call below is refused
    or has nothing to do before it would launch."""
    buf = (ctypes.c_char * (1 << 16))()
    base = ctypes.addressof(buf)
    base += -base % 64
    yield lambda off=0: ctypes.c_void_p(base + off)
    del buf


def test_struct_layouts(tmp_path):
    specs = {"lla_tree": (lla.Tree, [f for f, _ in lla.Tree._fields_]),
             "lla_logit_rules": (lla.LogitRulesC, [f for f, _ in lla.LogitRulesC._fields_])}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "lla.h"', "int main(void) {",
             'printf("%d\\n", LLA_TREE_MAX_NODES);']
    for c, (_, fields) in specs.items():
        lines.append('printf("%%zu\\n", sizeof(%s));' % c)
        lines += ['printf("%%zu\\n", offsetof(%s, %s));' % (c, f) for f in fields]
    src = tmp_path / "l.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-o", str(tmp_path / "l"), str(src)], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout.split()]
    want = [lla.LLA_TREE_MAX_NODES]
    for cls, fields in specs.values():
        want += [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f in fields]
    assert got == want


def test_sizes(L):
    dm = lla.dims(4, 2, 96, 160)
    size = lambda d=dm, B=3, N=16, cap=1000: L.lla_tree_workspace_size(ctypes.byref(d), B, N, cap)  # noqa: E731
    assert size() > 256 and size(N=17) > size() and size(B=300) > size()
    assert size(N=0) == 0 and size(N=129) == 0 and size(B=-1) == 0 and size(cap=-1) == 0
    assert size(d=lla.dims(4, 2, 96, 160, variant=lla.LLA_2D)) == 0 and size(d=lla.dims(4, 2, 100, 160)) == 0
    assert L.lla_logits_workspace_size(5, 32000) > 256 and L.lla_logits_workspace_size(0, 1) == 256
    assert L.lla_logits_workspace_size(-1, 8) == 0 and L.lla_logits_workspace_size(1, 0) == 0
    assert L.lla_logits_workspace_size(1, (1 << 22) + 1) == 0


def test_kernel_names(L):
    assert lla.tree_kernel(lla.dims(4, 2, 96, 160, dtype=lla.LLA_F32)) == "plain"
    assert lla.tree_kernel(lla.dims(4, 2, 96, 160, variant=lla.LLA_2D)) is None
    bf = lla.dims(4, 2, 96, 160)
    assert all(lla.tree_kernel(bf, p) == "tensor" for p in (0, 1, 4, 8, 16, 24, 32, 64, 100, 128, 192, 256))
    assert lla.tree_kernel(lla.dims(4, 2, 256, 256)) == "plain" and lla.tree_kernel(lla.dims(4, 2, 16, 256)) == "tensor"
    assert lla.tree_kernel(lla.dims(4, 2, 100, 160)) is None and lla.tree_kernel(lla.dims(4, 2, 96, 160), -1) is None


def test_tree_attn_refusals(L, mem):
    def call(d=lla.dims(4, 2, 96, 160), t=0, B=1, cB=None, n=4, N=4, start=mem(), parent=mem(), pos=mem(), q=mem(32768), qs=256,
             ks=256, vs=256, k=mem(32768), ck=mem(), cap=128, lens=mem(), rl=128, out=mem(), lse=None, ws=mem(), wb=1 << 30,
             paged=None, tree=True):
        tr = lla.Tree(B, n, N, start, parent, pos)
        p = mem()
        args = [ctypes.byref(d) if d else None, t, ctypes.byref(tr) if tree else None, q, qs, k, ks, mem(32768), vs]
        rest = [lens, p, p, p, p, p, p, rl, out, lse, ws, wb, None]
        cB = B if cB is None else cB
        if paged is None:
            return L.lla_tree_attn(*args, lla.Cache(ck, p, cB, cap), *rest)
        bt, mp, P, num = paged
        return L.lla_tree_attn_paged(*args, lla.PagedCache(ck, p, bt, cB, mp, P, num), *rest)

    assert call(B=0) == OK and call(n=0) == OK
    for bad in (dict(d=None), dict(t=-1), dict(t=4), dict(tree=False), dict(B=-1, cB=-1), dict(cB=2), dict(n=-1), dict(N=0),
                dict(cap=0), dict(rl=127), dict(cap=200, rl=199), dict(qs=255), dict(ks=128), dict(vs=257), dict(q=None),
                dict(q=mem(32768 + 8)), dict(k=None), dict(ck=None), dict(out=mem(8)), dict(out=None), dict(ws=None), dict(wb=255),
                dict(start=None), dict(start=mem(2)), dict(parent=None), dict(pos=None), dict(lens=None), dict(lse=mem(2)),
                dict(out=mem(32768)), dict(out=mem(32768 + 2032)), dict(out=mem(32768 - 16)),   # out over q, k or v
                dict(paged=(None, 1, 128, 4)), dict(paged=(mem(2), 1, 128, 4)), dict(paged=(mem(), 0, 128, 4)),
                dict(paged=(mem(), 1, 0, 4)), dict(paged=(mem(), 1, 128, 0)), dict(paged=(mem(), 2, 100, 4), rl=199)):
        assert call(**bad) == INV, bad
    for bad in (dict(N=129), dict(d=lla.dims(4, 2, 96, 160, variant=lla.LLA_2D)), dict(d=lla.dims(4, 2, 100, 160)),
                dict(cap=(1 << 30) + 1, rl=1 << 31), dict(B=1 << 24), dict(n=1 << 30),
                dict(paged=(mem(), 1 << 20, 1 << 11, 4)), dict(paged=(mem(), 1, 16, 1 << 31)), dict(paged=(mem(), 1, 16, 1 << 62))):
        assert call(**bad) == UNS, bad


def test_logits_refusals(L, mem):
    def rules(**over):
        a = dict(history=mem(), hist_len=mem(), prompt_len=mem(), max_history=4, repetition=mem(), presence=mem(), frequency=mem(),
                 bias_token=mem(), bias=mem(), max_bias=2, allowed=mem(), allowed_row=mem(), n_masks=1)
        a.update(over)
        return lla.LogitRulesC(*[a[f] for f, _ in lla.LogitRulesC._fields_])

    def call(B=1, n=4, N=4, start=mem(), parent=mem(), token=mem(), dtype=lla.LLA_BF16, x=mem(), rs=100, V=100, r=None,
             out=mem(8192), os_=100, best=None, lse=None, ws=mem(16384), wb=1 << 20, tree=True):
        tr = lla.Tree(B, n, N, start, parent, None)
        r = rules() if r is None else r
        return L.lla_logits_adjust(ctypes.byref(tr) if tree else None, token, dtype, x, rs, V, ctypes.byref(r), out, os_, best,
                                   lse, ws, wb, None)

    assert call(B=0) == OK and call(n=0) == OK
    for bad in (dict(tree=False), dict(B=-1), dict(n=-1), dict(N=0), dict(V=0), dict(dtype=2), dict(rs=99), dict(os_=99), dict(x=None),
                dict(x=mem(1)), dict(x=mem(2), dtype=lla.LLA_F32, out=None, lse=mem()), dict(out=mem(8193)),
                dict(out=None), dict(start=None), dict(parent=None), dict(token=None), dict(token=mem(2)), dict(best=mem(2)),
                dict(lse=mem(1)), dict(ws=None), dict(ws=mem(16384 + 8)), dict(wb=256),
                dict(out=mem(), os_=101), dict(out=mem(798)), dict(out=mem(2)),              # partly over the input
                dict(r=rules(max_history=-1)), dict(r=rules(max_bias=-1)), dict(r=rules(n_masks=-1)), dict(r=rules(history=None)),
                dict(r=rules(hist_len=None)), dict(r=rules(prompt_len=mem(2))), dict(r=rules(bias=None)), dict(r=rules(bias_token=mem(2))),
                dict(r=rules(allowed=None)), dict(r=rules(allowed_row=None)), dict(r=rules(repetition=mem(2)))):
        assert call(**bad) == INV, bad
    assert L.lla_logits_adjust(ctypes.byref(lla.Tree(1, 1, 1, mem(), mem(), None)), mem(), 0, mem(), 8, 8, None, mem(64), 8, None,
                               None, mem(1024), 4096, None) == INV
    assert call(N=129) == UNS and call(V=(1 << 22) + 1, rs=1 << 23, os_=1 << 23) == UNS
    assert call(B=1 << 30, V=1 << 20, rs=1 << 20, os_=1 << 20) == UNS


def test_accept_refusals(L, mem):
    base = dict(B=2, n=8, N=8, start=mem(0), parent=mem(64), token=mem(128), chosen=mem(192), ctx=mem(256), count=mem(320),
                nxt=mem(384), lens=mem(448), path=mem(512), seq=mem(576), pos=mem(640), ws=mem(1024), wb=256)

    def call(tree=True, **over):
        a = dict(base, **over)
        tr = lla.Tree(a["B"], a["n"], a["N"], a["start"], a["parent"], None)
        return L.lla_tree_accept(ctypes.byref(tr) if tree else None, a["token"], a["chosen"], a["ctx"], a["count"], a["nxt"],
                                 a["lens"], a["path"], a["seq"], a["pos"], a["ws"], a["wb"], None)

    assert call(B=0) == OK
    for bad in (dict(tree=False), dict(B=-1), dict(n=-1), dict(N=0), dict(wb=255), *(dict([(k, None)]) for k in base if k not in ("B", "n", "N", "wb")),
                dict(ctx=mem(258)), dict(path=mem(514)),
                dict(lens=mem(256)), dict(lens=mem(260)),       # the lengths, or part of them, in place
                dict(path=mem(128)), dict(pos=mem(64)), dict(count=mem(8))):
        assert call(**bad) == INV, bad
    assert call(N=129) == UNS


def test_binding_argument_checks(L):
    """The binding names what does not fit before it passes a pointer on."""
    i32 = torch.int32
    with pytest.raises(ValueError):                  # on the CPU
        lla.DraftTree(torch.zeros(2, dtype=i32), torch.zeros(3, dtype=i32), 4)
    with pytest.raises(ValueError):
        lla.LogitRules(repetition=torch.ones(2))
    with pytest.raises(ValueError):
        lla.LogitRules(prompt_len=torch.ones(2, dtype=i32))
    assert lla.LogitRules().dev is None              # no rule at all


# ------------------------------------------------------------------ the oracle itself

def test_oracle_tree_is_the_decode_oracle():
    """A node that is the only one, with the same token's latent behind the cache, against the decode
    oracle over the cache alone merged with its own exact key by log-sum-exp."""
    T, H, d, rk, rv, n = 2, 2, 128, 16, 32, 7
    g = np.random.default_rng(3)
    dm = oracle.dims(T, H, d, rk, rv)
    wk, wv = g.standard_normal((T, H, d, rk)) / 4, g.standard_normal((T, H, d, rv)) / 5
    mk, mv = g.standard_normal((H, T * d)) / 3, g.standard_normal((H, T * d)) / 3
    ck, cv = g.standard_normal((1, H, n, rk)), g.standard_normal((1, H, n, rv))
    q, k, v = (g.standard_normal((1, H, d)) for _ in range(3))
    t = 1
    o, lse, _ = oracle.decode(dm, t, q, ck, cv, np.array([n], np.int32), np.array([n], np.int32), wk, wv, mk, mv)
    pos = np.arange(n + 1)[:, None] * 10000.0 ** (-2.0 * np.arange(64) / 128)
    cos, sin = np.cos(pos), np.sin(pos)
    got, got_lse, tol, _ = otree.tree_attn(q, k, v, [0, 1], [-1], [n], lambda b, h: (ck[b, h], cv[b, h]), wk[t], wv[t],
                                           mk[:, t * d:(t + 1) * d], mv[:, t * d:(t + 1) * d], cos, sin, 0)
    for h in range(H):
        s = otree.turn(q[0, h], cos[n], sin[n], 0) @ otree.turn(k[0, h], cos[n], sin[n], 0) / math.sqrt(d)
        both = np.logaddexp(s, lse[0, h])
        want = o[0, h] * math.exp(lse[0, h] - both) + v[0, h] * math.exp(s - both)
        np.testing.assert_allclose(got[0, h], want, rtol=1e-11, atol=1e-11)
        assert abs(got_lse[0, h] - both) < 1e-11
    assert (tol > 0).all() and tol.max() < 0.1


def test_oracle_paths_and_acceptance():
    assert otree.path_of([-1, 0, 0, 1, 9, -5], 3) == [3, 1, 0]
    assert otree.path_of([-1, 0, 0, 1, 9, -5], 4) == [4] and otree.path_of([-1, 0, 0, 1, 9, -5], 5) == [5]
    #        0
    #      1   2      tokens: 1 -> 7, 2 -> 8, 3 -> 8, 4 -> 9
    #     3 4
    got = otree.tree_accept([0, 5, 5], [-1, 0, 0, 1, 1], [5, 7, 8, 8, 9], [7, 9, 0, 0, 3], [10, -4])
    assert got[0] == (3, 3, 13, [0, 1, 4], [10, 11, 13, 14, 12]) and got[1] == (0, -1, 0, [], [])
    # two children with the chosen token: the lower one
    assert otree.tree_accept([0, 3], [-1, 0, 0], [1, 4, 4], [4, 6, 7], [0])[0][:2] == (2, 6)


def test_oracle_logits():
    x = np.array([[2.0, -1.0, 0.5, 3.0], [1.0, 1.0, -2.0, 0.0]])
    y, best, lse = otree.logits_adjust(x, [0, 2], [-1, 0], [1, 3], [[0, 1, 1]], [1], [2.0], [0.5], [0.25], [[(2, 1.0), (2, 1.0)]],
                                       [None, {0, 1}])
    # row 0: prompt {0}, output [1, 1], path [1]; row 1: path [3, 1]
    np.testing.assert_allclose(y[0], [1.0, -2.0 - 0.75 - 0.5, 2.5, 3.0])
    np.testing.assert_allclose(y[1], [0.5, 0.5 - 0.75 - 0.5, -np.inf, -np.inf])
    assert list(best) == [3, 0] and abs(lse[0] - math.log(sum(math.exp(t) for t in y[0]))) < 1e-12


@pytest.mark.parametrize("d", [lla.dims(4, 1, 96, 160, dtype=lla.LLA_F32), lla.dims(4, 1, 256, 256), lla.dims(4, 3, 96, 160),
                               lla.dims(4, 2, 16, 240)])
def test_sizes_do_not_fall(L, d):
    """A workspace for a larger batch, cache or tree does for a smaller one."""
    size = lambda B, N, cap: L.lla_tree_workspace_size(ctypes.byref(d), B, N, cap)  # noqa: E731
    sizes = [1, 2, 3, 4, 5, 7, 8, 31, 32, 33, 127, 128]
    lengths = [0, 1, 31, 32, 33, 64, 95, 96, 97, 128, 129, 1000, 4096, 5000]
    for N in sizes:
        for cap in lengths:
            by_batch = [size(B, N, cap) for B in range(1, 40)]
            assert by_batch == sorted(by_batch)
    for B in (1, 2, 3, 5, 20):
        for N in sizes:
            by_length = [size(B, N, cap) for cap in lengths]
            assert by_length == sorted(by_length)
        for cap in lengths:
            by_nodes = [size(B, N, cap) for N in sizes]
            assert by_nodes == sorted(by_nodes)


@pytest.mark.parametrize("rv,nodes,B,ok", [(192, 128, 32, False), (192, 128, 31, True), (192, 33, 64, False), (160, 128, 64, False),
                                           (160, 64, 127, True), (160, 1, 128, False)])
def test_tiles_of_all_blocks_of_nodes_are_counted(L, mem, rv, nodes, B, ok):
    """2^23 tiles of 128 tokens a sequence and head, through a table that names its pages again and again: once for each
    block of nodes, 2^30 of them are refused (others here for their workspace)."""
    d = lla.dims(1, 1, 96, rv)
    p = mem()
    tr = lla.Tree(B, 4, nodes, p, p, p)
    st = L.lla_tree_attn_paged(ctypes.byref(d), 0, ctypes.byref(tr), mem(32768), 128, mem(32768), 128, mem(32768), 128,
                               lla.PagedCache(p, p, p, B, 1 << 23, 128, 4), p, p, p, p, p, p, p, 1 << 30, p, None, p, 255, None)
    assert (st == INV) if ok else (st == UNS)


@pytest.fixture(scope="module")
def room():
    """Megabytes of a host buffer, cut into pieces that stand in for device pointers."""
    buf = (ctypes.c_char * (16 << 20))()
    base = ctypes.addressof(buf)
    base += -base % 256
    yield lambda k: base + k * (1 << 18)
    del buf


def _refuses_overlaps(call, base, outs):
    """Every output over the start and the inside of every input and of every other output."""
    for o in outs:
        for other in (x for x in base if x != o):
            for off in (0, 4 if other in ("best", "lse", "count", "next", "seq_lens", "path", "seq_idx", "pos_out") else 16):
                if off % 16 == 0 or o not in ("out", "ws"):      # (those two lie on 16 bytes)
                    assert call(**{o: base[other] + off}) == INV, (o, other, off)


@pytest.mark.parametrize("paged", [False, True])
def test_tree_attn_overlaps(L, room, paged):
    d = lla.dims(2, 2, 16, 32, dtype=lla.LLA_F32)
    names = ["out", "lse", "ws", "q", "k", "v", "ck", "cv", "wk", "wv", "mk", "mv", "cos", "sin", "lens", "start", "parent", "pos"]
    base = {n: room(i) for i, n in enumerate(names + ["table"] * paged)}

    def call(**over):
        a = {n: ctypes.c_void_p(x) for n, x in dict(base, **over).items()}
        tr = lla.Tree(5, 6, 4, a["start"], a["parent"], a["pos"])
        head = [ctypes.byref(d), 1, ctypes.byref(tr), a["q"], 256, a["k"], 256, a["v"], 256]
        tail = [a["lens"], a["wk"], a["wv"], a["mk"], a["mv"], a["cos"], a["sin"], 128, a["out"], a["lse"], a["ws"], 1 << 24, None]
        if paged:
            return L.lla_tree_attn_paged(*head, lla.PagedCache(a["ck"], a["cv"], a["table"], 5, 4, 32, 8), *tail)
        return L.lla_tree_attn(*head, lla.Cache(a["ck"], a["cv"], 5, 128), *tail)

    _refuses_overlaps(call, base, names[:3])
    # an output whose end lies inside an input
    assert call(q=base["out"] + 6 * 256 * 4 - 16) == INV and call(lens=base["lse"] + 6 * 2 * 4 - 4) == INV


def test_logits_overlaps(L, room):
    names = ["out", "best", "lse", "ws", "logits", "token", "start", "parent", "history", "hist_len", "prompt_len", "rep", "pres", "freq",
             "bias_token", "bias", "allowed", "allowed_row"]
    base = {n: room(i) for i, n in enumerate(names)}

    def call(**over):
        a = {n: ctypes.c_void_p(x) for n, x in dict(base, **over).items()}
        tr = lla.Tree(5, 6, 4, a["start"], a["parent"], None)
        r = lla.LogitRulesC(a["history"], a["hist_len"], a["prompt_len"], 9, a["rep"], a["pres"], a["freq"], a["bias_token"], a["bias"], 6,
                            a["allowed"], a["allowed_row"], 3)
        return L.lla_logits_adjust(ctypes.byref(tr), a["token"], lla.LLA_F32, a["logits"], 1000, 1000, ctypes.byref(r), a["out"], 1000,
                                   a["best"], a["lse"], a["ws"], 1 << 20, None)

    _refuses_overlaps(call, {n: x for n, x in base.items() if n != "logits"}, names[:4])      # (out may be logits)
    for o in names[1:4]:
        assert call(**{o: base["logits"] + 48}) == INV
    assert call(out=base["logits"] + 16) == INV and call(token=base["out"] + 24000 - 4) == INV
    # in place it is an input and an output, which nothing else may lie over
    assert call(out=base["logits"], best=base["logits"] + 48) == INV


def test_accept_overlaps(L, room):
    names = ["count", "next", "seq_lens", "path", "seq_idx", "pos_out", "ws", "start", "parent", "token", "chosen", "ctx"]
    base = {n: room(i) for i, n in enumerate(names)}

    def call(**over):
        a = {n: ctypes.c_void_p(x) for n, x in dict(base, **over).items()}
        tr = lla.Tree(5, 6, 4, a["start"], a["parent"], None)
        return L.lla_tree_accept(ctypes.byref(tr), a["token"], a["chosen"], a["ctx"], a["count"], a["next"], a["seq_lens"], a["path"],
                                 a["seq_idx"], a["pos_out"], a["ws"], 256, None)

    _refuses_overlaps(call, base, names[:7])
