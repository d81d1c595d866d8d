"""Host-side checks (no GPU) of the RoPE operators, the page plan and the 4-bit cache: what
they refuse before any launch, sizes, the binding's structures, and its argument checks."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from looped_transformer_cross_gb300 import build, lla
from oracle import q4

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
    specs = {"lla_rope_scaling": (lla.RopeScaling, ["kind", "factor", "original_len", "fast", "slow"]),
             "lla_q4_cache": (lla.Q4Cache, ["rows", "block_table", "B", "max_pages", "page_size", "num_pages"])}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "lla.h"', "int main(void) {"]
    for c, (_, fields) in specs.items():
        lines.append('printf("%%zu\\n", sizeof(%s));' % c)
        lines += ['printf("%%zu\\n", offsetof(%s, %s));' % (c, f) for f in fields]
    src = tmp_path / "l.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-o", str(tmp_path / "l"), str(src)], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for cls, fields in specs.values():
        want += [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f in fields]
    assert got == want


@pytest.mark.parametrize("r_k,r_v,n", [(96, 160, 144), (16, 32, 32), (16, 16, 32), (256, 256, 288), (48, 80, 80)])
def test_row_bytes(L, r_k, r_v, n):
    assert lla.q4_row_bytes(lla.dims(4, 2, r_k, r_v)) == n == q4.row_bytes(r_k, r_v)


def test_row_bytes_refusals(L):
    z = lambda **k: L.lla_q4_row_bytes(ctypes.byref(lla.dims(4, 2, k.pop("r_k", 96), 160, **k)))
    assert z(variant=lla.LLA_2D) == 0 and z(r_k=100) == 0 and z(r_k=272) == 0 and z(d_head=64) == 0
    with pytest.raises(lla.LLAError):
        lla.q4_row_bytes(lla.dims(4, 2, 96, 160, variant=lla.LLA_2D))
    assert L.lla_q4_workspace_size(ctypes.byref(lla.dims(4, 2, 96, 160, variant=lla.LLA_2D)), 1, 128) == 0
    assert L.lla_q4_workspace_size(ctypes.byref(lla.dims(4, 2, 96, 160)), -1, 128) == 0
    assert L.lla_q4_workspace_size(ctypes.byref(lla.dims(4, 2, 96, 160)), 1, -1) == 0


def test_rope_table_refusals(L, mem):
    def call(d=128, base=10000.0, sc=None, pos0=0, n=4, c=mem(), s=mem(4096)):
        dm = lla.dims(1, 1, 16, 16, d_head=d, rope_base=base)
        return L.lla_rope_table_scaled(ctypes.byref(dm), None if sc is None else ctypes.byref(sc), pos0, n, c, s, None)

    assert call(d=0) == INV and call(d=127) == INV and call(base=-1.0) == INV and call(base=float("inf")) == INV
    assert call(n=-1) == INV and call(pos0=-1) == INV and call(c=None) == INV and call(s=mem(4)) == INV
    assert call(d=258) == UNS and call(n=(1 << 31) + 1) == UNS and call(pos0=(1 << 31) + 1) == UNS
    assert call(n=0) == OK
    sc = lla.rope_scaling
    assert call(sc=lla.RopeScaling(7, 1, 0, 32, 1)) == INV and call(sc=lla.RopeScaling(-1, 1, 0, 32, 1)) == INV
    for f in (0.0, -2.0, float("nan"), float("inf")):
        assert call(sc=sc("linear", f)) == INV
    assert call(sc=sc("by_parts", 2.0, 0)) == INV                    # no original length
    assert call(sc=sc("by_parts", 2.0, 4096, fast=1.0, slow=1.0)) == INV
    assert call(sc=sc("by_parts", 2.0, 4096, fast=2.0, slow=-1.0)) == INV
    assert call(sc=sc("base", 2.0), d=2) == INV
    assert call(sc=sc("base", 1e308)) == INV                          # no frequency left
    assert L.lla_rope_table_scaled(None, None, 0, 4, mem(), mem(4096), None) == INV
    with pytest.raises(ValueError):
        sc("other")


def test_rope_apply_refusals(L, mem):
    base = dict(x=mem(), xt=256, xh=128, out=mem(16384), ot=256, oh=128, N=2, heads=2, d_x=128, off=0, d=128,
                pos=mem(32768), cos=mem(33024), sin=mem(40960), rl=16, inv=0, ws=mem(49152), wb=256,
                dtype=lla.LLA_BF16, style=0)

    def call(**over):
        a = dict(base, **over)
        dm = lla.dims(1, 1, 16, 16, dtype=a["dtype"], rope_style=a["style"])
        return L.lla_rope_apply(ctypes.byref(dm), a["x"], a["xt"], a["xh"], a["out"], a["ot"], a["oh"], a["N"], a["heads"],
                                a["d_x"], a["off"], a["d"], a["pos"], a["cos"], a["sin"], a["rl"], 1.0, a["inv"],
                                a["ws"], a["wb"], None)

    assert call(N=0) == OK
    for bad in (dict(N=-1), dict(heads=0), dict(d_x=0), dict(off=-1), dict(d=0), dict(d=3), dict(d=130), dict(off=2),
                dict(rl=0), dict(wb=255), dict(x=None), dict(out=None), dict(pos=None), dict(cos=None), dict(sin=None),
                dict(ws=None), dict(x=mem(1)), dict(pos=mem(32769)), dict(dtype=3), dict(style=2), dict(xt=-1),
                dict(oh=127),                                   # heads of out overlap
                dict(ot=255),                                   # tokens of out overlap
                dict(out=mem(), ot=512),                        # in place with other strides
                dict(out=mem(2)),                               # shifted onto its own input
                dict(out=mem(256), xt=512, ot=512)):            # heads of out on heads of x
        assert call(**bad) == INV, bad
    assert call(heads=(1 << 20) + 1, N=1) == UNS
    # outputs laid out head-major: tokens of one head next to each other
    assert call(N=4, ot=128, oh=511) == INV
    assert L.lla_rope_apply(None, mem(), 1, 1, mem(), 1, 1, 1, 1, 2, 0, 2, mem(), mem(), mem(), 1, 1.0, 0, mem(), 256,
                            None) == INV


def test_page_plan_refusals(L, mem):
    base = dict(B=2, P=16, mp=4, num=64, ctx=mem(0), new=mem(64), free=mem(128), nf=8, head=mem(192), table=mem(256),
                lens=mem(320), start=mem(384), granted=mem(448), n=8, seq=mem(512), pos=mem(576), slots=mem(640),
                counts=mem(768), ws=mem(1024), wb=256)

    def call(**over):
        a = dict(base, **over)
        return L.lla_page_plan(a["B"], a["P"], a["mp"], a["num"], a["ctx"], a["new"], a["free"], a["nf"], a["head"],
                               a["table"], a["lens"], a["start"], a["granted"], a["n"], a["seq"], a["pos"], a["slots"],
                               a["counts"], a["ws"], a["wb"], None)

    for bad in (dict(B=-1), dict(P=0), dict(mp=0), dict(num=0), dict(nf=-1), dict(n=-1), dict(wb=255), dict(ws=None),
                dict(ctx=None), dict(new=None), dict(free=None), dict(table=None), dict(lens=None), dict(start=None),
                dict(granted=None), dict(seq=None), dict(pos=None), dict(slots=None), dict(counts=None),
                dict(ctx=mem(2)), dict(slots=mem(644)),
                dict(lens=mem(0)), dict(lens=mem(4)),           # the lengths, or part of them, updated in place
                dict(counts=mem(192)),                          # the free list's head updated in place
                dict(table=mem(124))):                          # a table that runs into the free list
        assert call(**bad) == INV, bad
    assert call(B=8193) == UNS and call(P=1 << 20, mp=1 << 11) == UNS and call(num=1 << 31) == UNS


def test_q4_copy_and_decode_refusals(L, mem):
    dm = lla.dims(4, 2, 96, 160)

    def cache(**over):
        a = dict(rows=mem(), bt=mem(64), B=1, mp=4, P=16, num=8)
        a.update(over)
        return lla.Q4Cache(a["rows"], a["bt"], a["B"], a["mp"], a["P"], a["num"])

    def store(d=dm, k=mem(), v=mem(4096), N=2, slots=mem(128), c=None, ws=mem(256), wb=256):
        c = cache() if c is None else c
        r = {L.lla_q4_store(ctypes.byref(d), k, v, N, slots, ctypes.byref(c), ws, wb, None),
             L.lla_q4_load(ctypes.byref(d), slots, N, ctypes.byref(c), k, v, ws, wb, None)}
        assert len(r) == 1
        return r.pop()

    assert store(N=0) == OK
    for bad in (dict(N=-1), dict(k=None), dict(v=mem(8)), dict(slots=None), dict(slots=mem(4)), dict(ws=None),
                dict(wb=255), dict(c=cache(rows=None)), dict(c=cache(rows=mem(8))), dict(c=cache(P=0)),
                dict(c=cache(num=0)), dict(d=lla.dims(0, 2, 96, 160))):
        assert store(**bad) == INV, bad
    for bad in (dict(d=lla.dims(4, 2, 96, 160, variant=lla.LLA_2D)), dict(d=lla.dims(4, 2, 100, 160)),
                dict(c=cache(num=1 << 31)), dict(c=cache(num=1 << 29, P=1 << 12))):
        assert store(**bad) == UNS, bad
    assert L.lla_q4_store(ctypes.byref(dm), mem(), mem(), 1, mem(), None, mem(), 256, None) == INV

    def dec(d=dm, c=None, t=0, q=mem(), rl=128, out=mem(), lse=None, ws=mem(), wb=1 << 30):
        c = cache() if c is None else c
        p = mem()
        return L.lla_decode_attn_q4(ctypes.byref(d), t, q, ctypes.byref(c), p, p, p, p, p, p, p, p, rl, out, lse, ws, wb, None)

    assert dec(c=cache(B=0)) == OK
    for bad in (dict(t=-1), dict(t=4), dict(rl=127), dict(c=cache(mp=0)), dict(c=cache(mp=40), rl=639), dict(q=None),
                dict(out=mem(8)), dict(lse=mem(2)), dict(c=cache(bt=None)), dict(c=cache(bt=mem(2))), dict(c=cache(B=-1)),
                dict(ws=None)):
        assert dec(**bad) == INV, bad
    for bad in (dict(d=lla.dims(4, 2, 96, 160, variant=lla.LLA_2D)), dict(c=cache(mp=1 << 20, P=1 << 11)),
                dict(c=cache(B=1 << 24))):
        assert dec(**bad) == UNS, bad


@pytest.mark.parametrize("num", [1 << 62, (1 << 63) - 1, (1 << 60) + 1])
def test_pool_sizes_past_64_bits(L, mem, num):
    """Page counts whose products with the heads or the page size do not fit 64 bits are refused."""
    dm, p = lla.dims(4, 16, 96, 160), mem()
    c = lla.Q4Cache(p, p, 1, 4, 16, num)
    assert L.lla_q4_store(ctypes.byref(dm), p, p, 2, p, ctypes.byref(c), p, 256, None) == UNS
    assert L.lla_q4_load(ctypes.byref(dm), p, 2, ctypes.byref(c), p, p, p, 256, None) == UNS
    assert L.lla_decode_attn_q4(ctypes.byref(dm), 0, p, ctypes.byref(c), p, p, p, p, p, p, p, p, 128, p, None, p, 1 << 30,
                                None) == UNS


def test_binding_argument_checks(L):
    """The binding names the argument that does not fit before it passes a pointer on."""
    dm = lla.dims(4, 2, 96, 160)
    pool = torch.zeros((4, 2, 16, 144), dtype=torch.uint8)
    slots = torch.zeros(3, dtype=torch.int64)
    k, v = torch.zeros(3, 2, 96, dtype=torch.bfloat16), torch.zeros(3, 2, 160, dtype=torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8)
    for bad in (dict(k=k.float()), dict(k=k[:2]), dict(v=v[..., :96]), dict(slots=slots.int()),
                dict(pool=pool[..., :128].contiguous()), dict(pool=pool.to(torch.int8))):
        a = dict(dict(k=k, v=v, slots=slots, pool=pool), **bad)
        with pytest.raises(ValueError):
            lla.q4_store(dm, a["k"], a["v"], a["slots"], a["pool"], ws)
    with pytest.raises(ValueError):      # everything fits, but it is on the CPU
        lla.q4_store(dm, k, v, slots, pool, ws)
    x = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    c = torch.zeros(8, 64)
    for xx, pos in ((x.float(), torch.zeros(3, dtype=torch.int32)), (x, torch.zeros(2, dtype=torch.int32)),
                    (x[0], torch.zeros(3, dtype=torch.int32)),
                    (torch.zeros(3, 2, 256, dtype=torch.bfloat16)[..., ::2], torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            lla.rope_apply(dm, xx, pos, c, c, workspace=ws)


def test_oracle_pins():
    """The oracle itself: known rows, and the two forms of reading one."""
    codes, scales = q4.round_latent([7.0, -7.0, 0.5, 1.5, 2.5, 0.0, -0.5, 3.49] + [0.0] * 8)
    assert scales == [0x3F80] and codes[:8] == [7, -7, 0, 2, 2, 0, 0, 3]      # scale 1; halves to even
    assert q4.round_latent([0.0] * 16) == ([0] * 16, [0])
    assert q4.round_latent([float("inf")] + [1.0] * 15)[1] == [0x7FC0]
    assert q4.round_latent([float("nan")] * 16)[1] == [0x7FC0]
    assert q4.bf16_bits(1.0 + 2**-8) == 0x3F80 and q4.bf16_bits(1.0 + 3 * 2**-8) == 0x3F82
    g = np.random.default_rng(5)
    ck, cv = g.standard_normal(48).astype(np.float32), g.standard_normal(80).astype(np.float32)
    row = q4.row_of(ck, cv)
    assert len(row) == 80
    k, v = q4.values_of(row, 48, 80)
    k2, v2 = q4.values(np.frombuffer(row, np.uint8), 48, 80)
    np.testing.assert_array_equal(k, k2)
    np.testing.assert_array_equal(v, v2)
    # half a step of the group's grid, and a bf16 half step of the scale at code 7
    for x, y in ((ck, k), (cv, v)):
        for i in range(0, len(x), 32):
            top = np.abs(x[i:i + 32]).max()
            assert np.abs(x[i:i + 32] - y[i:i + 32]).max() <= top / 7 * (0.5 + 7 * 2**-8)
    p = q4.page_plan(4, 3, 10, [3, 8, 0, 12], [2, 4, 0, 1], [9, 8, 7], 0, np.full((4, 3), 5), 8)
    assert p["granted"] == [1, 1, 1, 0] and p["counts"] == [2, 6] and p["tok_start"] == [0, 2, 6, 6, 7]
    assert p["slots"][:6] == [5 * 4 + 3, 9 * 4, 8 * 4, 8 * 4 + 1, 8 * 4 + 2, 8 * 4 + 3] and p["slots"][6] == -1
