"""The 4-bit paged latent cache: lla_q4_store, lla_q4_load and lla_decode_attn_q4 against the
64-bit oracle on the same rows, and the whole step (plan, encode, store, decode) together.

Rows that hold no token of a call (unused pages, the rest of a last page) are 0xFF bytes:
scales that read as NaN, so a result that touched one shows it.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from lla_cases import TOL, lse_err, rel_err, widen
from looped_transformer_cross_gb300 import lla
from oracle import q4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from looped_transformer_cross_gb300 import build
    build.build()


def _sd(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _dims(T, H, rk, rv, dtype="bf16", style=0):
    return lla.dims(T, H, rk, rv, dtype=lla.LLA_BF16 if dtype == "bf16" else lla.LLA_F32, rope_style=style)


# ------------------------------------------------------------------ store and load

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,H,rk,rv,P", [(1, 1, 16, 16, 1), (5, 3, 96, 160, 16), (9, 16, 16, 32, 24), (3, 2, 256, 256, 64),
                                         (4, 5, 48, 80, 7), (2, 1, 240, 16, 128)])
def test_store_writes_the_oracle_rows(dtype, N, H, rk, rv, P):
    """Bit for bit the oracle's rows at the given slots, nothing elsewhere; the load gives their
    values, rounded once."""
    dm = _dims(1, H, rk, rv, dtype)
    g = torch.Generator().manual_seed(rk + rv + N)
    ck, cv = (torch.randn(N, H, r, generator=g) * torch.exp(2 * torch.randn(N, H, 1, generator=g)) for r in (rk, rv))
    ck, cv = ck.to(_sd(dtype)), cv.to(_sd(dtype))
    ck[0, 0] = 0.0                                             # a row of zeros
    cv[-1, -1, :16] = torch.tensor([3.5, 7.0] * 8)             # quotients half way between codes
    pages = N // P + 2
    slots = torch.randperm(pages * P, generator=g)[:N]
    pool = torch.full((pages, H, P, q4.row_bytes(rk, rv)), 0xFF, dtype=torch.uint8)
    want = pool.numpy().copy()
    for n in range(N):
        for h in range(H):
            row = q4.row_of(ck[n, h].float().numpy(), cv[n, h].float().numpy())
            want[int(slots[n]) // P, h, int(slots[n]) % P] = np.frombuffer(row, np.uint8)
    pool, ws = pool.cuda(), torch.zeros(256, dtype=torch.uint8, device="cuda")
    lla.q4_store(dm, ck.cuda(), cv.cuda(), slots.cuda(), pool, ws)
    np.testing.assert_array_equal(pool.cpu().numpy(), want)
    ok, ov = torch.empty_like(ck).cuda(), torch.empty_like(cv).cuda()
    lla.q4_load(dm, slots.cuda(), pool, ok, ov, ws)
    vk, vv = q4.values(want[slots.numpy() // P, :, slots.numpy() % P], rk, rv)
    for got, v in ((ok, vk), (ov, vv)):
        assert torch.equal(got.cpu(), torch.from_numpy(v).float().to(_sd(dtype)))
    assert lla.device_status(ws) == lla.LLA_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,H,rk,rv,P", [(3, 37, 112, 240, 16), (2, 130, 16, 16, 3), (1, 9, 256, 240, 1)])
def test_store_many_heads(dtype, N, H, rk, rv, P):
    """More heads than a block's threads hold at a time, and the last step of them not full."""
    test_store_writes_the_oracle_rows(dtype, N, H, rk, rv, P)


def test_store_fp32_next_to_ties():
    """fp32 latents at, just above and just below the half-way points of their group's grid, for scales
    of any mantissa and size: the codes of the fp32 quotients."""
    dm, g = _dims(1, 1, 256, 16, "f32"), np.random.default_rng(6)
    N = 400
    ck = np.zeros((N, 1, 256), np.float32)
    for n in range(N):
        for a in range(0, 256, 32):
            amax = np.float32(g.uniform(1, 2) * 2.0 ** int(g.integers(-100, 100)))
            bits = (np.array([amax / np.float32(7)], np.float32).view(np.uint32) + 0x7FFF + 0) & 0xFFFF0000
            sc = bits.view(np.float32)[0]
            c = (g.integers(-7, 7, 32) + 0.5).astype(np.float32) * sc
            step = g.integers(-2, 3, 32)
            c = np.where(step > 0, np.nextafter(c, np.float32(np.inf)), np.where(step < 0, np.nextafter(c, np.float32(-np.inf)), c))
            c = np.clip(c, -amax, amax)
            c[g.integers(32)] = amax
            ck[n, 0, a:a + 32] = c
    cv = g.standard_normal((N, 1, 16)).astype(np.float32)
    pool, ws = lla.q4_pool(dm, 1, N), torch.zeros(256, dtype=torch.uint8, device="cuda")
    lla.q4_store(dm, torch.from_numpy(ck).cuda(), torch.from_numpy(cv).cuda(), torch.arange(N, device="cuda"), pool, ws)
    want = np.stack([np.frombuffer(q4.row_of(ck[n, 0], cv[n, 0]), np.uint8) for n in range(N)])
    np.testing.assert_array_equal(pool.cpu().numpy()[0, 0], want)


def test_store_values_that_are_not_finite():
    """A group with an infinity or a NaN reads as NaN, its neighbours as themselves; the largest
    and the smallest finite values keep their group."""
    dm = _dims(1, 1, 96, 32, "f32")
    ck = torch.ones(2, 1, 96)
    ck[0, 0, 3], ck[0, 0, 70] = math.inf, math.nan
    ck[1, 0, :32], ck[1, 0, 32:64] = 3.0e38, 1e-38
    cv = torch.full((2, 1, 32), -2.0)
    pool, ws = lla.q4_pool(dm, 1, 2), torch.zeros(256, dtype=torch.uint8, device="cuda")
    slots = torch.arange(2, device="cuda")
    lla.q4_store(dm, ck.cuda(), cv.cuda(), slots, pool, ws)
    want = np.stack([np.frombuffer(q4.row_of(ck[i, 0].numpy(), cv[i, 0].numpy()), np.uint8) for i in range(2)])
    np.testing.assert_array_equal(pool.cpu().numpy()[0, 0], want)
    ok, ov = torch.empty_like(ck).cuda(), torch.empty_like(cv).cuda()
    lla.q4_load(dm, slots, pool, ok, ov, ws)
    assert ok[0, 0, :32].isnan().all() and ok[0, 0, 64:].isnan().all() and ok[0, 0, 32:64].isfinite().all()
    assert ok[1].isfinite().all() and ov.isfinite().all()


def test_slots_that_hold_no_token():
    """Negative slots are skipped in both directions, slots beyond the pool are reported."""
    dm = _dims(1, 2, 16, 32)
    ck, cv = torch.randn(3, 2, 16, device="cuda").bfloat16(), torch.randn(3, 2, 32, device="cuda").bfloat16()
    pool, ws = lla.q4_pool(dm, 2, 4), torch.zeros(256, dtype=torch.uint8, device="cuda")
    for slots, status in (([-1, 5, -9], lla.LLA_OK), ([8, 5, 1 << 40], lla.LLA_ERR_DEVICE_ARG)):
        pool.zero_()
        s = torch.tensor(slots, device="cuda")
        lla.q4_store(dm, ck, cv, s, pool, ws)
        assert lla.device_status(ws) == status
        rest = pool.clone()
        rest[1, :, 1] = 0
        assert not rest.any() and pool[1, :, 1].any()
        ok, ov = torch.full_like(ck, 5.0), torch.full_like(cv, 5.0)
        lla.q4_load(dm, s, pool, ok, ov, ws)
        assert lla.device_status(ws) == status
        assert (ok[[0, 2]] == 5.0).all() and (ov[[0, 2]] == 5.0).all() and (ok[1] != 5.0).all()
    lla.q4_store(dm, ck[:0], cv[:0], torch.empty(0, dtype=torch.int64, device="cuda"), pool, ws)


# ------------------------------------------------------------------ decode

def _inputs(lens, H, rk, rv, P, dtype, seed, T=2, extra=2, scale=1.0, max_pages=None):
    """Rows of random latents at shuffled pages, 0xFF elsewhere, and the call's other inputs."""
    g = np.random.default_rng(seed)
    tg = torch.Generator().manual_seed(seed)
    B, mp = len(lens), max_pages or max(1, max(-(-int(n) // P) for n in lens))
    held = [-(-int(n) // P) for n in lens]
    num = sum(held) + extra
    perm = g.permutation(num)
    table = np.full((B, mp), -1, np.int32)
    k = 0
    for b in range(B):
        table[b, :held[b]] = perm[k:k + held[b]]
        k += held[b]
    rb = q4.row_bytes(rk, rv)
    pool = np.full((num, H, P, rb), 0xFF, np.uint8)
    codes = lambda n, r: (g.integers(1, 16, (n, H, r // 2)) | (g.integers(1, 16, (n, H, r // 2)) << 4)).astype(np.uint8)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        # codes 1..15 and scales around 0.25 (codes of N(0, 1) latents have 0.3)
        s = torch.from_numpy(0.25 * scale * np.exp(0.3 * g.standard_normal((n, H, q4.groups(rk) + q4.groups(rv))))).bfloat16()
        rows = np.concatenate([codes(n, rk), codes(n, rv), s.view(torch.uint8).numpy().reshape(n, H, -1)], -1)
        rows = np.pad(rows, ((0, 0), (0, 0), (0, rb - rows.shape[-1])))
        j = np.arange(n)
        pool[table[b, j // P], :, j % P] = rows
    sd = _sd(dtype)
    rnd = lambda std, *s: torch.randn(*s, generator=tg) * std  # noqa: E731
    return dict(lens=np.asarray(lens, np.int32), table=table, pool=pool, H=H, rk=rk, rv=rv, P=P, T=T, dtype=dtype,
                q_pos=np.maximum(np.asarray(lens, np.int32) - 1, 0), q=rnd(1.0, B, H, 128).to(sd),
                wk=rnd(rk ** -0.5, T, H, 128, rk).to(sd), wv=rnd(rv ** -0.5, T, H, 128, rv).to(sd),
                mk=rnd(0.3, H, T * 128), mv=rnd(0.3, H, T * 128))


def _gpu(x, t, style=0, lse=True, ws=None, out=None, base=10000.0):
    dm = _dims(x["T"], x["H"], x["rk"], x["rv"], x["dtype"], style)
    cap = x["table"].shape[1] * x["P"]
    B = len(x["lens"])
    cos, sin = lla.rope_table(dm, max(cap, 128))
    ws = lla.q4_workspace(dm, B, cap) if ws is None else ws
    out = torch.full((B, x["H"], 128), math.nan, dtype=_sd(x["dtype"]), device="cuda") if out is None else out
    lse = torch.full((B, x["H"]), math.nan, device="cuda") if lse else None
    c = lambda v: (torch.from_numpy(v) if isinstance(v, np.ndarray) else v).cuda()  # noqa: E731
    lla.decode_attn_q4(dm, t, c(x["q"]), c(x["pool"]), c(x["table"]), c(x["lens"]), c(x["q_pos"]), c(x["wk"]), c(x["wv"]),
                       c(x["mk"]), c(x["mv"]), cos.cuda(), sin.cuda(), out, lse, ws)
    return out, lse, lla.device_status(ws)


def _oracle(x, t, style=0, bsel=None):
    """The fp64 oracle on the values that the rows stand for."""
    sel = range(len(x["lens"])) if bsel is None else bsel
    lens = x["lens"][list(sel)]
    L = max(1, int(lens.max()))
    ck, cv = np.zeros((len(lens), x["H"], L, x["rk"])), np.zeros((len(lens), x["H"], L, x["rv"]))
    for i, b in enumerate(sel):
        n = int(lens[i])
        j = np.arange(n)
        rows = x["pool"][np.maximum(x["table"][b, j // x["P"]], 0), :, j % x["P"]].transpose(1, 0, 2)
        ck[i, :, :n], cv[i, :, :n] = q4.values(rows, x["rk"], x["rv"])
    od = oracle.dims(x["T"], x["H"], 128, x["rk"], x["rv"], 0, 10000.0, style)
    out, lse, _ = oracle.decode(od, t, widen(x["q"][list(sel)]), ck, cv, lens, x["q_pos"][list(sel)], widen(x["wk"]),
                                widen(x["wv"]), widen(x["mk"]), widen(x["mv"]))
    return out, lse


def _check(x, t, style=0, bsel=None):
    out, lse, st = _gpu(x, t, style)
    assert st == lla.LLA_OK, lla.status_string(st)
    ro, rl = _oracle(x, t, style, bsel)
    go, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(go).all()
    if bsel is not None:
        go, gl = go[list(bsel)], gl[list(bsel)]
    e = rel_err(go, ro), lse_err(gl, rl)
    assert max(e) <= TOL[x["dtype"]], e
    return e


RANKS = [(96, 160), (16, 32), (16, 16), (256, 256), (48, 80), (112, 240), (32, 64), (240, 16)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rk,rv", RANKS)
def test_decode_ranks(dtype, rk, rv):
    """Every kind of rank (whole and half scale groups), lengths from zero to past several tiles."""
    x = _inputs([0, 1, 127, 128, 129, 400, 257], 3, rk, rv, 24, dtype, rk * 7 + rv)
    for t in range(x["T"]):
        _check(x, t, style=t)


@pytest.mark.parametrize("P", [1, 5, 8, 16, 64, 100, 128, 200, 256])
def test_decode_page_sizes(P):
    """Pages smaller than, equal to and larger than a tile, and ones that end inside a tile."""
    _check(_inputs([300, 1, 0, 131], 4, 96, 160, P, "bf16", 900 + P), 1)


@pytest.mark.parametrize("H", [1, 2, 3, 5, 16])
@pytest.mark.parametrize("rk,rv", [(96, 160), (16, 32)])
def test_decode_heads(H, rk, rv):
    _check(_inputs([200, 3, 513], H, rk, rv, 64, "bf16", 40 + H), 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[1], [0], [0, 0, 0], [5000], [2, 4097, 0, 1, 700]])
def test_decode_splits(dtype, lens):
    """One token, none at all, and long sequences split over many blocks."""
    x = _inputs(lens, 2, 96, 160, 64, dtype, 77 + len(lens))
    out, lse, _ = _gpu(x, 0)
    for b, n in enumerate(lens):
        if n == 0:
            assert (out[b] == 0).all() and (lse[b] == -math.inf).all()
    _check(x, 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_many_short_sequences(dtype):
    """More sequence-heads than blocks, several per block."""
    g = np.random.default_rng(1)
    _check(_inputs(list(g.integers(0, 150, 300)), 4, 32, 48, 16, dtype, 11), 1, bsel=range(0, 300, 17))


@pytest.mark.parametrize("rk,rv,H,lens", [(240, 240, 1, [60000, 0, 40001]), (256, 256, 3, [20000, 13333]), (96, 160, 5, [1, 20001]),
                                          (96, 160, 4, [50001]), (176, 64, 2, [99999]), (48, 80, 4, [100001]),
                                          (16, 32, 8, [60000, 40001])])
def test_decode_long_runs(rk, rv, H, lens):
    """Blocks with several positions of a sequence, at every number of heads that share one: each
    buffer and barrier is used again, by either of the groups that take turns."""
    x = _inputs(lens, H, rk, rv, 128, "bf16", 500 + rk + H, T=1)
    first, _, _ = _gpu(x, 0)
    _check(x, 0)
    for _ in range(3):                                         # and always with the same bits
        again, _, _ = _gpu(x, 0)
        assert torch.equal(first, again)


def test_decode_full_size_sampled():
    """The serving shape (32 x 4096 tokens, 16 heads, 96 / 160) on sampled sequences."""
    g = np.random.default_rng(2)
    _check(_inputs(list(g.integers(3584, 4097, 32)), 16, 96, 160, 64, "bf16", 5, T=1), 0, bsel=[0, 17, 31])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** -20, 1.0, 16.0])
def test_decode_scales_of_any_size(dtype, scale):
    """Latents from far below to far above one: no operand leaves its type's range."""
    x = _inputs([150, 64], 2, 96, 160, 16, dtype, 31, scale=scale)
    out, lse, st = _gpu(x, 0)
    assert st == lla.LLA_OK
    ro, rl = _oracle(x, 0)
    # at scale 16 scores reach tens: an operand's half step (f16 2^-11 on K, 2^-11 on the folded
    # query) moves a score by up to its size times 2^-10, and an output by that share of the spread
    tol = TOL[dtype] * max(1.0, scale)
    e = rel_err(out.double().cpu().numpy(), ro), lse_err(lse.double().cpu().numpy(), rl)
    assert max(e) <= tol, e


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rk,rv", [(96, 160), (16, 32)])
@pytest.mark.parametrize("wide,mean", [(2.0 ** -30, 1.0), (2.0 ** 24, 1.0), (2.0 ** -18, 0.0), (2.0 ** 30, 2.0 ** -20)])
def test_decode_weights_of_any_size(dtype, rk, rv, wide, mean):
    """Small weights over large latents and the reverse are the same keys: the folded query keeps its
    digits whatever its size."""
    x = _inputs([150, 700, 1], 4, rk, rv, 16, dtype, 33, scale=1.0 / wide)
    x = dict(x, wk=(x["wk"].double() * wide).to(_sd(dtype)), mk=x["mk"] * mean)
    _check(x, 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("wide", [2.0 ** 12, 2.0 ** 20, 2.0 ** 32])
def test_decode_scores_of_any_size(dtype, sign, wide):
    """Scores of thousands to 10^10: the largest takes all of the weight.  Keys are one mean per head,
    its share by a latent, so the scores have one sign; the two best are a tenth apart at least."""
    L, rk, rv = 700, 32, 48
    x = _inputs([L], 2, rk, rv, 16, dtype, 35, T=1)
    # one rotation angle for all positions (a table of one row), a key of length c_0 along the query
    q, rows = widen(x["q"])[0], x["pool"][x["table"][0, np.arange(L) // 16], :, np.arange(L) % 16]
    order = np.random.default_rng(4).permutation(L)
    for h in range(2):
        ck = np.zeros((L, rk), np.float32)
        ck[:, 0] = np.where(order == 0, 1.0, 0.5 + 0.4 * order / L) if sign > 0 else np.where(order == 0, 0.5, 0.6 + 0.4 * order / L)
        for j in range(L):
            row = np.frombuffer(q4.row_of(ck[j], q4.values_of(rows[j, h].tobytes(), rk, rv)[1].astype(np.float32)), np.uint8)
            x["pool"][x["table"][0, j // 16], h, j % 16] = row
    wk = np.zeros((1, 2, 128, rk))
    wk[0, :, :, 0] = sign * wide * np.sign(q)
    x = dict(x, wk=torch.from_numpy(wk).to(_sd(dtype)), mk=torch.zeros(2, 128))
    dm = _dims(1, 2, rk, rv, dtype)
    cos, sin = torch.ones(704, 64, device="cuda"), torch.zeros(704, 64, device="cuda")
    ws = lla.q4_workspace(dm, 1, 704)
    out, lse = torch.empty(1, 2, 128, dtype=_sd(dtype), device="cuda"), torch.empty(1, 2, device="cuda")
    c = lambda v: torch.as_tensor(v).cuda()  # noqa: E731
    lla.decode_attn_q4(dm, 0, c(x["q"]), c(x["pool"]), c(x["table"]), c(x["lens"]), c(x["q_pos"]), c(x["wk"]), c(x["wv"]),
                       c(x["mk"]), c(x["mv"]), cos, sin, out, lse, ws)
    assert lla.device_status(ws) == lla.LLA_OK
    best = int(np.flatnonzero(order == 0)[0])
    for h in range(2):
        vk, vv = q4.values_of(x["pool"][x["table"][0, best // 16], h, best % 16].tobytes(), rk, rv)
        want = widen(x["wv"])[0, h] @ vv + widen(x["mv"])[h]
        assert rel_err(out.double().cpu().numpy()[0, h], want) <= TOL[dtype]
        score = q[h] @ (widen(x["wk"])[0, h] @ vk) / math.sqrt(128)
        assert abs(float(lse[0, h]) - score) <= TOL[dtype] * abs(score)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_nan_stays_in_its_sequence_head(dtype):
    """A row whose scale is NaN makes its own (sequence, head) NaN and no other."""
    x = _inputs([200, 130, 64], 2, 96, 160, 16, dtype, 8)
    clean, _, _ = _gpu(x, 0)
    rb_scale = (96 + 160) // 2
    for at in (rb_scale, rb_scale + 2 * 3):                  # a K scale, then a V scale
        y = dict(x, pool=x["pool"].copy())
        y["pool"][y["table"][1, 40 // 16], 1, 40 % 16, at:at + 2] = 0xFF
        out, _, st = _gpu(y, 0)
        assert st == lla.LLA_OK and out[1, 1].isnan().all()
        keep = torch.ones(3, 2, dtype=torch.bool)
        keep[1, 1] = False
        assert torch.equal(out.cpu()[keep], clean.cpu()[keep])


def test_decode_reports_bad_values():
    """Lengths, positions and table entries outside their ranges are clamped and reported; no
    access leaves the pool."""
    for dtype in ("bf16", "f32"):
        x = _inputs([100, 50], 2, 96, 160, 16, dtype, 9)
        x["pool"][:] = 0x11
        x["pool"][..., 128:144] = 0
        for bad in (dict(lens=np.array([100, -4], np.int32)), dict(lens=np.array([100, 1 << 30], np.int32)),
                    dict(q_pos=np.array([-1, 49], np.int32)), dict(q_pos=np.array([99, 1 << 30], np.int32)),
                    dict(table=np.where(x["table"] == x["table"][0, 0], 10**6, x["table"]).astype(np.int32)),
                    dict(table=np.where(x["table"] == x["table"][1, 1], -7, x["table"]).astype(np.int32))):
            y = dict(x, **bad)
            out, _, st = _gpu(y, 0)
            assert st == lla.LLA_ERR_DEVICE_ARG, bad
            assert out.isfinite().all()


def test_decode_shared_pages_and_repeats():
    """Two sequences that name the same pages, and a second call on the same workspace, give the
    same bits; without lse the output is the same."""
    x = _inputs([250, 250], 4, 96, 160, 64, "bf16", 10)
    x["table"][1] = x["table"][0]
    x["q"][1] = x["q"][0]
    dm = _dims(2, 4, 96, 160)
    ws = lla.q4_workspace(dm, 2, x["table"].shape[1] * 64)
    a, la, _ = _gpu(x, 1, ws=ws)
    b, _, _ = _gpu(x, 1, ws=ws, lse=False)
    assert torch.equal(a, b) and torch.equal(a[0], a[1]) and torch.equal(la[0], la[1])
    _check(x, 1)


def test_decode_captured_graph_and_side_stream():
    """Captured once, replayed with other lengths, queries and rows; then on a side stream."""
    x = _inputs([300, 129, 40], 2, 96, 160, 16, "bf16", 12, max_pages=20)
    y = _inputs([17, 320, 0], 2, 96, 160, 16, "bf16", 13, max_pages=20)
    num = max(x["pool"].shape[0], y["pool"].shape[0])
    dm = _dims(2, 2, 96, 160)
    dev = {}
    for n in ("q", "table", "lens", "q_pos", "wk", "wv", "mk", "mv"):
        dev[n] = (torch.from_numpy(x[n]) if isinstance(x[n], np.ndarray) else x[n]).cuda()
    pool = torch.zeros((num,) + x["pool"].shape[1:], dtype=torch.uint8, device="cuda")
    pool[:x["pool"].shape[0]] = torch.from_numpy(x["pool"]).cuda()
    cos, sin = (v.cuda() for v in lla.rope_table(dm, 320))
    ws = lla.q4_workspace(dm, 3, 320)
    out, lse = torch.empty(3, 2, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 2, device="cuda")
    call = lambda stream=None: lla.decode_attn_q4(dm, 0, dev["q"], pool, dev["table"], dev["lens"], dev["q_pos"], dev["wk"],  # noqa: E731
                                                  dev["wv"], dev["mk"], dev["mv"], cos, sin, out, lse, ws, stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for case in (x, y, x):
        for n, d in dev.items():
            d.copy_(torch.from_numpy(case[n]) if isinstance(case[n], np.ndarray) else case[n])
        pool[:case["pool"].shape[0]] = torch.from_numpy(case["pool"]).cuda()
        graph.replay()
        torch.cuda.synchronize()
        ro, rl = _oracle(case, 0)
        assert rel_err(out.double().cpu().numpy(), ro) <= TOL["bf16"] and lse_err(lse.double().cpu().numpy(), rl) <= TOL["bf16"]
    kept = out.clone()
    out.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call(side)
    side.synchronize()
    assert torch.equal(out, kept) and lla.device_status(ws) == lla.LLA_OK


def test_decode_pool_past_32_bits():
    """Rows more than 2^32 bytes into the pool."""
    H, P, rb = 16, 256, 144
    num = (1 << 32) // (H * P * rb) + 3
    x = _inputs([300, 40], H, 96, 160, P, "bf16", 14, extra=0)
    order = np.array([num - 1, num - 2, 0])
    pool = torch.zeros((num, H, P, rb), dtype=torch.uint8, device="cuda")
    for i, p in enumerate(order):
        pool[int(p)] = torch.from_numpy(x["pool"][i]).cuda()
    table = order[np.maximum(x["table"], 0)].astype(np.int32)
    dm = _dims(2, H, 96, 160)
    cos, sin = (v.cuda() for v in lla.rope_table(dm, 512))
    ws = lla.q4_workspace(dm, 2, 512)
    out = torch.empty(2, H, 128, dtype=torch.bfloat16, device="cuda")
    c = lambda v: torch.as_tensor(v).cuda()  # noqa: E731
    lla.decode_attn_q4(dm, 1, c(x["q"]), pool, c(table), c(x["lens"]), c(x["q_pos"]), c(x["wk"]), c(x["wv"]), c(x["mk"]),
                       c(x["mv"]), cos, sin, out, None, ws)
    assert lla.device_status(ws) == lla.LLA_OK
    assert rel_err(out.double().cpu().numpy(), _oracle(x, 1)[0]) <= TOL["bf16"]


def test_decode_page_past_32_bits():
    """One page of more than 2^31 bytes: rows of zeros (score and value 0 without means) but for the
    last token, whose score outweighs all of them, so its value is the result."""
    rk = rv = 256
    L = (1 << 31) // q4.row_bytes(rk, rv) + 1000
    dm = _dims(1, 1, rk, rv)
    g = np.random.default_rng(3)
    q, wk, wv = (torch.from_numpy(g.standard_normal(s) * f).bfloat16()
                 for s, f in (((1, 1, 128), 1.0), ((1, 1, 128, rk), 1 / 16), ((1, 1, 128, rv), 1 / 16)))
    # the query and the token share a position, so the score is q . W c / sqrt(128): 60 for this c
    u = widen(q)[0, 0] @ widen(wk)[0, 0]
    ck, cv = u * (60 * math.sqrt(128) / (u @ u)), g.standard_normal(rv)
    row = np.frombuffer(q4.row_of(ck.astype(np.float32), cv.astype(np.float32)), np.uint8)
    pool = torch.zeros((1, 1, L, q4.row_bytes(rk, rv)), dtype=torch.uint8, device="cuda")
    pool[0, 0, L - 1] = torch.from_numpy(row.copy()).cuda()
    cos, sin = lla.rope_table_scaled(dm, L)
    ws = lla.q4_workspace(dm, 1, L)
    out, lse = torch.empty(1, 1, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 1, device="cuda")
    i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    zero = torch.zeros(1, 128, device="cuda")
    lla.decode_attn_q4(dm, 0, q.cuda(), pool, i([[0]]), i([L]), i([L - 1]), wk.cuda(), wv.cuda(), zero, zero, cos, sin,
                       out, lse, ws)
    assert lla.device_status(ws) == lla.LLA_OK
    vk, vv = q4.values(row[None], rk, rv)
    s = float(u @ vk[0]) / math.sqrt(128)
    assert s > 40                                              # exp(-40) of 7.5e6 zeros is 3e-11
    assert abs(float(lse) - s) <= TOL["bf16"] * s
    assert rel_err(out.double().cpu().numpy()[0, 0], widen(wv)[0, 0] @ vv[0]) <= TOL["bf16"]


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype,rk,rv,P", [("bf16", 96, 160, 16), ("f32", 48, 80, 24), ("bf16", 16, 32, 64)])
def test_serving_steps_together(dtype, rk, rv, P):
    """Prefill and two decode steps as a serving loop makes them: the plan on the GPU, the new
    tokens' latents from lla_encode, stored in 4 bits at the plan's slots, and attention with
    rows of a scaled table over everything stored; against the oracle on the same latents."""
    T, H, B = 2, 2, 4
    dm = _dims(T, H, rk, rv, dtype)
    sd = _sd(dtype)
    g = torch.Generator().manual_seed(rk)
    rnd = lambda std, *s: (torch.randn(*s, generator=g) * std)  # noqa: E731
    wdk, wdv = rnd((T * 128) ** -0.5, H, T * 128, rk).to(sd).cuda(), rnd((T * 128) ** -0.5, H, T * 128, rv).to(sd).cuda()
    wk, wv = rnd(rk ** -0.5, T, H, 128, rk).to(sd), rnd(rv ** -0.5, T, H, 128, rv).to(sd)
    mk, mv = rnd(0.3, H, T * 128), rnd(0.3, H, T * 128)
    scaling = lla.rope_scaling("by_parts", 4.0, 128)
    mp = 20 if P == 16 else 16
    cap = mp * P
    cos, sin = lla.rope_table_scaled(dm, max(cap, 128), scaling)
    num = 60
    perm = torch.randperm(num, generator=g).to(torch.int32).cuda()
    table = torch.full((B, mp), -1, dtype=torch.int32, device="cuda")
    pool = torch.full((num, H, P, lla.q4_row_bytes(dm)), 0xFF, dtype=torch.uint8, device="cuda")
    ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
    head = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = lla.q4_workspace(dm, B, cap)
    seen = [[] for _ in range(B)]
    for new in ([130, 1, 0, 77], [1, 1, 1, 1], [1, 0, 2, 1]):
        n = sum(new)
        plan = lla.PagePlan(B, n)
        plan(P, num, ctx, torch.tensor(new, dtype=torch.int32, device="cuda"), perm, table, head)
        assert plan.granted.tolist() == [1] * B
        x_k, x_v = rnd(1.0, n, H, T * 128).to(sd).cuda(), rnd(1.0, n, H, T * 128).to(sd).cuda()
        ck, cv = torch.empty(n, H, 1, rk, dtype=sd, device="cuda"), torch.empty(n, H, 1, rv, dtype=sd, device="cuda")
        every, zero = torch.arange(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
        lla.encode(dm, x_k, x_v, every, zero, wdk, wdv, mk.cuda(), mv.cuda(), ck, cv, lla.make_workspace(dm, n, 1, n))
        lla.q4_store(dm, ck.view(n, H, rk), cv.view(n, H, rv), plan.slots, pool, ws)
        start = plan.tok_start.tolist()
        for b in range(B):
            for i in range(start[b], start[b + 1]):
                seen[b].append([q4.row_of(ck[i, h, 0].float().cpu().numpy(), cv[i, h, 0].float().cpu().numpy()) for h in range(H)])
        ctx, head = plan.seq_lens.clone(), plan.counts[:1].clone()
        lens = ctx.cpu().numpy()
        assert lens.tolist() == [len(s) for s in seen]
        q = rnd(1.0, B, H, 128).to(sd)
        q_pos = (ctx - 1).clamp(min=0).to(torch.int32)
        out, lse = torch.empty(B, H, 128, dtype=sd, device="cuda"), torch.empty(B, H, device="cuda")
        lla.decode_attn_q4(dm, 1, q.cuda(), pool, table, ctx, q_pos, wk.cuda(), wv.cuda(), mk.cuda(), mv.cuda(), cos, sin,
                           out, lse, ws)
        assert lla.device_status(ws) == lla.LLA_OK and lla.device_status(plan.workspace) == lla.LLA_OK
        for b in range(B):
            for h in range(H):
                o, l = _attend(q[b, h].double().numpy(), int(q_pos[b]), [r[h] for r in seen[b]], rk, rv, wk[1, h].double().numpy(),
                               wv[1, h].double().numpy(), mk[h, 128:].double().numpy(), mv[h, 128:].double().numpy(),
                               q4.thetas(128, 10000.0, "by_parts", 4.0, 128))
                e = rel_err(out[b, h].double().cpu().numpy()[None], o[None]), lse_err(lse[b, h].double().cpu().numpy(), np.float64(l))
                assert max(e) <= TOL[dtype], (b, h, e)


def _attend(q, q_pos, rows, rk, rv, wk, wv, mk, mv, theta):
    """One sequence-head written out: reconstruct, rotate by theta * position, softmax, values."""
    if not rows:
        return np.zeros(128), -math.inf
    vals = [q4.values_of(r, rk, rv) for r in rows]
    rot = lambda x, p: np.concatenate([x[:64] * np.cos(p * theta) - x[64:] * np.sin(p * theta),  # noqa: E731
                                       x[:64] * np.sin(p * theta) + x[64:] * np.cos(p * theta)])
    qr = rot(q, q_pos)
    s = np.array([qr @ rot(wk @ c + mk, j) for j, (c, _) in enumerate(vals)]) / math.sqrt(128)
    p = np.exp(s - s.max())
    o = sum(pj * (wv @ v + mv) for pj, (_, v) in zip(p, vals)) / p.sum()
    return o, s.max() + math.log(p.sum())
