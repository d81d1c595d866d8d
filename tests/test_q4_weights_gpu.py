"""The 4-bit decode where softmax weights, V scales and score sizes are far apart: attention
sinks above long tails, V outliers, scores of any size, scale groups of different size, keys
whose weights share a sign.

A table of cos = 1, sin = 0 leaves keys unrotated, so every score is set by its latent: with
W_up,k's column 0 along the query, score_j = g_h c_j,0 / sqrt(128).  The expected results are
written out in 64 bits on the values that the rows hold.
"""
import math

import numpy as np
import pytest
import torch

from lla_cases import TOL, rel_err, widen
from looped_transformer_cross_gb300 import lla
from oracle import q4

pytestmark = pytest.mark.gpu

LOG2 = math.log2(math.e)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from looped_transformer_cross_gb300 import build
    build.build()


def _bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16()


def _row_parts(codes, scales):
    """Bytes of signed codes [..., r] and of the bf16 scales [..., groups]."""
    r = codes.shape[-1]
    c = np.arange(r)
    w = ((codes + 8).astype(np.uint64) << (4 * ((c % 8) // 2) + 16 * (c % 2)).astype(np.uint64))
    w = w.reshape(*codes.shape[:-1], r // 8, 8).sum(-1).astype(np.uint32)
    return w.view(np.uint8), _bf16(scales).view(torch.uint8).numpy()


class Cache:
    """One sequence's rows [L][H], as pages of 64 tokens, and the values that they stand for."""

    def __init__(self, kc, ks, vc, vs, P=64):
        L, H, self.rk = kc.shape
        self.rv, self.H, self.L, self.P = vc.shape[-1], H, L, P
        (k, sk), (v, sv) = _row_parts(kc, ks), _row_parts(vc, vs)
        rows = np.concatenate([k, v, sk, sv], -1)
        rows = np.pad(rows, ((0, 0), (0, 0), (0, q4.row_bytes(self.rk, self.rv) - rows.shape[-1])))
        self.pages = -(-L // P)
        pool = np.full((self.pages * P,) + rows.shape[1:], 0xFF, np.uint8)
        pool[:L] = rows
        self.pool = np.ascontiguousarray(pool.reshape(self.pages, P, H, -1).transpose(0, 2, 1, 3))
        wide = lambda s, r: widen(_bf16(s)).repeat(32, -1)[..., :r]  # noqa: E731
        self.k, self.v = kc * wide(ks, self.rk), vc * wide(vs, self.rv)          # [L][H][r], fp64


def _decode(c, q, wk, wv, dtype, B):
    """B sequences that name the same rows, all with the query q [H][128]; their common result."""
    sd = torch.bfloat16 if dtype == "bf16" else torch.float32
    dm = lla.dims(1, c.H, c.rk, c.rv, dtype=lla.LLA_BF16 if dtype == "bf16" else lla.LLA_F32)
    cap = c.pages * c.P
    n = max(cap, 128)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.arange(c.pages, **i32).repeat(B, 1)
    lens, q_pos = torch.full((B,), c.L, **i32), torch.full((B,), c.L - 1, **i32)
    out, lse = torch.empty(B, c.H, 128, dtype=sd, device="cuda"), torch.empty(B, c.H, device="cuda")
    ws, mu = lla.q4_workspace(dm, B, cap), torch.zeros(c.H, 128, device="cuda")
    lla.decode_attn_q4(dm, 0, q.to(sd).cuda().repeat(B, 1, 1), torch.from_numpy(c.pool).cuda(), table, lens, q_pos,
                       wk.to(sd).cuda()[None], wv.to(sd).cuda()[None], mu, mu, torch.ones(n, 64, device="cuda"),
                       torch.zeros(n, 64, device="cuda"), out, lse, ws)
    assert lla.device_status(ws) == lla.LLA_OK
    # (sequences are cut into runs at different places: the order of the sums differs, not more)
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def _expect(c, q, wk, wv):
    out, lse = np.empty((c.H, 128)), np.empty(c.H)
    for h in range(c.H):
        s = c.k[:, h] @ (widen(wk)[h].T @ widen(q)[h]) / math.sqrt(128)
        m = s.max()
        p = np.exp(s - m)
        lse[h] = m + math.log(p.sum())
        out[h] = widen(wv)[h] @ (p @ c.v[:, h]) / p.sum()
    return out, lse


def _problem(scores, H, rk, rv, seed, v_scale=0.25, v_codes=None, gain=1.0):
    """Rows whose scores are close to `scores` [L] (log2 units) in every head, q, W_up,k and W_up,v.
    v_scale: [L] or [L][groups] or a number."""
    g = np.random.default_rng(seed)
    scores = np.asarray(scores, np.float64)
    L = len(scores)
    q = torch.from_numpy(g.standard_normal((H, 128))).bfloat16()
    wk = np.zeros((H, 128, rk))
    wk[:, :, 0] = gain * np.sign(widen(q))
    wk = torch.from_numpy(wk).bfloat16()
    wv = torch.from_numpy(g.standard_normal((H, 128, rv)) / math.sqrt(rv)).bfloat16()
    kc, ks = np.zeros((L, H, rk), np.int64), np.zeros((L, H, q4.groups(rk)))
    for h in range(H):
        unit = gain * np.abs(widen(q)[h]).sum() / math.sqrt(128) * LOG2      # score (log2) of a latent of 1
        kc[:, h, 0] = np.where(scores < 0, -7, 7)
        ks[:, h, 0] = np.abs(scores) / unit / 7
    vc = g.integers(1, 8, (L, H, rv)) if v_codes is None else v_codes        # a mean that is not zero
    vs = np.broadcast_to(np.asarray(v_scale, np.float64).reshape(-1, 1, 1) if np.ndim(v_scale) < 2 else
                         np.asarray(v_scale, np.float64)[:, None, :], (L, H, q4.groups(rv)))
    return Cache(kc, ks, vc, vs), q, wk, wv


# (r_k, r_v, H): 8, 8, 4, 2, 1 and 1 heads share a position's tile in the tensor-core kernel
GROUPS = [(16, 32, 8), (16, 256, 8), (48, 80, 4), (96, 160, 2), (96, 160, 1), (240, 64, 1)]


# Tolerance 2e-2 of the largest output (bf16), as for every decode.  What moves an output here: the
# sink's score, below 14 nats, by one f16 half step of Z and of nothing else (the table is exact):
# 14 * 2^-11 = 0.7 %; the output's own rounding 2^-9, the weights' 2^-11.
def _check(problem, dtype="bf16", B=160, lse_tol=None):
    got, lse = _decode(*problem, dtype, B)
    want, wl = _expect(*problem)
    assert np.isfinite(got).all()
    for b in (0, B // 3, B - 1):
        assert rel_err(got[b], want) <= TOL[dtype], (b, rel_err(got[b], want))
        assert np.abs(lse[b] - wl).max() <= (TOL[dtype] if lse_tol is None else lse_tol)


@pytest.mark.parametrize("rk,rv,H", GROUPS)
@pytest.mark.parametrize("above,L", [(12.0, 2500), (16.0, 4096), (18.0, 9000), (20.0, 4096)])
def test_sink_over_a_long_tail(rk, rv, H, above, L):
    """Token 0 far above thousands of others, its V zero: the result is the tail's."""
    g = np.random.default_rng(int(above) + rk)
    s = 0.3 * g.standard_normal(L)
    s[0] = above
    v = np.full(L, 0.25)
    v[0] = 0.0
    _check(_problem(s, H, rk, rv, rk + H, v_scale=v), B=160 if H > 1 else 40)


@pytest.mark.parametrize("rk,rv,H", GROUPS)
def test_sink_and_scores_that_rise_later(rk, rv, H):
    """The tail rises by eight bits after the first tile: weights far above their own warp's
    first maximum, far below the sink's."""
    L = 4096
    g = np.random.default_rng(rk + H)
    s = 12.5 + 0.2 * g.standard_normal(L)
    s[:128] = 4.5
    s[0] = 20.0
    v = np.full(L, 0.25)
    v[0] = 0.0
    _check(_problem(s, H, rk, rv, rk + H, v_scale=v))


@pytest.mark.parametrize("rk,rv,H", GROUPS[:1] + GROUPS[2:])
@pytest.mark.parametrize("at", [0, 2000, 4095])
def test_sink_anywhere(rk, rv, H, at):
    """The far token first, in the middle, last; its V as the others'."""
    s = 0.3 * np.random.default_rng(at).standard_normal(4096)
    s[at] = 15.0
    _check(_problem(s, H, rk, rv, rk + at))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_falling_scores(dtype):
    """Every tile's scores lie ten bits below the last one's, and the other way round."""
    L = 1500
    for sign in (1.0, -1.0):
        s = sign * (np.arange(L) // 128 * 10.0 - 50.0)
        # scores reach 50 log2 = 35 nats: a Z half step moves them by 35 * 2^-11 = 0.017 each
        p = _problem(s, 2, 32, 64, 3)
        got, lse = _decode(*p, dtype, 9)
        want, wl = _expect(*p)
        assert rel_err(got[0], want) <= TOL[dtype] and np.abs(lse[0] - wl).max() <= max(TOL[dtype], 35 * 2.0 ** -20)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rk,rv,H", GROUPS)
@pytest.mark.parametrize("size,below,L", [(14, 40.0, 2500), (16, 40.0, 2500), (30, 80.0, 700), (30, 80.0, 30), (60, 110.0, 40)])
def test_v_outlier_without_weight(dtype, rk, rv, H, size, below, L):
    """One early token with V 2^size above the others' and no weight to speak of."""
    s = 0.3 * np.random.default_rng(size).standard_normal(L)
    s[3] = -below
    v = np.full(L, 0.25)
    v[3] = 0.25 * 2.0 ** size
    # (the outlier adds 2^(size - below) <= 2^-24 of one token's share)
    _check(_problem(s, H, rk, rv, size, v_scale=v), dtype, B=40 if dtype == "bf16" else 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v_scale", [2.0 ** -20, 0.1, 0.3, 0.6, 3.0, 2.0 ** 20])
@pytest.mark.parametrize("size", [2.0 ** 22, 2.0 ** 26, 2.0 ** 30, 2.0 ** 35])
def test_large_scores_and_any_v_scale(dtype, v_scale, size):
    """Scores of 2^22 to 2^35: the best token's V is the result, whatever its scale."""
    L = 300
    g = np.random.default_rng(5)
    for sign in (1.0, -1.0):
        s = sign * size * (0.5 + 0.4 * g.permutation(L) / L)
        best = int(np.argmin(np.abs(s)) if sign < 0 else np.argmax(np.abs(s)))
        s[best] *= 1.2 if sign > 0 else 0.8
        p = _problem(s, 3, 32, 48, 6, v_scale=v_scale, gain=2.0 ** 20)
        got, lse = _decode(*p, dtype, 2)
        want, wl = _expect(*p)
        assert rel_err(got[0], want) <= TOL[dtype] and rel_err(got[1], want) <= TOL[dtype]
        assert (np.abs(lse[0] - wl) <= TOL[dtype] * np.abs(wl)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", [1, 2, 8])
@pytest.mark.parametrize("L", [1, 3, 40])
@pytest.mark.parametrize("step", [10.0, 21.0])
def test_v_groups_of_different_size(dtype, H, L, step):
    """Scale groups of V 2^step apart, each read by outputs of its own: every group keeps its
    digits.  (f16 keeps 11 bits down to 2^-14, the weights' largest is 2^7 at least.)"""
    rk, rv = 16, 64
    g = np.random.default_rng(L + H)
    vs = np.array([[0.3, 0.3 * 2.0 ** -step]]) * np.exp(0.3 * g.standard_normal((L, 2)))
    c, q, wk, wv = _problem(0.5 * g.standard_normal(L), H, rk, rv, 7, v_scale=vs)
    wv = wv.clone()
    wv[:, :64, 32:] = 0.0                                      # outputs 0..63 of group 0, 64..127 of group 1
    wv[:, 64:, :32] = 0.0
    got, _ = _decode(c, q, wk, wv, dtype, 3)
    want, _ = _expect(c, q, wk, wv)
    for part in (slice(0, 64), slice(64, 128)):
        assert rel_err(got[0][:, part], want[:, part]) <= TOL[dtype], part


@pytest.mark.parametrize("rk", [16, 32, 96, 160, 224, 240, 256])
def test_offset_of_columns_that_share_a_sign(rk):
    """Columns of W_up,k of one sign under codes of zero leave no trace in the score.

    One token, so lse is its score: code 1 in column 0 of every scale group, 7 in a column whose
    weights are zero, zeros elsewhere.  The score's terms have one sign and each carries one f16 half
    step of Z, 2^-11; sums with the codes' offset are up to 256 / 1 times larger in fp32
    (2^-23 a step): 2^-12 more covers four of them."""
    H, rv = 4, 32
    g = np.random.default_rng(rk)
    q = torch.from_numpy(g.standard_normal((H, 128))).bfloat16()
    wk = torch.from_numpy(np.sign(widen(q))[:, :, None] * (1.0 + 0.4 * g.random((H, 128, rk)))).bfloat16()
    kc = np.zeros((1, H, rk), np.int64)
    kc[..., 0::32] = 1
    kc[..., 15::32] = 7
    wk[:, :, 15::32] = 0.0
    wv = torch.from_numpy(g.standard_normal((H, 128, rv))).bfloat16()
    c = Cache(kc, np.full((1, H, q4.groups(rk)), 0.5), g.integers(-7, 8, (1, H, rv)), np.full((1, H, 1), 0.25))
    got, lse = _decode(c, q, wk, wv, "bf16", 2)
    want, wl = _expect(c, q, wk, wv)
    assert (np.abs(lse - wl) <= np.abs(wl) * (2.0 ** -11 + 2.0 ** -12)).all(), np.abs(lse / wl - 1).max()
    assert rel_err(got[0], want) <= TOL["bf16"]
