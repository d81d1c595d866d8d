"""Plain statements of the 4-bit latent cache, the page plan and the RoPE operators (numpy,
64 bits, loops written out); shares no code with the library.

4-bit rows: per 32 columns scale = bf16(max|c| / 7) (fp32 quotient), code = round half even
of the fp32 quotient c / scale, clamped to [-7, 7]; zeros have scale 0, a group with a
value that is not finite reads as NaN.  Row bytes: K codes, V codes, K scales, V scales
(bf16), zeros up to a multiple of 16; column c of a 32-bit word of eight is bits
4(c//2) + 16(c%2) .. +3 as code + 8.
"""
import math

import numpy as np


def bf16_bits(x) -> int:
    """Bits of an fp32 value rounded to bf16 (half to even; NaN stays NaN)."""
    u = int(np.float32(x).view(np.uint32))
    if (u & 0x7FFFFFFF) > 0x7F800000:
        return 0x7FC0
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16) & 0xFFFF


def bf16_value(bits: int) -> float:
    return float(np.uint32(bits << 16).view(np.float32))


def groups(r: int) -> int:
    return (r + 31) // 32


def row_bytes(r_k: int, r_v: int) -> int:
    return (r_k // 2 + r_v // 2 + 2 * (groups(r_k) + groups(r_v)) + 15) // 16 * 16


def round_latent(c):
    """(codes, scale bits) of one latent (fp32 values), group by group."""
    codes, scales = [], []
    for g in range(0, len(c), 32):
        x = np.asarray(c[g:g + 32], np.float32)
        if not np.all(np.isfinite(x)):
            scales.append(0x7FC0)
            codes += [0] * len(x)
            continue
        bits = bf16_bits(np.float32(np.abs(x).max()) / np.float32(7))
        s = np.float32(bf16_value(bits))
        scales.append(bits)
        codes += [0 if s == 0 else int(min(7, max(-7, np.rint(np.float32(v) / s)))) for v in x]
    return codes, scales


def row_of(c_k, c_v) -> bytes:
    """The stored row of one token-head."""
    out, tail = b"", b""
    for c in (c_k, c_v):
        codes, scales = round_latent(c)
        for w in range(0, len(codes), 8):
            word = 0
            for i, q in enumerate(codes[w:w + 8]):
                word |= (q + 8) << (4 * (i // 2) + 16 * (i % 2))
            out += int(word).to_bytes(4, "little")
        for b in scales:
            tail += int(b).to_bytes(2, "little")
    out += tail
    return out + bytes(row_bytes(len(c_k), len(c_v)) - len(out))


def values_of(row, r_k: int, r_v: int):
    """The K and V latents (fp64) that a stored row stands for."""
    row = bytes(row)
    res, at, sat = [], 0, (r_k + r_v) // 2
    for r in (r_k, r_v):
        v = np.empty(r)
        for c in range(r):
            word = int.from_bytes(row[at + 4 * (c // 8): at + 4 * (c // 8) + 4], "little")
            code = ((word >> (4 * ((c % 8) // 2) + 16 * (c % 2))) & 15) - 8
            s = bf16_value(int.from_bytes(row[sat + 2 * (c // 32): sat + 2 * (c // 32) + 2], "little"))
            v[c] = code * s
        res.append(v)
        at += r // 2
        sat += 2 * groups(r)
    return res


def values(rows, r_k: int, r_v: int):
    """values_of over an array [..., row bytes] (vectorised over the leading dimensions)."""
    rows = np.asarray(rows, np.uint8)
    res, at, sat = [], 0, (r_k + r_v) // 2
    for r in (r_k, r_v):
        words = np.ascontiguousarray(rows[..., at:at + r // 2]).view("<u4")
        sc = np.ascontiguousarray(rows[..., sat:sat + 2 * groups(r)]).view("<u2").astype(np.uint32) << 16
        sc = sc.view(np.float32).astype(np.float64)
        c = np.arange(r)
        code = ((words[..., c // 8] >> (4 * ((c % 8) // 2) + 16 * (c % 2)).astype(np.uint32)) & 15).astype(np.int64) - 8
        with np.errstate(invalid="ignore"):
            res.append(code * sc[..., c // 32])
        at += r // 2
        sat += 2 * groups(r)
    return res


def page_plan(page_size, max_pages, num_pages, ctx, new, free, head, table, n_tok):
    """One step's plan, request by request; returns a dict of the outputs."""
    B, P = len(ctx), page_size
    table = np.array(table, np.int32).reshape(B, max_pages).copy()
    head = head if 0 <= head <= len(free) else len(free)
    out = dict(seq_lens=[], tok_start=[], granted=[], seq_idx=[-1] * n_tok, pos=[-1] * n_tok, slots=[-1] * n_tok)
    start, at, taken, live = 0, head, 0, 0
    for b in range(B):
        c, n = max(int(ctx[b]), 0), max(int(new[b]), 0)
        held = -(-c // P)
        fits = c + n <= max_pages * P and start + n <= n_tok
        need = -(-(c + n) // P) - held if fits else 0
        ok = fits and (need == 0 or at + need <= len(free))
        if ok:
            for i in range(need):
                table[b, held + i] = free[at + i]
            for i in range(n):
                p = int(table[b, (c + i) // P])
                out["seq_idx"][start + i], out["pos"][start + i] = b, c + i
                if 0 <= p < num_pages:
                    out["slots"][start + i] = p * P + (c + i) % P
            taken += need
            live += n
        out["seq_lens"].append(c + n if ok else c)
        out["granted"].append(int(ok))
        out["tok_start"].append(min(start, 2**31 - 1))
        start += n
        at += need          # a request that the pages do not reach still stands in the queue
    out["tok_start"].append(min(start, 2**31 - 1))
    out["counts"] = [head + taken, live]
    out["table"] = table
    return out


def thetas(d, base, kind="plain", factor=1.0, original_len=0, fast=32.0, slow=1.0):
    """Frequencies of a head of width d under a long-context scaling."""
    if kind == "base":
        base = base * factor ** (d / (d - 2))
    res = []
    for f in range(d // 2):
        t = base ** (-2.0 * f / d)
        if kind == "linear":
            t = t / factor
        if kind == "by_parts":
            turns = original_len * t / (2 * math.pi)
            g = min(1.0, max(0.0, (turns - slow) / (fast - slow)))
            t = (1 - g) * t / factor + g * t
        res.append(t)
    return np.array(res)


def rope_apply(x, pos, cos, sin, offset, style, scale=1.0, inverse=False):
    """Rotation of x [N][heads][d_x] (fp64) by table rows; pairs (f, f + half) or (2f, 2f + 1)."""
    y = np.array(x, np.float64)
    half = cos.shape[1]
    for f in range(half):
        i, j = (offset + f, offset + f + half) if style == 0 else (offset + 2 * f, offset + 2 * f + 1)
        c = cos[pos, f].astype(np.float64)[:, None]
        s = sin[pos, f].astype(np.float64)[:, None] * (-1 if inverse else 1)
        a, b = x[..., i].astype(np.float64), x[..., j].astype(np.float64)
        y[..., i], y[..., j] = scale * (a * c - b * s), scale * (a * s + b * c)
    return y
