"""Plain statements of the calls that verify drafted tokens (numpy, 64 bits, written out node by
node); shares no code with the library.

``tree_attn`` also bounds what the roundings to bf16 of a tensor-core evaluation may do to a
result.  Keys k^, queries q^ and weights p are each rounded once, by at most half a step (2^-8 of
the value), independently of each other; a rounding error is spread evenly over its step, so its
variance is at most (2^-8)^2 / 3 of the value's square.  To first order
    d s_j = sum_i (dq_i k_ij + q_i dk_ij) / sqrt d,   d out = sum_j p_j (d s_j + dp_j / p_j) (v_j - out)
(the weights are normalised by the sum of their rounded values), which gives the variances below;
the bound is six standard deviations, and half a step of the result itself where it is stored in
bf16.
"""
import math

import numpy as np

HALF = 2.0 ** -8          # half a step of bf16, relative to the value


def path_of(parent, i):
    """Node i and its ancestors (a parent that is not below its node counts as none)."""
    out = []
    while i >= 0:
        out.append(i)
        p = int(parent[i])
        i = p if -1 <= p < i else -1
    return out


def turn(x, cos, sin, style):
    """x [..., d] rotated by angles whose cosines and sines [..., d/2] are given."""
    h = x.shape[-1] // 2
    i0, i1 = (np.arange(h), np.arange(h) + h) if style == 0 else (2 * np.arange(h), 2 * np.arange(h) + 1)
    y = np.array(x, np.float64)
    y[..., i0], y[..., i1] = x[..., i0] * cos - x[..., i1] * sin, x[..., i0] * sin + x[..., i1] * cos
    return y


def tree_attn(q, k, v, tok_start, parent, pos, latents, w_k, w_v, mu_k, mu_v, cos, sin, style):
    """q, k, v [n_tok][H][d]; latents(b, h) -> (c_k [L][r_k], c_v [L][r_v]) of sequence b; w_k, w_v [H][d][r]
    and mu_k, mu_v [H][d] of the loop; cos, sin [rope_len][d/2].  Returns out [n_tok][H][d], lse
    [n_tok][H], and the bounds of both for a tensor-core evaluation (before out's own rounding);
    entries of no sequence stay NaN."""
    n_tok, H, d = q.shape
    out, lse = np.full((n_tok, H, d), np.nan), np.full((n_tok, H), np.nan)
    tol, tol_lse = np.zeros_like(out), np.zeros_like(lse)
    for b in range(len(tok_start) - 1):
        s0, n = int(tok_start[b]), int(tok_start[b + 1]) - int(tok_start[b])
        for h in range(H if n > 0 else 0):
            ck, cv = latents(b, h)
            L = len(ck)
            keys = turn(ck @ w_k[h].T + mu_k[h], cos[:L], sin[:L], style)
            vals = cv @ w_v[h].T + mu_v[h]
            p0 = [int(pos[s0 + i]) for i in range(n)]
            kd = turn(k[s0:s0 + n, h], cos[p0], sin[p0], style)
            for i in range(n):
                anc = path_of(parent[s0:s0 + n], i)
                kk = np.concatenate((keys, kd[anc]))
                vv = np.concatenate((vals, v[s0:s0 + n, h][anc]))
                qq = turn(q[s0 + i, h], cos[p0[i]], sin[p0[i]], style) / math.sqrt(d)
                s = kk @ qq
                m = s.max()
                p = np.exp(s - m)
                z = p.sum()
                p /= z
                o = p @ vv
                out[s0 + i, h], lse[s0 + i, h] = o, m + math.log(z)
                dv = vv - o
                own = ((qq * kk) ** 2).sum(1) + 1.0            # of s_j by its key, and of p_j
                var = (qq ** 2) @ ((p[:, None] * kk).T @ dv) ** 2 + (p ** 2 * own) @ dv ** 2
                tol[s0 + i, h] = 6 * HALF / math.sqrt(3) * np.sqrt(var)
                var = (qq ** 2) @ ((p[:, None] * kk).sum(0)) ** 2 + (p ** 2) @ own
                tol_lse[s0 + i, h] = 6 * HALF / math.sqrt(3) * math.sqrt(var)
    return out, lse, tol, tol_lse


def logits_adjust(logits, tok_start, parent, token, history, prompt_len, repetition, presence, frequency, bias, allowed):
    """logits [n_tok][V]; history[b]: list of tokens; bias[b]: list of (token, value); allowed[n]: set
    of tokens or None.  Returns x [n_tok][V] (64 bits), best, lse; rows of no sequence stay NaN / -2."""
    n_tok, V = logits.shape
    x, lse, best = np.full((n_tok, V), np.nan), np.full(n_tok, np.nan), np.full(n_tok, -2)
    for b in range(len(tok_start) - 1):
        s0, n = int(tok_start[b]), int(tok_start[b + 1]) - int(tok_start[b])
        for i in range(n):
            words = [int(token[s0 + a]) for a in path_of(parent[s0:s0 + n], i)]
            words += [int(t) for t in history[b][prompt_len[b]:]]
            prompt = {int(t) for t in history[b][:prompt_len[b]]}
            row = logits[s0 + i].astype(np.float64).copy()
            for t in (set(words) | prompt):
                if 0 <= t < V:
                    c = words.count(t)
                    row[t] = row[t] / repetition[b] if row[t] > 0 else row[t] * repetition[b]
                    row[t] -= frequency[b] * c
                    row[t] -= presence[b] if c else 0.0
            for t, val in bias[b]:
                if 0 <= t < V:
                    row[t] += val
            if allowed[s0 + i] is not None:
                off = np.ones(V, bool)
                off[sorted(allowed[s0 + i])] = False
                row[off] = -np.inf
            x[s0 + i] = row
            top = np.nanmax(row) if not np.all(np.isnan(row)) else -np.inf
            best[s0 + i] = int(np.flatnonzero(row == top)[0]) if top > -np.inf else -1
            if top == -np.inf:
                lse[s0 + i] = np.nan if np.isnan(row).any() else -np.inf
            else:
                lse[s0 + i] = top + math.log(np.exp(row - top).sum()) if np.isfinite(top) else top
    return x, best, lse


def tree_accept(tok_start, parent, token, chosen, ctx_lens):
    """Per sequence: (count, next token, length, entries of the path, slots of its entries)."""
    res = []
    for b in range(len(tok_start) - 1):
        s0, n = int(tok_start[b]), int(tok_start[b + 1]) - int(tok_start[b])
        ctx = max(0, int(ctx_lens[b]))
        path = [0] if n > 0 else []
        while path:
            cur = path[-1]
            nxt = [i for i in range(n) if int(parent[s0 + i]) == cur and i > cur and token[s0 + i] == chosen[s0 + cur]]
            if not nxt:
                break
            path.append(nxt[0])
        slot = {i: ctx + r for r, i in enumerate(path)}
        for i in range(n):
            slot.setdefault(i, ctx + len(slot))
        res.append((len(path), int(chosen[s0 + path[-1]]) if path else -1, ctx + len(path), [s0 + i for i in path],
                    [slot[i] for i in range(n)]))
    return res
