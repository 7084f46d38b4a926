"""Plain 64-bit statements of the speculative-decoding operators, for their tests."""
from __future__ import annotations

import math

import numpy as np
import torch


# ---------------------------------------------------------------------------- rotary
def rotated(x, positions, inv_freq, interleaved, factor):
    """(y, size): x [T][H][D] with its pairs turned, in fp64, and |x| + |x'| of each element's
    pair (0 where nothing is rotated)."""
    x = x.double().cpu().numpy()
    half = len(inv_freq)
    a, b = ((np.arange(0, 2 * half, 2), np.arange(1, 2 * half, 2)) if interleaved
            else (np.arange(half), np.arange(half, 2 * half)))
    # whole turns removed with Python integers: 64 bits of a turn per position
    turns = [int(round(f / (2 * math.pi) * 2 ** 64)) for f in inv_freq]
    frac = np.array([[((int(p) * t) % 2 ** 64) / 2 ** 64 for t in turns] for p in positions])
    c, s = np.cos(2 * np.pi * frac)[:, None] * factor, np.sin(2 * np.pi * frac)[:, None] * factor
    y, size = x.copy(), np.zeros_like(x)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, size


# ------------------------------------------------------------------------------ tree
def tree_attention(q, k, v, k_cache, v_cache, k_scale, v_scale, tables, lens, starts, parents, scale, values=0.0, sums=0.0,
                   small=0.0):
    """(out, spread, taken): the attention, sum_t w_t |v_t|, and what cached values off by `values`
    relative, or 2^-31 of the cache's largest scale, scores off by `sums` times scale * sum |q||k|, and
    weights of cached tokens off by `small`, or lost, may change, all [T][Hq][D] fp64 (NaN in rows of no sequence)."""
    q, k, v = (t.double().cpu() for t in (q, k, v))
    T, Hq, D = q.shape
    Hkv, bs = k_cache.shape[1], k_cache.shape[2]
    G = Hq // Hkv
    out = torch.full((T, Hq, D), float("nan"), dtype=torch.float64)
    spread, taken = out.clone(), torch.zeros_like(out)
    tables, k_cache, v_cache = tables.cpu(), k_cache.cpu(), v_cache.cpu()

    def context(cache, scales, s, n):
        ids = tables[s, : -(-n // bs)].long()
        raw = cache[ids].float() if cache.dtype != torch.uint8 else cache[ids].view(torch.float8_e4m3fn).float()
        x = raw.double()
        if scales is not None:
            x = x * scales.cpu()[ids].double()[..., None]
        return x.permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :n]

    for s, n in enumerate(lens):
        a, b = starts[s], starts[s + 1]
        L = b - a
        if L == 0:
            continue
        sees = torch.zeros((L, L), dtype=torch.bool)
        for i in range(L):
            at = i
            while at >= 0:
                sees[i, at] = True
                at = parents[a + at]
        mask = torch.cat((torch.ones((L, n), dtype=torch.bool), sees), 1)
        kk = torch.cat((context(k_cache, k_scale, s, n), k[a:b].permute(1, 0, 2)), 1)
        vv = torch.cat((context(v_cache, v_scale, s, n), v[a:b].permute(1, 0, 2)), 1)
        for h in range(Hq):
            w = torch.softmax((q[a:b, h] @ kk[h // G].T * scale).masked_fill(~mask, -math.inf), -1)
            out[a:b, h] = w @ vv[h // G]
            spread[a:b, h] = w @ vv[h // G].abs()
            if values and n:
                vc = vv[h // G][:n].abs() * values + 2.0 ** -31 * _largest(v_scale, tables, lens)
                taken[a:b, h] += w[:, :n] @ vc
            taken[a:b, h] += w[:, :n].clamp(max=small) @ vv[h // G][:n].abs()
            if sums:
                # Scores off by e_t change a weight's logarithm by at most e_t + log sum w exp(e), which
                # is at most e_t + E' exp(E) with E' = sum w e, E = max e; so the weight by at most
                # w_t (e_t + E') exp(4 E) while E is below 0.2.
                e = sums * abs(scale) * (q[a:b, h].abs() @ kk[h // G].abs().T)
                assert e.max() < 0.2
                mean, grow = (w * e).sum(-1, keepdim=True), torch.exp(4 * e.amax(-1, keepdim=True))
                taken[a:b, h] += grow * ((w * (e + mean)) @ vv[h // G].abs())
    return out, spread, taken


def _largest(scales, tables, lens):
    """The largest scale of the sequences' cached tokens."""
    top, bs = 0.0, scales.shape[2]
    for s, n in enumerate(lens):
        ids = tables[s, : -(-n // bs)].long()
        if n:
            x = scales.cpu()[ids].abs().permute(1, 0, 2).reshape(scales.shape[1], -1)[:, :n]
            top = max(top, float(x.max()))
    return top


def random_parents(lens, gen, kind="tree"):
    """In-sequence parents of every row: chains, stars, random trees or forests."""
    out = []
    for L in lens:
        for i in range(L):
            if i == 0 or kind == "roots":
                out.append(-1)
            elif kind == "chain":
                out.append(i - 1)
            elif kind == "star":
                out.append(0)
            else:
                low = -1 if kind == "forest" else 0
                out.append(int(torch.randint(low, i, (1,), generator=gen)))
    return out


# ---------------------------------------------------------------------------- verify
def verify_tree(tokens, p, q, starts, parents, u, u_final, W, tables=None, lens=None, bs=16):
    """The walk by its definition: residual distributions one after another.  Lists."""
    p = p.double().cpu().numpy()
    q = None if q is None else q.double().cpu().numpy()
    p = np.where(p > 0, p, 0.0)
    q = None if q is None else np.where(q > 0, q, 0.0)
    V = p.shape[1]
    tokens_out, path, n_out, slots = [], [], [], [-1] * len(tokens)
    for s in range(len(starts) - 1):
        a, b = starts[s], starts[s + 1]
        if a == b:
            tokens_out.append([-1] * W)
            path.append([-1] * W)
            n_out.append(0)
            continue
        at, way, said = a, [a], []
        while True:
            left, mass, step = p[at].copy(), 1.0, None
            for r in range(at + 1, b):
                if parents[r] != at - a:
                    continue
                x = tokens[r]
                if 0 <= x < V:
                    drafted = 1.0 if q is None else q[at][x]
                    if float(u[r]) * mass * drafted < left[x]:
                        step = r
                        break
                if q is None:
                    if 0 <= x < V:
                        left[x] = 0.0
                else:
                    left = np.maximum(left - mass * q[at], 0.0)
                mass = left.sum()
            if step is None:
                break
            at = step
            way.append(at)
            said.append(tokens[at])
        if not left.sum() > 0:
            left = p[at].copy()
        total = left.sum()
        if not (total > 0 and np.isfinite(total)):
            said.append(-1)
        else:
            run = left.cumsum()
            over = np.nonzero((run > float(u_final[s]) * total) & (left > 0))[0]
            said.append(int(over[0]) if len(over) else int(np.nonzero(left > 0)[0][-1]))
        if tables is not None:
            for j, r in enumerate(way):
                pos = lens[s] + j
                slots[r] = tables[s][pos // bs] * bs + pos % bs
        tokens_out.append(said + [-1] * (W - len(said)))
        path.append(way + [-1] * (W - len(way)))
        n_out.append(len(way))
    return tokens_out, path, n_out, slots
