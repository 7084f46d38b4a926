"""Plain 64-bit statements of the operators at a step's two ends, for their tests: norms with rotary
positions, and the distribution that a row of logits and its filters leave."""
from __future__ import annotations

import numpy as np
import torch

import draft_reference


def norm_rotated(x, weight, eps, positions, inv_freq, interleaved, factor):
    """(y, size): the heads of x [T][H][D] over their root mean square, times weight, with their pairs
    turned, in fp64, and the sizes of what each element is summed from."""
    y = x.double().cpu()
    y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt()
    if weight is not None:
        y = y * weight.double().cpu()
    want, size = draft_reference.rotated(y, positions, inv_freq, interleaved, factor)
    return want, np.where(size > 0, size * factor, np.abs(want))


def quantised(values, kv):
    """Codes times scales, and scales, of fp64 rows by the cache's rules (a scale of 1 for zeros)."""
    top = 127.0 if kv == "int8" else 448.0
    scale = np.abs(values).max(-1) / top
    return np.where(scale > 0, scale, 1.0)


def distribution(x, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Probabilities [V] (fp64) that a row of logits leaves, None if nothing can be drawn."""
    x = np.where(np.isnan(x), -np.inf, np.asarray(x, dtype=np.float64))
    V, top = len(x), x.max()
    if top == -np.inf:
        return None
    if temperature == 0:
        w = np.zeros(V)
        w[int(np.argmax(x))] = 1.0
        return w
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(x == top, 1.0, np.exp((x - top) / np.float64(temperature)))
    order = np.argsort(-x, kind="stable")
    n = top_k if 0 < top_k < V else V
    kept = order[:n]
    if top_p < 1:
        upto = np.cumsum(w[kept])
        before = upto - w[kept]
        before[0] = 0.0
        stay = before < max(np.float64(top_p), 0.0) * upto[-1]
        stay[0] = True
        kept = kept[stay]
    if min_p > 0:
        kept = kept[w[kept] >= min(np.float64(min_p), 1.0)]
    out = np.zeros(V)
    out[kept] = w[kept] / w[kept].sum()
    return out


def drawn(p, u):
    """The first token whose running sum exceeds u; the last one with weight past all of them."""
    passed = np.nonzero(np.cumsum(p) > np.float64(u) * p.sum())[0]
    return int(passed[0]) if len(passed) else int(np.nonzero(p)[0][-1])


def as_double(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()
