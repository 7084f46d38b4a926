"""Cases that measure what a serving step does on either side of its attention over a paged KV cache: queries and keys
normalised, rotated and appended; cached rows read back; logits turned into the next tokens, or into the
probabilities that the verification of drafted tokens reads.

``own`` chooses what run() does: False computes each operator in its plain form (elementary torch
operations in 32 bits, 64 where 32 lose what matters), True makes the calls of paged_kv_cache_197_gb300.
"""
from __future__ import annotations

import math

import torch

own = False
DEV = "cuda"
FACTOR = 1.2079441541679836  # attention factor of frequencies stretched eightfold


# ------------------------------------------------------------------------------- cases
def _norm(name, T, Hq, Hkv, D, bs, rot, interleaved, kv, far, scaled, fused, weights):
    """T tokens of Hq / Hkv heads, each head normalised and the first `rot` of its D elements rotated; positions below
    `far`; `scaled`: long-context frequencies and factor; `fused`: q, k and v are slices of one projection's output;
    `weights`: the norms have learned weights."""
    return dict(name=name, op="norm", T=T, Hq=Hq, Hkv=Hkv, D=D, bs=bs, rot=rot, interleaved=interleaved, kv=kv, far=far,
                scaled=scaled, fused=fused, weights=weights)


def _gather(name, T, Hkv, D, bs, kv):
    """T cached tokens read back into dense rows, from whole blocks in any order."""
    return dict(name=name, op="gather", T=T, Hkv=Hkv, D=D, bs=bs, kv=kv)


def _logits(name, op, R, V, logits, k_max, p_min, p_max, m_max, greedy, masked, probs="fp32"):
    """R rows of V logits in fp32 or bf16.  top-k up to `k_max` (0: off), top-p within p_min .. p_max (1: off), min-p up to
    `m_max` (0: off); `greedy`: every fourth row has temperature 0; `masked`: every third row has forbidden tokens."""
    return dict(name=name, op=op, R=R, V=V, logits=logits, k_max=k_max, p_min=p_min, p_max=p_max, m_max=m_max,
                greedy=greedy, masked=masked, probs=probs)


def listed():
    return [
        # one request's decode step: launch and latency
        _norm("norm 1 token", 1, 32, 8, 128, 16, 128, False, "bf16", 8192, False, False, True),
        # a decode batch out of one fused projection, fp8 cache
        _norm("norm 256 tokens fp8", 256, 32, 8, 128, 32, 128, False, "fp8", 32768, False, True, True),
        # a prefill step at far positions with scaled frequencies
        _norm("norm 8192 tokens", 8192, 64, 8, 128, 16, 128, False, "bf16", 1 << 20, True, True, True),
        # an odd number of tokens, part of a small head, adjacent pairs, int8 cache
        _norm("norm 1003 part int8", 1003, 24, 8, 64, 16, 32, True, "int8", 131072, False, False, True),
        # one request's context, read back to be handed on
        _gather("gather 501 tokens", 501, 8, 128, 16, "bf16"),
        # a batch's contexts out of an fp8 cache
        _gather("gather 131072 tokens fp8", 131072, 8, 128, 32, "fp8"),
        # one request's next token with the usual three filters
        _logits("sample 1 row", "sample", 1, 32000, "fp32", 50, 0.95, 0.95, 0.0, False, False),
        # a serving batch with top-p, large vocabulary
        _logits("sample 64 rows", "sample", 64, 131072, "fp32", 0, 0.8, 0.99, 0.0, False, False),
        # mixed requests: bf16 logits, odd vocabulary, min-p, greedy rows, forbidden tokens
        _logits("sample 20 rows mixed", "sample", 20, 50021, "bf16", 1000, 0.9, 1.0, 0.1, True, True),
        # a chain of four drafts and its root: the target's rows for the verification
        _logits("probs 5 rows", "probs", 5, 32000, "fp32", 0, 0.9, 0.9, 0.0, False, False),
        # the same for a batch of 64 chains of six rows
        _logits("probs 384 rows", "probs", 384, 131072, "fp32", 0, 0.95, 0.95, 0.0, False, False),
        # the rows of 24 trees, bf16 on both sides, top-k and min-p
        _logits("probs 333 rows bf16", "probs", 333, 50021, "bf16", 64, 1.0, 1.0, 0.05, False, True, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "gather", "sample", "probs"])
    D, Hkv, bs = rng.choice([64, 128]), rng.choice([1, 2, 3, 8]), rng.choice([16, 32])
    kv = rng.choice(["bf16", "int8", "fp8"])
    if op == "norm":
        rot = rng.choice([D, D, D // 2, D // 4, 20])
        c = _norm("", _log(rng, 1, 8192), Hkv * rng.choice([1, 3, 4, 8]), Hkv, D, bs, rot, rng.choice([True, False]), kv,
                  rng.choice([4096, 131072, 1 << 20]), rng.choice([True, False]), rng.choice([True, False]), rng.random() < 0.8)
    elif op == "gather":
        c = _gather("", _log(rng, 1, 131072), Hkv, D, bs, kv)
    else:
        R = _log(rng, 1, 64 if op == "sample" else 384)
        V = max(2, min(_log(rng, 30, 200000), (64 if op == "sample" else 384) * 131072 // R))
        p_min = rng.choice([1.0, rng.uniform(0.1, 0.99)])
        c = _logits("", op, R, V, rng.choice(["fp32", "bf16"]), rng.choice([0, _log(rng, 1, V), _log(rng, 1, min(V, 100))]), p_min,
                    rng.uniform(p_min, 1.0), rng.choice([0.0, rng.uniform(0.001, 0.5)]), rng.choice([True, False]),
                    rng.choice([True, False]), rng.choice(["fp32", "bf16"]))
    del c["name"]
    return c


# ------------------------------------------------------------------------------ inputs
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def _quantised(x, kv):
    """[..][D] as 8-bit codes and one fp32 scale a row."""
    x = x.float()
    top = 127.0 if kv == "int8" else 448.0
    scale = x.abs().amax(-1) / top
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    y = x / scale[..., None]
    return (y.round().clamp(-127, 127).to(torch.int8) if kv == "int8" else y.clamp(-448, 448).to(torch.float8_e4m3fn)), scale


def _pool(g, N, Hkv, bs, D, kv):
    k, v = _randn(g, N, Hkv, bs, D), _randn(g, N, Hkv, bs, D)
    if kv == "bf16":
        return dict(k_cache=k, v_cache=v, k_scale=None, v_scale=None)
    (k, ks), (v, vs) = _quantised(k, kv), _quantised(v, kv)
    return dict(k_cache=k, v_cache=v, k_scale=ks, v_scale=vs)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return {"norm": _prepare_norm, "gather": _prepare_gather, "sample": _prepare_logits, "probs": _prepare_logits}[case["op"]](case, g)


def _prepare_norm(case, g):
    T, Hq, Hkv, D, bs = (case[k] for k in ("T", "Hq", "Hkv", "D", "bs"))
    # projections whose heads differ in size, as they do before a norm
    size = torch.exp(0.7 * torch.randn((T, Hq + 2 * Hkv, 1), generator=g, device=DEV))
    qkv = (torch.randn((T, Hq + 2 * Hkv, D), generator=g, device=DEV) * size).to(torch.bfloat16)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if not case["fused"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    n, N = case["rot"] // 2, T // bs + 3
    inv = 500000.0 ** (-torch.arange(n, dtype=torch.float64) / n)
    if case["scaled"]:
        inv = torch.where(inv * 8192 < 2 * math.pi, inv / 8, inv)
    inv = inv.to(DEV)
    # turns per position as 64-bit fractions, as the framework's table holds them
    table = (inv / (2 * math.pi) * 2.0 ** 64).round().to(torch.int64)
    weights = [1 + 0.3 * torch.randn(D, generator=g, device=DEV) if case["weights"] else None for _ in range(2)]
    return dict(case=case, q=q, k=k, v=v, inv=inv, table=table, factor=FACTOR if case["scaled"] else 1.0, eps=1e-6,
                q_weight=weights[0], k_weight=weights[1], positions=torch.randint(0, case["far"], (T,), generator=g, device=DEV),
                slots=torch.randperm(N * bs, generator=g, device=DEV)[:T].contiguous(),
                q_out=torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV), **_pool(g, N, Hkv, bs, D, case["kv"]))


def _prepare_gather(case, g):
    T, Hkv, D, bs = (case[k] for k in ("T", "Hkv", "D", "bs"))
    blocks = -(-T // bs)
    N = blocks + 3
    table = torch.randperm(N, generator=g, device=DEV)[:blocks]
    slots = (table[:, None] * bs + torch.arange(bs, device=DEV)).flatten()[:T].contiguous()
    out = [torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    return dict(case=case, slots=slots, k_out=out[0], v_out=out[1], **_pool(g, N, Hkv, bs, D, case["kv"]))


def _prepare_logits(case, g):
    R, V = case["R"], case["V"]
    rows = torch.arange(R, device=DEV)
    x = torch.randn((R, V), generator=g, device=DEV) * 2.2
    # a few likely tokens a row, from hardly above the others to far above them
    likely = (torch.randperm(V, generator=g, device=DEV)[:40] + torch.randint(0, V, (R, 1), generator=g, device=DEV)) % V
    lift = torch.rand((R, likely.shape[1]), generator=g, device=DEV) * 12 * torch.rand((R, 1), generator=g, device=DEV)
    x.scatter_(1, likely, x.gather(1, likely) + lift)
    if case["masked"]:
        hide = (torch.rand((R, V), generator=g, device=DEV) < 0.3) & (rows % 3 == 0)[:, None]
        hide[:, 0] = False
        x[hide] = -math.inf
    x = x.to(torch.float32 if case["logits"] == "fp32" else torch.bfloat16)

    def uniform(lo, hi):
        return lo + (hi - lo) * torch.rand(R, generator=g, device=DEV)

    s = dict(case=case, x=x, u=torch.rand(R, generator=g, device=DEV), temperature=uniform(0.5, 1.2), top_k=None, top_p=None, min_p=None)
    if case["greedy"]:
        s["temperature"][rows % 4 == 3] = 0.0
    if case["k_max"]:
        s["top_k"] = torch.randint(1, case["k_max"] + 1, (R,), generator=g, device=DEV, dtype=torch.int32)
    if case["p_min"] < 1:
        s["top_p"] = uniform(case["p_min"], case["p_max"])
    if case["m_max"]:
        s["min_p"] = uniform(0.0, case["m_max"])
    if case["op"] == "sample":
        s["out"] = dict(tokens=torch.empty(R, dtype=torch.int32, device=DEV), probs=torch.empty(R, device=DEV))
    else:
        s["out"] = torch.empty((R, V), dtype=torch.float32 if case["probs"] == "fp32" else torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------------------- one pass
def run(state):
    return {"norm": _run_norm, "gather": _run_gather, "sample": _run_sample, "probs": _run_probs}[state["case"]["op"]](state)


def _cache_outputs(s):
    """The caches as the values they hold (int8 codes times their scales)."""
    kc, vc, ks, vs = s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    if s["case"]["kv"] == "int8":
        return dict(k_cache=(kc * ks[..., None]).to(torch.bfloat16), v_cache=(vc * vs[..., None]).to(torch.bfloat16))
    return dict(k_cache=kc, v_cache=vc) if ks is None else dict(k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs)


def _normed(x, weight, eps):
    x = x.float()
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    return y if weight is None else y * weight


def _rotate(x, cos, sin, rot, interleaved):
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    y, z = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((y, z), -1).flatten(-2) if interleaved else torch.cat((y, z), -1)
    return torch.cat((r, x[..., rot:]), -1)


def _store(cache, scales, slots, rows, kv, bs):
    if kv != "bf16":
        rows, scale = _quantised(rows, kv)
        scales[slots // bs, :, slots % bs] = scale
    else:
        rows = rows.to(torch.bfloat16)
    kind = torch.int8 if kv == "fp8" else cache.dtype
    cache.view(kind)[slots // bs, :, slots % bs] = rows.view(kind)


def _run_norm(s):
    c = s["case"]
    if own:
        import paged_kv_cache_197_gb300 as pa
        pa.pa_norm_rotary_and_cache(s["q_out"], s["q"], s["k"], s["positions"], s["table"], s["eps"], query_weight=s["q_weight"],
                                    key_weight=s["k_weight"], interleaved=c["interleaved"], attention_factor=s["factor"],
                                    value=s["v"], k_cache=s["k_cache"], v_cache=s["v_cache"], slot_mapping=s["slots"],
                                    k_scale=s["k_scale"], v_scale=s["v_scale"])
        return dict(q=s["q_out"], **_cache_outputs(s))
    angle = s["positions"].double()[:, None, None] * s["inv"]  # far positions: 64 bits
    cos, sin = (angle.cos() * s["factor"]).float(), (angle.sin() * s["factor"]).float()
    q, k = _normed(s["q"], s["q_weight"], s["eps"]), _normed(s["k"], s["k_weight"], s["eps"])
    s["q_out"].copy_(_rotate(q, cos, sin, c["rot"], c["interleaved"]))
    _store(s["k_cache"], s["k_scale"], s["slots"], _rotate(k, cos, sin, c["rot"], c["interleaved"]), c["kv"], c["bs"])
    _store(s["v_cache"], s["v_scale"], s["slots"], s["v"].float(), c["kv"], c["bs"])
    return dict(q=s["q_out"], **_cache_outputs(s))


def _run_gather(s):
    if own:
        import paged_kv_cache_197_gb300 as pa
        pa.pa_gather_cache(s["k_out"], s["v_out"], s["k_cache"], s["v_cache"], s["slots"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return dict(k=s["k_out"], v=s["v_out"])
    bs = s["case"]["bs"]
    at = (s["slots"] // bs, slice(None), s["slots"] % bs)
    for name in ("k", "v"):
        cache, scale = s[name + "_cache"], s[name + "_scale"]
        if scale is None:
            s[name + "_out"].copy_(cache[at])
            continue
        x = (cache.view(torch.int8)[at].view(cache.dtype) if cache.dtype == torch.float8_e4m3fn else cache[at]).float()
        s[name + "_out"].copy_(x * scale[at][..., None])
    return dict(k=s["k_out"], v=s["v_out"])


def _weights(s):
    """The rows' weights relative to their largest, 0 for the tokens that are filtered out: in 64 bits, since a token near a
    border is kept or not."""
    x, V = s["x"].float(), s["case"]["V"]
    t = s["temperature"][:, None].double()
    top = x.amax(-1, keepdim=True)
    w = ((x.double() - top.double()) / torch.where(t > 0, t, torch.ones_like(t))).exp()
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    sorted_w, rank = w.gather(1, order), torch.arange(V, device=DEV)
    k = torch.full_like(t, V) if s["top_k"] is None else s["top_k"][:, None]
    keep = rank < torch.where(t > 0, k, torch.ones_like(k))
    sorted_w = sorted_w * keep
    if s["top_p"] is not None:
        upto = sorted_w.cumsum(-1)
        keep = keep & ((upto - sorted_w < s["top_p"][:, None].double() * upto[:, -1:]) | (rank == 0))
    if s["min_p"] is not None:
        keep = keep & (sorted_w >= s["min_p"][:, None].double())
    return torch.zeros_like(w).scatter(1, order, sorted_w * keep)


def _run_sample(s):
    """The tokens drawn, and their probabilities."""
    o = s["out"]
    if own:
        import paged_kv_cache_197_gb300 as pa
        pa.pa_sample_tokens(o["tokens"], s["x"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                            min_p=s["min_p"], probs_out=o["probs"])
        return o
    w = _weights(s)
    upto = w.cumsum(-1)
    token = (upto <= s["u"][:, None].double() * upto[:, -1:]).sum(-1, keepdim=True)
    o["tokens"].copy_(token[:, 0])
    o["probs"].copy_((w.gather(1, token) / upto[:, -1:])[:, 0])
    return o


def _run_probs(s):
    if own:
        import paged_kv_cache_197_gb300 as pa
        pa.pa_sampling_probs(s["out"], s["x"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
        return s["out"]
    w = _weights(s)
    s["out"].copy_(w / w.sum(-1, keepdim=True))
    return s["out"]


# ------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "norm":
        T, Hq, Hkv, D, e = case["T"], case["Hq"], case["Hkv"], case["D"], 2 if case["kv"] == "bf16" else 1
        scales = 0 if case["kv"] == "bf16" else 8 * Hkv
        return dict(bytes=T * (2 * D * (2 * Hq + 2 * Hkv) + 2 * Hkv * D * e + scales + 16) + 8 * (case["rot"] // 2) + (8 * D if case["weights"] else 0),
                    flops=T * (Hq + Hkv) * (4 * D + 3 * case["rot"]))
    if case["op"] == "gather":
        T, Hkv, D, e = case["T"], case["Hkv"], case["D"], 2 if case["kv"] == "bf16" else 1
        return dict(bytes=T * (2 * Hkv * (D * (e + 2) + (0 if case["kv"] == "bf16" else 4)) + 8),
                    flops=0 if case["kv"] == "bf16" else 2 * T * Hkv * D)
    R, V, e = case["R"], case["V"], 4 if case["logits"] == "fp32" else 2
    out = 8 if case["op"] == "sample" else V * (4 if case["probs"] == "fp32" else 2)
    return dict(bytes=R * (V * e + out + 20), flops=4 * R * V)


# ------------------------------------------------------------------------------ exact
def exact(case, seed):
    """run()'s outputs from the definitions, in 64 bits."""
    s = prepare(case, seed)
    return {"norm": _exact_norm, "gather": _exact_gather, "sample": _exact_logits, "probs": _exact_logits}[case["op"]](case, s)


def _exact_norm(case, s):
    """Each head over its root mean square; each pair as a complex number times the unit number of its angle."""
    half, bs = case["rot"] // 2, case["bs"]
    j = torch.arange(half, device=DEV)
    lo, hi = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + half)
    turn = torch.polar(torch.full_like(s["inv"], s["factor"]).expand(case["T"], half), s["positions"].double()[:, None] * s["inv"])

    def rotated(x, weight):
        y = x.double()
        y = y * torch.rsqrt((y * y).sum(-1, keepdim=True) / case["D"] + s["eps"])
        if weight is not None:
            y = y * weight.double()
        z = torch.complex(y[..., lo], y[..., hi]) * turn[:, None]
        y[..., lo], y[..., hi] = z.real, z.imag
        return y

    out = dict(q=rotated(s["q"], s["q_weight"]))
    for name, rows in (("k", rotated(s["k"], s["k_weight"])), ("v", s["v"].double())):
        cache, scale = s[name + "_cache"].float().double(), s[name + "_scale"]
        at = (s["slots"] // bs, slice(None), s["slots"] % bs)
        if scale is None:
            cache[at] = rows
            out[name + "_cache"] = cache
            continue
        scale, top = scale.double(), 127.0 if case["kv"] == "int8" else 448.0
        step = rows.abs().amax(-1) / top
        scale[at] = torch.where(step > 0, step, torch.ones_like(step))
        codes = rows / scale[at][..., None]
        cache[at] = codes.round() if case["kv"] == "int8" else codes.float().to(torch.float8_e4m3fn).double()
        if case["kv"] == "int8":
            out[name + "_cache"] = cache * scale[..., None]
        else:
            out[name + "_cache"], out[name + "_scale"] = cache, scale
    return out


def _exact_gather(case, s):
    """Block by block, through the tokens' places in it."""
    blocks, place = torch.div(s["slots"], case["bs"], rounding_mode="floor"), s["slots"].remainder(case["bs"])
    out = {}
    for name in ("k", "v"):
        x = s[name + "_cache"].float().double()
        if s[name + "_scale"] is not None:
            x = x * s[name + "_scale"].double()[..., None]
        out[name] = torch.stack([x[:, h].flatten(0, 1)[blocks * case["bs"] + place] for h in range(case["Hkv"])], 1)
    return out


def _exact_logits(case, s):
    """Row by row: the tokens in order of their probability, cut where each filter says, and the distribution over what is
    left."""
    R, V = case["R"], case["V"]
    probs = case["op"] == "probs"
    out = torch.zeros((R, V) if probs else R, dtype=torch.float64, device=DEV)
    tokens = torch.empty(R, dtype=torch.int32, device=DEV)
    temperature = s["temperature"].double().tolist()
    some = {n: None if s[n] is None else s[n].double().tolist() for n in ("top_k", "top_p", "min_p")}
    u = s["u"].double().tolist()
    for r in range(R):
        x = s["x"][r].double()
        order = torch.argsort(-x, stable=True)
        n = V
        if temperature[r] == 0:
            n, p = 1, torch.ones(1, dtype=torch.float64, device=DEV)
        else:
            if some["top_k"]:
                n = min(n, int(some["top_k"][r]))
            p = torch.softmax(x[order[:n]] / temperature[r], 0)
            if some["top_p"] and some["top_p"][r] < 1:
                # the first place where the sum has reached top_p is the last one kept
                n = min(n, int(torch.searchsorted(p.cumsum(0), some["top_p"][r])) + 1)
            if some["min_p"]:
                n = min(n, int((p / p[0] >= some["min_p"][r]).sum()))
            p = p[:n] / p[:n].sum()
        if probs:
            out[r, order[:n]] = p
        else:
            kept, place = torch.sort(order[:n])
            p = p[place]
            drawn = int((p.cumsum(0) > u[r]).to(torch.int8).argmax())
            tokens[r], out[r] = kept[drawn], p[drawn]
    return out if probs else dict(tokens=tokens, probs=out)
