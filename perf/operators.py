"""Cases that measure the operators of one speculative-decoding step over a paged KV cache: rotary positions
with the append, attention of a tree of drafted tokens, and the verification of the drafts.

``own`` chooses what run() does: False computes each operator in its plain form (elementary torch
operations in 32 bits, 64 where 32 lose what matters), True makes the calls of paged_kv_cache_197_gb300.
"""
from __future__ import annotations

import math

import torch

own = False
DEV = "cuda"


# ------------------------------------------------------------------------------- cases
def _rotary(name, T, Hq, Hkv, D, bs, rot, interleaved, kv, far, scaled, fused):
    """T tokens of Hq / Hkv heads; the first `rot` of D elements rotated; positions below `far`; `scaled`: long-context
    frequencies and factor; `fused`: q, k and v are slices of one projection's output."""
    return dict(name=name, op="rotary", T=T, Hq=Hq, Hkv=Hkv, D=D, bs=bs, rot=rot, interleaved=interleaved, kv=kv,
                far=far, scaled=scaled, fused=fused)


def _tree(name, S, L, L_min, Hq, Hkv, D, bs, ctx_min, ctx_max, kv):
    """S trees of L_min .. L nodes over contexts of ctx_min .. ctx_max cached tokens."""
    return dict(name=name, op="tree", S=S, L=L, L_min=L_min, Hq=Hq, Hkv=Hkv, D=D, bs=bs, ctx_min=ctx_min, ctx_max=ctx_max, kv=kv)


def _verify(name, S, L, L_min, V, probs, drafter, chain):
    """S trees (or chains) of L_min .. L rows over V tokens; probabilities in fp32 or bf16, with or without the
    drafter's."""
    return dict(name=name, op="verify", S=S, L=L, L_min=L_min, V=V, probs=probs, drafter=drafter, chain=chain)


def listed():
    return [
        # one request's decode step: launch and latency
        _rotary("rotary 1 token", 1, 32, 8, 128, 16, 128, False, "bf16", 8192, False, False),
        # a decode batch out of one fused projection, fp8 cache
        _rotary("rotary 256 tokens fp8", 256, 32, 8, 128, 32, 128, False, "fp8", 32768, False, True),
        # a prefill step at far positions with scaled frequencies
        _rotary("rotary 8192 tokens", 8192, 64, 8, 128, 16, 128, False, "bf16", 1 << 20, True, True),
        # an odd number of tokens, part of a small head, adjacent pairs
        _rotary("rotary 1003 part", 1003, 24, 8, 64, 16, 32, True, "bf16", 131072, False, False),
        # one request with a few drafts on a short context: launch and latency
        _tree("tree 8 nodes", 1, 8, 8, 32, 8, 128, 16, 501, 501, "bf16"),
        # a 70B-shaped batch of long contexts with small trees
        _tree("tree 16 nodes 70b", 20, 16, 16, 64, 8, 128, 16, 8000, 8000, "bf16"),
        # an 8B-shaped batch, ragged contexts, large trees
        _tree("tree 64 nodes ragged", 16, 64, 33, 32, 8, 128, 16, 700, 8191, "bf16"),
        # the same kind of batch on an fp8 cache
        _tree("tree 16 nodes fp8", 64, 16, 9, 32, 8, 128, 32, 128, 4096, "fp8"),
        # one request, a chain of four drafts: launch and latency
        _verify("verify chain", 1, 5, 5, 32000, "fp32", True, True),
        # a serving batch of chains, large vocabulary
        _verify("verify 64 chains", 64, 6, 2, 131072, "fp32", True, True),
        # trees of a drafter that proposes its best tokens: no draft probabilities, odd vocabulary
        _verify("verify 16 trees", 16, 48, 20, 50021, "fp32", False, False),
        # sampled trees with bf16 probabilities
        _verify("verify 24 trees bf16", 24, 32, 9, 131072, "bf16", True, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "tree", "verify"])
    if op == "rotary":
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 3, 8])
        rot = rng.choice([D, D, D // 2, D // 4, 20])
        c = _rotary("", _log(rng, 1, 8192), Hkv * rng.choice([1, 3, 4, 8]), Hkv, D, rng.choice([16, 32]), rot,
                    rng.choice([True, False]), rng.choice(["bf16", "int8", "fp8"]), rng.choice([4096, 131072, 1 << 20]),
                    rng.choice([True, False]), rng.choice([True, False]))
    elif op == "tree":
        Hkv, G = rng.choice([1, 2, 8]), rng.choice([1, 3, 4, 8])
        S, L = _log(rng, 1, 32), _log(rng, 1, 96)
        hi = max(1, min(8191, _log(rng, 1, 24000) // S))
        c = _tree("", S, L, rng.randint(1, L), Hkv * G, Hkv, rng.choice([64, 128]), rng.choice([16, 32]),
                  rng.randint(0, hi), hi, rng.choice(["bf16", "int8", "fp8"]))
    else:
        S, L = _log(rng, 1, 48), _log(rng, 1, 48)
        c = _verify("", S, L, rng.randint(1, L), max(2, min(_log(rng, 30, 200000), 50_000_000 // (S * L))),
                    rng.choice(["fp32", "bf16"]), rng.choice([True, False]), rng.choice([True, False]))
    del c["name"]
    return c


# ------------------------------------------------------------------------------ inputs
def _spread(lo, hi, n):
    """n lengths spread evenly over lo .. hi: the same for every seed (their order is not)."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


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


def _inv_freq(case):
    """Angular frequencies of a base of 500000, slow ones stretched eightfold where the case is `scaled`."""
    n = case["rot"] // 2
    inv = 500000.0 ** (-torch.arange(n, dtype=torch.float64) / n)
    if case["scaled"]:
        inv = torch.where(inv * 8192 < 2 * math.pi, inv / 8, inv)
    return inv


def _parents(g, lens, chain):
    """In-sequence parents of all rows: the row before in a chain, else a node drawn towards the newer ones."""
    L = max(lens)
    i = torch.arange(L, device=DEV)
    if chain:
        p = (i - 1).expand(len(lens), L)
    else:
        u = torch.rand((len(lens), L), generator=g, device=DEV).sqrt()
        p = (u * i).floor().long().clamp(max=L)
        p = torch.minimum(p, (i - 1).clamp(min=0))
        p[:, 0] = -1
    keep = i[None, :] < _ints(lens, torch.int64)[:, None]
    return p[keep].to(torch.int32).contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return {"rotary": _prepare_rotary, "tree": _prepare_tree, "verify": _prepare_verify}[case["op"]](case, g)


def _prepare_rotary(case, g):
    T, Hq, Hkv, D, bs = (case[k] for k in ("T", "Hq", "Hkv", "D", "bs"))
    if case["fused"]:
        qkv = _randn(g, T, Hq + 2 * Hkv, D)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = _randn(g, T, Hq, D), _randn(g, T, Hkv, D), _randn(g, T, Hkv, D)
    N = T // bs + 3
    inv = _inv_freq(case).to(DEV)
    # turns per position as 64-bit fractions, as the framework's table holds them
    table = (inv / (2 * math.pi) * 2.0 ** 64).round().to(torch.int64)
    return dict(case=case, q=q, k=k, v=v, inv=inv, table=table, factor=1.2079441541679836 if case["scaled"] else 1.0,
                positions=torch.randint(0, case["far"], (T,), generator=g, device=DEV),
                slots=torch.randperm(N * bs, generator=g, device=DEV)[:T].contiguous(),
                q_out=torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV), **_pool(g, N, Hkv, bs, D, case["kv"]))


def _prepare_tree(case, g):
    S, Hq, Hkv, D, bs = (case[k] for k in ("S", "Hq", "Hkv", "D", "bs"))
    order = torch.randperm(S, generator=g, device=DEV)
    lens = _ints(_spread(case["ctx_min"], case["ctx_max"], S))[order].contiguous()
    nodes = _spread(case["L_min"], case["L"], S)
    start = _ints([sum(nodes[:i]) for i in range(S + 1)])
    T = sum(nodes)
    M = max(1, -(-case["ctx_max"] // bs))
    N = S * M
    return dict(case=case, q=_randn(g, T, Hq, D), k=_randn(g, T, Hkv, D), v=_randn(g, T, Hkv, D), lens=lens, start=start,
                parents=_parents(g, nodes, False), tables=torch.randperm(N, generator=g, device=DEV).view(S, M).int(),
                scale=D ** -0.5, out=torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV), workspace=[],
                **_pool(g, N, Hkv, bs, D, case["kv"]))


def _prepare_verify(case, g):
    S, V = case["S"], case["V"]
    nodes = _spread(case["L_min"], case["L"], S)
    start = _ints([sum(nodes[:i]) for i in range(S + 1)])
    T, L, bs = sum(nodes), max(nodes), 16
    first = start[:-1].long().repeat_interleave(_ints(nodes, torch.int64), output_size=T)
    parents = _parents(g, nodes, case["chain"])
    kind = torch.float32 if case["probs"] == "fp32" else torch.bfloat16
    p, q = torch.empty((T, V), dtype=kind, device=DEV), torch.empty((T, V), dtype=kind, device=DEV)
    step = max(1, 30_000_000 // V)
    for at in range(0, T, step):  # peaked rows, the drafter's near the target's
        x = torch.randn((min(step, T - at), V), generator=g, device=DEV) * 2.5
        p[at:at + step] = torch.softmax(x, -1)
        q[at:at + step] = torch.softmax(x + torch.randn(x.shape, generator=g, device=DEV) * 0.7, -1)
    up = first + parents.long().clamp(min=0)  # the row each token was drafted from
    tokens = torch.empty(T, dtype=torch.int64, device=DEV)
    for at in range(0, T, step):
        rows = q[up[at:at + step]].float()
        tokens[at:at + step] = torch.multinomial(rows, 1, generator=g)[:, 0]
    M = (700 + L) // bs + 1
    out = dict(tokens_out=torch.empty((S, L), dtype=torch.int32, device=DEV), path=torch.empty((S, L), dtype=torch.int32, device=DEV),
               n_out=torch.empty(S, dtype=torch.int32, device=DEV), slots=torch.empty(T, dtype=torch.int64, device=DEV))
    return dict(case=case, p=p, q=q if case["drafter"] else None, tokens=tokens.int(), parents=parents, start=start, L=L,
                u=torch.rand(T, generator=g, device=DEV), u_next=torch.rand(S, generator=g, device=DEV), bs=bs, N=S * M,
                lens=torch.randint(1, 700, (S,), generator=g, device=DEV, dtype=torch.int32),
                tables=torch.randperm(S * M, generator=g, device=DEV).view(S, M).int(), out=out)


# ------------------------------------------------------------------------- one pass
def run(state):
    return {"rotary": _run_rotary, "tree": _run_tree, "verify": _run_verify}[state["case"]["op"]](state)


def _cache_outputs(s):
    """The caches as the values they hold (int8 codes times their scales)."""
    kc, vc, ks, vs = s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    if s["case"]["kv"] == "int8":
        return dict(k_cache=(kc * ks[..., None]).to(torch.bfloat16), v_cache=(vc * vs[..., None]).to(torch.bfloat16))
    return dict(k_cache=kc, v_cache=vc) if ks is None else dict(k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs)


def _rows(cache, at):
    """Entries of a cache in fp32 (fp8 ones picked as bytes)."""
    return (cache.view(torch.int8)[at].view(cache.dtype) if cache.dtype == torch.float8_e4m3fn else cache[at]).float()


def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
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


def _run_rotary(s):
    c = s["case"]
    if own:
        import paged_kv_cache_197_gb300 as pa
        pa.pa_rotary_and_cache(s["q_out"], s["q"], s["k"], s["positions"], s["table"], interleaved=c["interleaved"],
                               attention_factor=s["factor"], value=s["v"], k_cache=s["k_cache"], v_cache=s["v_cache"],
                               slot_mapping=s["slots"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return dict(q=s["q_out"], **_cache_outputs(s))
    angle = s["positions"].double()[:, None, None] * s["inv"]  # far positions: 64 bits
    cos, sin = (angle.cos() * s["factor"]).float(), (angle.sin() * s["factor"]).float()
    s["q_out"].copy_(_rotate(s["q"], cos, sin, c["rot"], c["interleaved"]))
    _store(s["k_cache"], s["k_scale"], s["slots"], _rotate(s["k"], cos, sin, c["rot"], c["interleaved"]), c["kv"], c["bs"])
    _store(s["v_cache"], s["v_scale"], s["slots"], s["v"].float(), c["kv"], c["bs"])
    return dict(q=s["q_out"], **_cache_outputs(s))


def _run_tree(s):
    c = s["case"]
    S, L, Hq, Hkv, D, bs = (c[k] for k in ("S", "L", "Hq", "Hkv", "D", "bs"))
    if own:
        import paged_kv_cache_197_gb300 as pa
        if not s["workspace"]:  # a user's program keeps its workspace
            n = pa.pa_tree_workspace_size(S, s["q"].shape[0], Hq, Hkv, D, bs, pa.kv_dtype_of(s["k_cache"]), c["ctx_max"], L)
            s["workspace"].append(torch.empty(max(n, 1), dtype=torch.uint8, device=DEV))
        pa.pa_tree_attention(s["out"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["tables"], s["lens"],
                             s["start"], s["parents"], s["scale"], c["ctx_max"], L, workspace=s["workspace"][0],
                             k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["out"]
    start, lens, n = s["start"].long(), s["lens"].long(), c["ctx_max"]
    node = torch.arange(L, device=DEV)
    real = node < (start[1:] - start[:-1])[:, None]                                    # [S][L]
    rows = (start[:-1, None] + node).clamp(max=s["q"].shape[0] - 1)
    up = torch.where(real, s["parents"][rows].long(), torch.full_like(rows, -1))
    sees = torch.eye(L + 1, device=DEV).expand(S, -1, -1)[:, :L].clone()               # self, and a column for "none"
    link = torch.nn.functional.one_hot(torch.where(up < 0, torch.full_like(up, L), up), L + 1).float()
    link = torch.cat((link, torch.nn.functional.one_hot(torch.full((S, 1), L, device=DEV), L + 1).float()), 1)
    hops = torch.eye(L + 1, device=DEV) + link                                         # one hop or none
    for _ in range(max(1, L.bit_length())):                                            # 2, 4, 8, .. hops
        hops = (hops @ hops).clamp(max=1)
    sees = (hops[:, :L, :L] > 0) & real[:, None, :]

    def context(cache, scale):
        x = _rows(cache, s["tables"].long())                                           # [S][M][Hkv][bs][D]
        x = x if scale is None else x * scale[s["tables"].long()][..., None]
        return x.permute(0, 2, 1, 3, 4).reshape(S, Hkv, -1, D)[:, :, :n]

    def both(cache, scale, new):
        x = torch.cat((context(cache, scale), new.float()[rows].permute(0, 2, 1, 3)), 2)
        return x[:, :, None]

    q = s["q"].float()[rows].permute(0, 2, 1, 3).view(S, Hkv, Hq // Hkv, L, D)
    w = (q @ both(s["k_cache"], s["k_scale"], s["k"]).transpose(-1, -2)) * s["scale"]  # [S][Hkv][G][L][n + L]
    cached = (torch.arange(n, device=DEV) < lens[:, None])[:, None].expand(S, L, n)
    w = w.masked_fill(~torch.cat((cached, sees), 2)[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True)
    w = (w - torch.where(top.isinf(), torch.zeros_like(top), top)).exp()
    o = (w @ both(s["v_cache"], s["v_scale"], s["v"])) / w.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.reshape(S, Hq, L, D).permute(0, 2, 1, 3)[real].to(torch.bfloat16)


def _run_verify(s):
    """Borders and sums in 64 bits: a draft is kept or not, a token drawn or not."""
    if own:
        import paged_kv_cache_197_gb300 as pa
        o = s["out"]
        pa.pa_verify_tree(o["tokens_out"], o["path"], o["n_out"], s["tokens"], s["p"], s["start"], s["parents"], s["u"],
                          s["u_next"], draft_probs=s["q"], slot_mapping=o["slots"], block_tables=s["tables"],
                          context_lens=s["lens"], block_size=s["bs"], num_blocks=s["N"])
        return o
    S, L, T, bs = s["case"]["S"], s["L"], s["tokens"].shape[0], s["bs"]
    start, node = s["start"].long(), torch.arange(s["L"], device=DEV)
    real = node < (start[1:] - start[:-1])[:, None]
    rows = (start[:-1, None] + node).clamp(max=T - 1)
    tokens, up, u = s["tokens"][rows].long(), s["parents"][rows].long(), s["u"][rows].double()
    here = torch.zeros(S, dtype=torch.long, device=DEV)                # the node reached
    kept = (node == 0).expand(S, L) & real
    left, mass = s["p"][rows[:, 0]].double(), torch.ones(S, dtype=torch.float64, device=DEV)
    for i in range(1, L):  # a node is tested after its parent and its older siblings: one step a node, all sequences
        child = real[:, i] & (up[:, i] == here)
        x, at = tokens[:, i:i + 1], rows.gather(1, here[:, None])[:, 0]
        if s["q"] is None:
            rest = left.scatter(1, x, 0.0)
            wanted = u[:, i] * mass
        else:
            drafted = s["q"][at].double()
            rest = (left - mass[:, None] * drafted).clamp(min=0)
            wanted = u[:, i] * mass * drafted.gather(1, x)[:, 0]
        yes = child & (wanted < left.gather(1, x)[:, 0])
        no = child & ~yes
        left = torch.where(yes[:, None], s["p"][rows[:, i]].double(), torch.where(no[:, None], rest, left))
        mass = torch.where(yes, torch.ones_like(mass), torch.where(no, rest.sum(1), mass))
        here = torch.where(yes, torch.full_like(here, i), here)
        kept = kept | (yes[:, None] & (node == i))
    whole = s["p"][rows.gather(1, here[:, None])[:, 0]].double()
    left = torch.where((left.sum(1) > 0)[:, None], left, whole)        # nothing left: the target's own row
    run_sum = left.cumsum(1)
    last = (run_sum <= (s["u_next"].double() * run_sum[:, -1])[:, None]).sum(1)
    place = kept.cumsum(1) - 1
    n = kept.sum(1)
    spot = torch.where(kept, place, torch.full_like(place, L))         # column L: dropped
    none = torch.full((S, L + 1), -1, dtype=torch.long, device=DEV)
    path = none.scatter(1, spot, rows)[:, :L]
    spoken = none.scatter(1, torch.where(kept & (node > 0), place - 1, torch.full_like(place, L)), tokens)
    spoken = spoken.scatter(1, n[:, None] - 1, last[:, None])[:, :L]
    pos = s["lens"].long()[:, None] + place.clamp(min=0)
    slot = s["tables"].long().gather(1, (pos // bs).clamp(max=s["tables"].shape[1] - 1)) * bs + pos % bs
    return dict(tokens_out=spoken.int(), path=path.int(), n_out=n.int(), slots=torch.where(kept, slot, torch.full_like(slot, -1))[real])


# ------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "rotary":
        T, Hq, Hkv, D, e = case["T"], case["Hq"], case["Hkv"], case["D"], 2 if case["kv"] == "bf16" else 1
        scales = 0 if case["kv"] == "bf16" else 8 * Hkv
        return dict(bytes=T * (2 * D * (2 * Hq + 2 * Hkv) + 2 * Hkv * D * e + scales + 16) + 8 * (case["rot"] // 2),
                    flops=T * (Hq + Hkv) * case["rot"] * 3)
    if case["op"] == "tree":
        S, Hq, Hkv, D = (case[k] for k in ("S", "Hq", "Hkv", "D"))
        lens, nodes = sum(_spread(case["ctx_min"], case["ctx_max"], S)), _spread(case["L_min"], case["L"], S)
        # the order of the lengths is drawn: each context meets the mean number of nodes
        T, e = sum(nodes), 2 if case["kv"] == "bf16" else 1
        row = 2 * D * e + (0 if case["kv"] == "bf16" else 8)
        return dict(bytes=lens * Hkv * row + T * D * 2 * (2 * Hq + 2 * Hkv) + 4 * (T + lens // case["bs"]),
                    flops=4 * D * Hq * (lens * T / S + sum(n * min(n, 4) for n in nodes)))
    e, T = 4 if case["probs"] == "fp32" else 2, sum(_spread(case["L_min"], case["L"], case["S"]))
    # the last node's row of the target's probabilities, and of the drafter's where it has one
    return dict(bytes=case["S"] * case["V"] * e * (2 if case["drafter"] else 1) + T * (4 + 4 + 4 + 8 + 8 + 2 * e),
                flops=case["S"] * case["V"] * 3)


# ------------------------------------------------------------------------------ exact
def exact(case, seed):
    """run()'s outputs from the definitions, in 64 bits."""
    return {"rotary": _exact_rotary, "tree": _exact_tree, "verify": _exact_verify}[case["op"]](case, prepare(case, seed))


def _exact_rotary(case, s):
    """Each pair as a complex number times the unit number of its angle."""
    half, bs = case["rot"] // 2, case["bs"]
    j = torch.arange(half, device=DEV)
    lo, hi = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + half)
    turn = torch.polar(torch.full_like(s["inv"], s["factor"]).expand(case["T"], half), s["positions"].double()[:, None] * s["inv"])

    def rotated(x):
        y = x.double().clone()
        z = torch.complex(y[..., lo], y[..., hi]) * turn[:, None]
        y[..., lo], y[..., hi] = z.real, z.imag
        return y

    out = dict(q=rotated(s["q"]))
    for name, rows in (("k", rotated(s["k"])), ("v", s["v"].double())):
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


def _exact_tree(case, s):
    """Sequence by sequence: its context and the rows on each node's way to the root."""
    G, bs, out = case["Hq"] // case["Hkv"], case["bs"], torch.empty(s["out"].shape, dtype=torch.float64, device=DEV)
    start, lens, parents = s["start"].tolist(), s["lens"].tolist(), s["parents"].tolist()
    for i in range(case["S"]):
        a, b, n = start[i], start[i + 1], lens[i]
        own_rows = torch.zeros((b - a, b - a), dtype=torch.bool)
        for r in range(b - a):
            at = r
            while at >= 0:
                own_rows[r, at] = True
                at = parents[a + at]
        hide = ~torch.cat((torch.ones((b - a, n), dtype=torch.bool), own_rows), 1).to(DEV)
        blocks = s["tables"][i].long()[: max(1, -(-n // bs))]
        for h in range(case["Hkv"]):
            k, v = (_rows(x, (blocks, h)).double() for x in (s["k_cache"], s["v_cache"]))
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][blocks, h].double()[..., None], v * s["v_scale"][blocks, h].double()[..., None]
            k = torch.cat((k.flatten(0, 1)[:n], s["k"][a:b, h].double()))
            v = torch.cat((v.flatten(0, 1)[:n], s["v"][a:b, h].double()))
            for f in range(h * G, h * G + G):
                scores = (s["q"][a:b, f].double() @ k.T * s["scale"]).masked_fill(hide, -math.inf)
                out[a:b, f] = torch.softmax(scores, -1) @ v
    return out


def _exact_verify(case, s):
    """Sequence by sequence, down from the root: residual distributions as they are defined, one child after another."""
    S, L, bs = case["S"], s["L"], s["bs"]
    start, parents, tokens = s["start"].tolist(), s["parents"].tolist(), s["tokens"].tolist()
    u, lens, tables = s["u"].double().tolist(), s["lens"].tolist(), s["tables"].tolist()
    said, path, count, slots = [], [], [], [-1] * len(tokens)
    for i in range(S):
        a, b = start[i], start[i + 1]
        way, words, at = [a], [], a
        while True:
            dist, step = s["p"][at].double(), None
            for c in (r for r in range(at + 1, b) if parents[r] == at - a):
                x = tokens[c]
                if s["q"] is None:
                    chance, rest = float(dist[x]), dist.clone()
                    rest[x] = 0
                else:
                    d = s["q"][at].double()
                    chance, rest = float(dist[x]) / max(float(d[x]), 1e-300), (dist - d).clamp(min=0)
                if u[c] < chance:
                    step = c
                    break
                if float(rest.sum()) <= 0:  # nothing left: the target's own row
                    dist = s["p"][at].double()
                    break
                dist = rest / rest.sum()
            if step is None:
                break
            words, way, at = words + [tokens[step]], way + [step], step
        passed = dist.cumsum(0) > float(s["u_next"][i].double()) * dist.sum()
        words.append(int(passed.to(torch.int8).argmax()))
        for j, r in enumerate(way):
            slots[r] = tables[i][(lens[i] + j) // bs] * bs + (lens[i] + j) % bs
        said.append(words + [-1] * (L - len(words)))
        path.append(way + [-1] * (L - len(way)))
        count.append(len(way))
    return dict(tokens_out=_ints(said), path=_ints(path), n_out=_ints(count), slots=_ints(slots, torch.int64))
