"""The speculative-decoding operators on the GPU against plain 64-bit statements of them: rotary positions
with the append, attention of a tree of drafted tokens, verification, and the three in a row."""
import math

import numpy as np
import pytest
import torch

import draft_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
HALF = {"bf16": 2.0 ** -8, "fp8": 2.0 ** -4}  # half a step of a type, relative to the value


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import paged_kv_cache_197_gb300 as pa

    pa.load_library()


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_197_gb300 as pa

    return pa


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g).to(torch.bfloat16).to(DEV)


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device=DEV)


def _flag():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _empty_cache(kv, N, Hkv, bs, D):
    if kv == "bf16":
        c = torch.full((2, N, Hkv, bs, D), float("nan"), dtype=torch.bfloat16, device=DEV)
        return dict(k_cache=c[0], v_cache=c[1])
    kind = torch.int8 if kv == "int8" else torch.uint8
    return dict(k_cache=torch.full((N, Hkv, bs, D), 77, dtype=kind, device=DEV),
                v_cache=torch.full((N, Hkv, bs, D), 77, dtype=kind, device=DEV),
                k_scale=torch.full((N, Hkv, bs), float("nan"), device=DEV),
                v_scale=torch.full((N, Hkv, bs), float("nan"), device=DEV))


def _values(cache):
    """Entries of a cache as fp64."""
    c = cache.cpu()
    return (c.view(torch.float8_e4m3fn) if c.dtype == torch.uint8 else c).float().double().numpy()


# ------------------------------------------------------------------------------ rotary
# The angle is rounded to 2^-33 turns and then to fp32 (half of 2^-24 half turns): below
# 2e-7 radians; sincospi is within 2 ulp (2.4e-7); the factor and the two products of an
# element round by 2^-24 each (1.8e-7).  Together below 2^-20 of (|x| + |x'|) * factor.
ROTARY = 2.0 ** -20


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("D,rot,interleaved,T,Hq,Hkv,bs", [
    (128, 128, False, 1, 32, 8, 16), (128, 128, True, 5, 8, 2, 32), (64, 64, False, 33, 3, 3, 16),
    (128, 64, False, 7, 5, 1, 16), (128, 32, True, 130, 6, 2, 32), (64, 20, False, 9, 4, 2, 16),
    (128, 100, False, 6, 17, 3, 16), (64, 2, False, 4, 2, 1, 32), (64, 6, True, 3, 1, 1, 16),
    (128, 128, False, 700, 64, 8, 16)])
def test_rotary(pa, D, rot, interleaved, T, Hq, Hkv, bs, kv):
    """Queries, keys and the appended cache rows, from slices of one projection's output, with padding
    tokens, at near, far and negative positions; everything else stays as it was."""
    g = _gen(D + rot + T)
    qkv = _randn(g, T, Hq + 2 * Hkv, D)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    inv = [10000.0 ** (-2 * j / rot) for j in range(rot // 2)]
    table = pa.pa_rotary_table(inv, DEV)
    far = [0, 1, -5, 8191, 1 << 20, (1 << 31) + 12345, (1 << 40) + 1]
    pos = [far[t % len(far)] if t < 14 else t for t in range(T)]
    factor = 1.25 if T % 2 else 1.0
    N = T // bs + 3
    slots = torch.randperm(N * bs, generator=g)[:T].to(DEV)
    if T > 3:
        slots[2] = -1
    q_out, k_out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV), torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=DEV)
    cache, flag = _empty_cache(kv, N, Hkv, bs, D), _flag()
    pa.pa_rotary_and_cache(q_out, q, k, torch.tensor(pos, device=DEV), table, interleaved=interleaved,
                           attention_factor=factor, key_out=k_out, value=v, slot_mapping=slots, err_flag=flag, **cache)
    torch.cuda.synchronize()
    assert flag.item() == 0
    want_q, size_q = ref.rotated(q, pos, inv, interleaved, factor)
    want_k, size_k = ref.rotated(k, pos, inv, interleaved, factor)
    for got, want, size in ((q_out, want_q, size_q), (k_out, want_k, size_k)):
        off = np.abs(_values(got) - want)
        assert (off <= HALF["bf16"] * np.abs(want) + ROTARY * factor * size).all(), off.max()
    kept = slots >= 0
    at = (slots[kept].cpu() // bs, slice(None), slots[kept].cpu() % bs)
    rest = torch.ones((N, bs), dtype=torch.bool)
    rest[at[0], at[2]] = False
    before = _empty_cache(kv, N, Hkv, bs, D)
    for name, c in cache.items():  # rows of no token are untouched, bit for bit
        bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[c.element_size()]
        x, y = (t.view(bits).cpu().transpose(1, 2)[rest] for t in (c, before[name]))
        assert torch.equal(x, y), name
    want, size = want_k[kept.cpu().numpy()], size_k[kept.cpu().numpy()]
    if kv == "bf16":
        plain = _empty_cache(kv, N, Hkv, bs, D)
        pa.pa_reshape_and_cache(k_out, v.contiguous(), plain["k_cache"], plain["v_cache"], slots)
        for name in cache:
            assert torch.equal(cache[name].view(torch.int16), plain[name].view(torch.int16)), name
        return
    plain = _empty_cache(kv, N, Hkv, bs, D)
    quantise = pa.pa_quantize_kv if kv == "int8" else pa.pa_quantize_kv_fp8
    quantise(k_out, v.contiguous(), plain["k_cache"], plain["v_cache"], plain["k_scale"], plain["v_scale"], slots)
    assert torch.equal(cache["v_cache"], plain["v_cache"])
    assert torch.equal(cache["v_scale"].view(torch.int32), plain["v_scale"].view(torch.int32))
    # keys: the scale is absmax / top of the rotated values (one more rounding, 2^-24), a code
    # half a step of value / scale
    top, err = (127.0 if kv == "int8" else 448.0), ROTARY * factor * size
    scale = cache["k_scale"].cpu().double().numpy()[at]
    want_scale = np.abs(want).max(-1) / top
    assert (np.abs(scale - want_scale) <= err.max(-1) / top + 2.0 ** -23 * want_scale).all()
    got = _values(cache["k_cache"])[at] * scale[..., None]
    # int8: half a step is scale / 2, and the quotient's rounding (2^-24 of up to 127) and the
    # scale's error (127 of its steps) may add to it; e4m3: half a step relative, or half of
    # 2^-9 below its smallest normal 2^-6
    if kv == "int8":
        bound = scale[..., None] * (0.5 + 127 * 2.0 ** -22) + 2 * err
    else:
        bound = HALF["fp8"] * np.abs(want) * (1 + 2.0 ** -20) + scale[..., None] * 2.0 ** -10 + 2 * err
    assert (np.abs(got - want) <= bound).all(), (np.abs(got - want) / bound).max()


@pytest.mark.parametrize("rot,interleaved", [(128, False), (100, False), (128, True)])
def test_rotary_in_place_and_without_a_cache(pa, rot, interleaved):
    """query_out is query and key_out is key: the same bits as out of place; no cache, no value."""
    g = _gen(rot)
    q, k = _randn(g, 50, 12, 128), _randn(g, 50, 4, 128)
    inv, _ = pa.pa_rotary_frequencies(rot, 500000.0, pa.PA_ROTARY_WAVELENGTH, 8.0, 8192, 1, 4)
    table, pos = pa.pa_rotary_table(inv, DEV), torch.arange(1000, 1050, device=DEV)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pa.pa_rotary_and_cache(qo, q, k, pos, table, interleaved=interleaved, key_out=ko)
    pa.pa_rotary_and_cache(q, q, k, pos, table, interleaved=interleaved, key_out=k)
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_rotary_turns_back(pa):
    """The rotation at -p undoes the one at p (each within half a bf16 step and the bound above)."""
    g = _gen(3)
    q, k = _randn(g, 20, 4, 64), _randn(g, 20, 2, 64)
    table, pos = pa.pa_rotary_table([0.9 ** j for j in range(32)], DEV), torch.arange(20, device=DEV) * 12345
    qo, ko, qb = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q)
    pa.pa_rotary_and_cache(qo, q, k, pos, table, key_out=ko)
    pa.pa_rotary_and_cache(qb, qo, ko, -pos, table, key_out=ko)
    x, back = q.double(), qb.double()
    size = x.abs() + x.roll(32, -1).abs()
    bound = HALF["bf16"] * x.abs() + (2 * HALF["bf16"] + 4 * ROTARY) * size  # the partner's rounding comes back too
    assert ((back - x).abs() <= bound).all()


def test_rotary_special_values_and_flags(pa):
    """Infinities and NaN behind rot_dim stay alone; a slot past the pool is flagged and not written; a
    negative zero that is not rotated keeps its sign."""
    g = _gen(4)
    q, k, v = _randn(g, 2, 2, 64), _randn(g, 2, 1, 64), _randn(g, 2, 1, 64)
    q[:, :, 40], q[:, :, 41], q[:, :, 42] = float("inf"), float("nan"), -0.0
    cache, flag = _empty_cache("bf16", 2, 1, 16, 64), _flag()
    qo = torch.empty_like(q)
    pa.pa_rotary_and_cache(qo, q, k, torch.tensor([3, 4], device=DEV), pa.pa_rotary_table([1.0] * 16, DEV), value=v,
                           slot_mapping=torch.tensor([32, 5], device=DEV), err_flag=flag, **cache)
    torch.cuda.synchronize()
    assert flag.item() == pa.PA_FLAG_SLOT_OUT_OF_RANGE
    assert torch.isfinite(qo[:, :, :32].float()).all()
    assert torch.equal(qo[:, :, 32:].view(torch.int16), q[:, :, 32:].contiguous().view(torch.int16))
    written = ~torch.isnan(cache["k_cache"].float()).any(-1)
    assert written.sum().item() == 1 and written[0, 0, 5]


def test_rotary_refuses_other_tensors(pa):
    g = _gen(5)
    q, k = _randn(g, 2, 4, 64), _randn(g, 2, 2, 64)
    pos, table = torch.arange(2, device=DEV), pa.pa_rotary_table([1.0] * 32, DEV)
    with pytest.raises(ValueError):
        pa.pa_rotary_and_cache(torch.empty_like(q), q.transpose(1, 2).contiguous().transpose(1, 2), k, pos, table, key_out=k)
    with pytest.raises(TypeError):
        pa.pa_rotary_and_cache(torch.empty_like(q), q, k, pos.int(), table, key_out=k)
    with pytest.raises(ValueError):
        pa.pa_rotary_and_cache(torch.empty_like(q), q, k, pos[:1], table, key_out=k)
    with pytest.raises(ValueError):  # a cache without slots
        pa.pa_rotary_and_cache(torch.empty_like(q), q, k, pos, table, value=k, **_empty_cache("bf16", 1, 2, 16, 64))
    with pytest.raises(pa.PagedAttentionError):  # more pairs than the head has
        pa.pa_rotary_and_cache(torch.empty_like(q), q, k, pos, pa.pa_rotary_table([1.0] * 33, DEV), key_out=k)


# -------------------------------------------------------------------------------- tree
def _tree_case(kv, D, bs, Hq, Hkv, lens, nodes, seed, kind="tree", before=0, behind=0, spare=2, wide=False):
    """Inputs of a tree call.  Cache slots of no token, rows of no sequence and unused blocks hold NaN
    (or NaN scales).  wide: key and value as slices of a wider tensor."""
    import paged_kv_cache_197_gb300 as pa

    g = _gen(seed)
    S, T = len(lens), before + sum(nodes) + behind
    starts = [before + sum(nodes[:s]) for s in range(S + 1)]
    need = [-(-n // bs) for n in lens]
    M = max(1, max(need)) + 1
    N = sum(need) + spare
    ids = torch.randperm(N, generator=g).tolist()
    tables = torch.full((S, M), 2 ** 30, dtype=torch.int32)  # entries past a context are never read
    slots = []
    for s in range(S):
        mine, ids = ids[: need[s]], ids[need[s]:]
        tables[s, : need[s]] = torch.tensor(mine, dtype=torch.int32)
        slots += [mine[t // bs] * bs + t % bs for t in range(lens[s])]
    cache = _empty_cache(kv, N, Hkv, bs, D)
    if kv != "bf16":  # codes of empty slots: any; their scales NaN
        cache["k_cache"].random_(-100, 100, generator=torch.Generator(DEV).manual_seed(seed)) if kv == "int8" else None
    if slots:
        rows = _randn(g, 2, len(slots), Hkv, D)
        at = torch.tensor(slots, device=DEV)
        if kv == "bf16":
            pa.pa_reshape_and_cache(rows[0], rows[1], cache["k_cache"], cache["v_cache"], at)
        else:
            (pa.pa_quantize_kv if kv == "int8" else pa.pa_quantize_kv_fp8)(
                rows[0], rows[1], cache["k_cache"], cache["v_cache"], cache["k_scale"], cache["v_scale"], at)
    parents = [-7] * before + ref.random_parents(nodes, g, kind) + [-9] * behind
    q = _randn(g, T, Hq, D)
    if wide:
        kv_rows = _randn(g, T, 2 * Hkv + 1, D)
        k, v = kv_rows[:, :Hkv], kv_rows[:, Hkv:2 * Hkv]
    else:
        k, v = _randn(g, T, Hkv, D), _randn(g, T, Hkv, D)
    for t in (q, k, v):
        t[:before] = float("nan")
        t[T - behind:] = float("nan")
    return dict(q=q, k=k, v=v, tables=tables.to(DEV), lens=lens, starts=starts, parents=parents, nodes=nodes, scale=D ** -0.5,
                cache=cache)


def _tree_call(pa, c, max_ctx=None, max_q=None, out=None, flag=None, workspace=None, stream=None):
    out = torch.full_like(c["q"], float("nan")) if out is None else out
    pa.pa_tree_attention(out, c["q"], c["k"], c["v"], c["cache"]["k_cache"], c["cache"]["v_cache"], c["tables"], _i32(c["lens"]),
                         _i32(c["starts"]), _i32(c["parents"]), c["scale"], max(c["lens"]) if max_ctx is None else max_ctx,
                         max(max(c["nodes"]), 1) if max_q is None else max_q, workspace=workspace,
                         k_scale=c["cache"].get("k_scale"), v_scale=c["cache"].get("v_scale"), err_flag=flag, stream=stream)
    return out


def _tree_reference(c):
    return _tree_taken(c)[:2]


def _tree_taken(c, values=0.0, sums=0.0, small=0.0):
    return ref.tree_attention(c["q"], c["k"], c["v"], c["cache"]["k_cache"], c["cache"]["v_cache"], c["cache"].get("k_scale"),
                              c["cache"].get("v_scale"), c["tables"], c["lens"], c["starts"], c["parents"], c["scale"], values, sums, small)


def _tree_check(out, c, sums=0.0, small=0.0):
    """The output is rounded to bf16 once (2^-8 of it), and each softmax weight once, to bf16 or fp16,
    before its product with v (2^-8 of sum w |v|; the sum of the weights takes them unrounded).
    Scores, exponentials and sums in fp32: |score| below 2^5 here, off by a few 2^-24 of it, is below
    2^-16 of a weight, ex2.approx 2^-22; together under 2^-12 of sum w |v|.  8-bit caches, heads of
    128: a value is off by 2^-11 for its scale's rounding and 2^-11 for its own (fp16).  sums: for larger
    scores, their error in units of scale * sum |q||k|, and small:
    what fp16 weights far below the largest are off by."""
    quant = "k_scale" in c["cache"] and c["q"].shape[2] == 128
    want, spread, taken = _tree_taken(c, 2.0 ** -10 * (1 + 2.0 ** -11) if quant else 0.0, sums, small)
    got = out.double().cpu()
    none = torch.isnan(want)
    assert torch.isnan(got[none]).all()  # rows of no sequence are not written
    off = (got - want).abs()[~none]
    bound = (2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * spread + taken)[~none]
    assert torch.isfinite(got[~none]).all()
    assert (off <= bound).all(), (off / bound).max().item()


HEADS = [(128, 16, 32, 8), (128, 32, 16, 2), (64, 16, 12, 4), (64, 32, 5, 5), (128, 16, 3, 1)]


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("D,bs,Hq,Hkv", HEADS)
def test_tree_small(pa, D, bs, Hq, Hkv, kv):
    """Contexts from nothing up with block edges on both sides, trees from one row up, rows of no sequence
    in front and behind, keys and values as slices."""
    c = _tree_case(kv, D, bs, Hq, Hkv, [0, 1, bs, bs + 1, 63, 64, 65, 300, 0], [1, 7, 3, 16, 1, 2, 33, 5, 4], D + Hq,
                   before=2, behind=3, wide=True)
    flag = _flag()
    out = _tree_call(pa, c, flag=flag)
    torch.cuda.synchronize()
    assert flag.item() == 0
    _tree_check(out, c)


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 32, 8), (64, 8, 2), (128, 2, 2)])
def test_tree_long_contexts(pa, D, Hq, Hkv, kv):
    """Split contexts: some sequences take one partition, some many, some none."""
    c = _tree_case(kv, D, 16, Hq, Hkv, [9000, 257, 0, 4097, 512], [17, 64, 5, 1, 31], 7 * D, kind="forest")
    _tree_check(_tree_call(pa, c), c)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("kind", ["tree", "chain", "star", "roots"])
@pytest.mark.parametrize("L", [127, 128, 129, 256])
def test_tree_large(pa, kind, L, kv):
    """The largest trees, deep and flat, on both sides of a tile of their rows."""
    c = _tree_case(kv, 128, 16, 8, 4, [200, 33], [L, 1], L, kind=kind)
    _tree_check(_tree_call(pa, c), c)


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (24, 2), (64, 1)])
def test_tree_head_layouts(pa, Hq, Hkv, kv):
    """One head per kv head, twelve, and 64 (several column blocks of one row)."""
    c = _tree_case(kv, 128, 32, Hq, Hkv, [700, 90], [9, 40], Hq)
    _tree_check(_tree_call(pa, c), c)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("L", [87, 88, 89, 94, 96, 97])
def test_tree_rows_at_the_staging_limit(pa, L, D):
    """Trees on both sides of the most rows whose own keys and values are kept on chip."""
    c = _tree_case("bf16", D, 16, 8, 2, [50, 0], [L, 3], L)
    _tree_check(_tree_call(pa, c), c)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
def test_tree_softmax_scales(pa, kv, D):
    """A negative scale, and 0: every token the same weight."""
    c = _tree_case(kv, D, 16, 12, 4, [300, 70, 129], [9, 30, 40], 23)
    for scale in (-(D ** -0.5), 0.0):
        c["scale"] = scale
        _tree_check(_tree_call(pa, c), c)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("kv", ["int8", "fp8"])
def test_tree_scales_of_all_sizes(pa, kv, D):
    """Scales of neighbouring tokens up to 2^18 apart, some of them 0 or negative."""
    c = _tree_case(kv, D, 16, 8, 2, [300, 70, 129, 1000], [9, 30, 40, 2], 29)
    g = _gen(1)
    for name in ("k_scale", "v_scale"):
        t = c["cache"][name]
        t *= (2.0 ** torch.randint(-18, 1, t.shape, generator=g)).to(DEV)
        t *= (torch.randint(0, 5, t.shape, generator=g) - 1).sign().to(DEV)
    _tree_check(_tree_call(pa, c), c)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("kv", ["int8", "fp8"])
def test_tree_scores_of_hundreds(pa, kv, D):
    """Keys up to 64 times as large as usual, token by token: scores of a few hundred, whose rounding shows
    in the weights.  A score is a sum of D products in fp32, in any order, D 2^-24 of sum |q||k|, and
    four more roundings (its token's scale, the row's factor, the exponent, and the key's own in the plain
    row); a rounding of the keys to 11 bits, 2^-12 at a time, would be ten times that.  fp16 weights below
    2^-14 have steps of 2^-24, so are off by 2^-25 of the largest, times at most 4 as they come in units
    of the tile's value scale (within a factor of four here)."""
    c = _tree_case(kv, D, 16, 8, 2, [300, 70, 1000], [9, 30, 2], 41)
    t = c["cache"]["k_scale"]
    t *= (2.0 ** torch.randint(0, 7, t.shape, generator=_gen(2))).to(DEV)
    _tree_check(_tree_call(pa, c), c, sums=(D + 4) * 2.0 ** -24, small=2.0 ** -23)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_tree_many_sequences(pa, kv):
    """More sequences than threads in a block, most of them short, some empty, in one call."""
    g = _gen(31)
    lens = torch.randint(0, 200, (700,), generator=g).tolist()
    nodes = torch.randint(0, 4, (700,), generator=g).tolist()
    c = _tree_case(kv, 128, 16, 4, 2, lens, nodes, 32)
    flag = _flag()
    out = _tree_call(pa, c, flag=flag)
    torch.cuda.synchronize()
    assert flag.item() == 0
    _tree_check(out, c)


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("L", [2, 70])
def test_tree_long_shares(pa, kv, L):
    """Dozens of tiles and several units to a block of threads, whatever the order of the lengths."""
    c = _tree_case(kv, 128, 32, 16, 4, [30000, 5, 20001, 640, 30000, 0, 128], [L, 3, 1, L, 4, 2, L], 37)
    _tree_check(_tree_call(pa, c), c)


def test_tree_empty_context_bound(pa):
    """max_context_len 0: the trees alone; a table that holds no valid block is not read."""
    c = _tree_case("bf16", 128, 16, 8, 2, [0, 0], [6, 20], 5)
    _tree_check(_tree_call(pa, c, max_ctx=0), c)


def test_tree_large_scores(pa):
    """Scores near +-400 in both parts: one part's weights vanish against the other's, nothing overflows."""
    for up in (3.0, -3.0):
        c = _tree_case("bf16", 128, 16, 4, 2, [300], [12], 9)
        c["k"].fill_(up)
        c["q"].fill_(1.0)
        want, spread = _tree_reference(c)
        got = _tree_call(pa, c).double().cpu()
        # scores of up to 384 * scale * log2 e = 49 in the exp2 domain: off by 2^-17 relative more
        assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -11) * spread).all()


def test_tree_infinite_masked_rows(pa):
    """NaN and infinities in rows that a row does not see do not reach it."""
    c = _tree_case("bf16", 128, 16, 8, 2, [100], [20], 21, kind="star")
    for t in (c["k"], c["v"]):
        t[7] = float("nan")
        t[8] = float("inf")
    out = _tree_call(pa, c).double().cpu()
    keep = [i for i in range(20) if i not in (7, 8)]
    c["k"][7:9], c["v"][7:9] = 0.0, 0.0
    want, spread = _tree_reference(c)
    off = (out - want).abs()[keep]
    assert (off <= (2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * spread)[keep]).all()


@pytest.mark.parametrize("kv,D", [("bf16", 128), ("bf16", 64), ("int8", 128), ("fp8", 128)])
def test_tree_leaves_out_bad_sequences(pa, kv, D):
    """A parent at or behind its row, one below -1, too many rows: flagged and not written; the other
    sequences are right."""
    for at, parent, flagged in ((3, 3, "parent"), (2, 9, "parent"), (4, -2, "parent"), (None, None, "query")):
        c = _tree_case(kv, D, 16, 8, 2, [40, 100, 7], [5, 8, 4], 11)
        flag = _flag()
        if at is not None:
            c["parents"][5 + at] = parent
        out = _tree_call(pa, c, flag=flag, max_q=8 if at is not None else 7)
        torch.cuda.synchronize()
        assert flag.item() == (pa.PA_FLAG_TREE_PARENT if flagged == "parent" else pa.PA_FLAG_QUERY_OUT_OF_RANGE)
        assert torch.isnan(out[5:13].float()).all()
        good = dict(c, starts=[0, 5, 13, 17])
        if at is not None:
            good["parents"] = list(c["parents"])
            good["parents"][5 + at] = 0
        want, spread, taken = _tree_taken(good, 2.0 ** -10 * (1 + 2.0 ** -11) if kv != "bf16" else 0.0)
        rows = [*range(5), *range(13, 17)]
        off = (out.double().cpu() - want).abs()[rows]
        assert (off <= (2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * spread + taken)[rows]).all()


@pytest.mark.parametrize("kv,D", [("bf16", 128), ("bf16", 64), ("int8", 128), ("fp8", 128)])
def test_tree_flags(pa, kv, D):
    """A block id outside the pool reads as zeros and is flagged; a context past max_context_len is
    clamped to it and flagged, a negative one to 0."""
    c = _tree_case(kv, D, 16, 8, 2, [90, 200], [9, 20], 13)
    for bad in (2 ** 30, -1):
        c["tables"][1, 2] = bad
        flag = _flag()
        out = _tree_call(pa, c, flag=flag)
        torch.cuda.synchronize()
        assert flag.item() == pa.PA_FLAG_BLOCK_OUT_OF_RANGE
        assert torch.isfinite(out.float()).all()
    c = _tree_case(kv, D, 16, 8, 2, [90, 200], [9, 20], 14)
    flag = _flag()
    out = _tree_call(pa, c, flag=flag, max_ctx=150)
    torch.cuda.synchronize()
    assert flag.item() == pa.PA_FLAG_CONTEXT_OUT_OF_RANGE
    _tree_check(out, dict(c, lens=[90, 150]))
    flag = _flag()
    out = _tree_call(pa, dict(c, lens=[90, -3]), flag=flag, max_ctx=200)
    torch.cuda.synchronize()
    assert flag.item() == pa.PA_FLAG_CONTEXT_OUT_OF_RANGE
    _tree_check(out, dict(c, lens=[90, 0]))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_tree_of_a_chain_is_multi_token_attention(pa, kv):
    """A chain whose rows are then appended attends what consecutive new tokens do (a bf16 cache: within
    two roundings; an fp8 one holds the new rows rounded, so only bf16 is compared)."""
    c = _tree_case("bf16", 128, 16, 16, 4, [130, 64], [6, 20], 17, kind="chain", spare=8)
    free = [b for b in range(c["cache"]["k_cache"].shape[0]) if b not in set(c["tables"][c["tables"] < 2 ** 30].tolist())]
    slots, lens = [], []
    wide = torch.full((2, 16), 2 ** 30, dtype=torch.int32, device=DEV)
    wide[:, : c["tables"].shape[1]] = c["tables"]
    for s, n in enumerate(c["lens"]):
        for t in range(n, n + c["nodes"][s]):
            if wide[s, t // 16] == 2 ** 30:
                wide[s, t // 16] = free.pop()
            slots.append(int(wide[s, t // 16]) * 16 + t % 16)
        lens.append(n + c["nodes"][s])
    a = _tree_call(pa, c)
    pa.pa_reshape_and_cache(c["k"], c["v"], c["cache"]["k_cache"], c["cache"]["v_cache"], torch.tensor(slots, device=DEV))
    b = torch.empty_like(a)
    pa.pa_multi_token_attention(b, c["q"], c["cache"]["k_cache"], c["cache"]["v_cache"], wide, _i32(lens), _i32(c["starts"]),
                                c["scale"], max(lens), 20)
    want, spread = _tree_reference(c)
    bound = 2 * (2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * spread)
    assert ((a.double() - b.double()).abs().cpu() <= bound).all()


@pytest.mark.parametrize("kv", ["int8", "fp8"])
def test_tree_of_a_chain_is_multi_token_attention_8bit(pa, kv):
    """The same on 8-bit caches whose rows lose nothing: codes times a power of two, the largest code among
    each row's, so that the chain's appended rows are the rows the tree saw.  Both results are
    then within the bounds of a bf16 cache."""
    g = _gen(57)
    top, step = (127.0, 2.0 ** -5) if kv == "int8" else (448.0, 2.0 ** -7)

    def rows(*shape):
        x = (torch.randn(shape, generator=g) * top / 3).clamp(-top, top)
        x = x.round() if kv == "int8" else x.to(torch.float8_e4m3fn).float()
        x[..., 5] = top
        return x

    c = _tree_case(kv, 128, 16, 16, 4, [130, 64], [6, 20], 58, kind="chain", spare=8)
    cache, N = c["cache"], c["cache"]["k_cache"].shape[0]
    for name in ("k", "v"):
        codes = rows(N, 4, 16, 128)
        cache[name + "_cache"].copy_(codes.to(torch.int8) if kv == "int8" else codes.to(torch.float8_e4m3fn).view(torch.uint8))
        cache[name + "_scale"].fill_(step)
        c[name] = (rows(26, 4, 128) * step).to(torch.bfloat16).to(DEV)
    a = _tree_call(pa, c)
    _tree_check(a, c)
    taken = set(c["tables"][c["tables"] < 2 ** 30].tolist())
    free = [b for b in range(N) if b not in taken]
    wide = torch.full((2, 16), 2 ** 30, dtype=torch.int32)
    wide[:, : c["tables"].shape[1]] = c["tables"].cpu()
    slots, lens = [], []
    for s, n in enumerate(c["lens"]):
        for t in range(n, n + c["nodes"][s]):
            if wide[s, t // 16] == 2 ** 30:
                wide[s, t // 16] = free.pop()
            slots.append(int(wide[s, t // 16]) * 16 + t % 16)
        lens.append(n + c["nodes"][s])
    at = torch.tensor(slots, device=DEV)
    (pa.pa_quantize_kv if kv == "int8" else pa.pa_quantize_kv_fp8)(c["k"], c["v"], *cache.values(), at)
    block, off = (at // 16).cpu().numpy(), (at % 16).cpu().numpy()
    for name in ("k", "v"):  # appended without loss
        held = _values(cache[name + "_cache"])[block, :, off] * cache[name + "_scale"].cpu().double().numpy()[block, :, off][..., None]
        assert (held == c[name].double().cpu().numpy()).all()
    b = torch.empty_like(a)
    pa.pa_multi_token_attention(b, c["q"], cache["k_cache"], cache["v_cache"], wide.to(DEV), _i32(lens), _i32(c["starts"]), c["scale"],
                                max(lens), 20, k_scale=cache["k_scale"], v_scale=cache["v_scale"])
    want, spread = _tree_reference(c)
    bound = 2 * (2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * spread)
    assert ((a.double() - b.double()).abs().cpu() <= bound).all()


@pytest.mark.parametrize("kv,D", [("bf16", 128), ("int8", 64), ("fp8", 128)])
def test_tree_graph_and_streams(pa, kv, D):
    """Captured and replayed on other inputs of the same shapes, and run on two side streams at once with a
    workspace each: the bits of an eager call."""
    c = _tree_case(kv, D, 16, 16, 4, [700, 33, 2000], [9, 30, 16], 19)
    d = _tree_case(kv, D, 16, 16, 4, [700, 33, 2000], [9, 30, 16], 20)
    eager = [_tree_call(pa, x) for x in (c, d)]
    n = pa.pa_tree_workspace_size(3, 55, 16, 4, D, 16, pa.kv_dtype_of(c["cache"]["k_cache"]), 2000, 30)
    ws = [torch.full((max(n, 1),), 0xff, dtype=torch.uint8, device=DEV) for _ in range(2)]
    out, lens, starts, parents = torch.empty_like(c["q"]), _i32(c["lens"]), _i32(c["starts"]), _i32(c["parents"])
    hold = {k: v.clone() for k, v in c["cache"].items()}
    q, k, v, tables = c["q"].clone(), c["k"].clone(), c["v"].clone(), c["tables"].clone()

    def call(o, w, stream=None):
        pa.pa_tree_attention(o, q, k, v, hold["k_cache"], hold["v_cache"], tables, lens, starts, parents, c["scale"], 2000, 30,
                             workspace=w, k_scale=hold.get("k_scale"), v_scale=hold.get("v_scale"), stream=stream)

    call(out, ws[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, ws[0])
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager[0])
    for mine, other in ((q, d["q"]), (k, d["k"]), (v, d["v"]), (tables, d["tables"]), (parents, _i32(d["parents"]))):
        mine.copy_(other)
    for name in hold:
        hold[name].copy_(d["cache"][name])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager[1])
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.empty_like(out) for _ in range(2)]
    torch.cuda.synchronize()
    for s, o, w in zip(streams, outs, ws):
        call(o, w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], eager[1]) and torch.equal(outs[1], eager[1])


def test_tree_graphs_that_share_a_workspace(pa):
    """Two captured calls of other shapes and cache types with one workspace, replayed in turn on one stream."""
    cases = [_tree_case("bf16", 128, 16, 8, 2, [700, 33], [40, 3], 43), _tree_case("fp8", 128, 32, 16, 4, [64, 0, 2100], [2, 9, 30], 44),
             _tree_case("int8", 64, 16, 8, 2, [500], [12], 45)]
    want = [_tree_call(pa, c) for c in cases]
    sizes = [pa.pa_tree_workspace_size(len(c["lens"]), len(c["parents"]), c["q"].shape[1], c["k"].shape[1], c["q"].shape[2],
                                       c["cache"]["k_cache"].shape[2], pa.kv_dtype_of(c["cache"]["k_cache"]), max(c["lens"]),
                                       max(c["nodes"])) for c in cases]
    ws = torch.full((max(sizes),), 0xff, dtype=torch.uint8, device=DEV)
    graphs, outs, held = [], [], []
    for c in cases:
        args = dict(out=torch.empty_like(c["q"]), query=c["q"], key=c["k"], value=c["v"], k_cache=c["cache"]["k_cache"],
                    v_cache=c["cache"]["v_cache"], block_tables=c["tables"], context_lens=_i32(c["lens"]), query_start=_i32(c["starts"]),
                    parents=_i32(c["parents"]), scale=c["scale"], max_context_len=max(c["lens"]), max_query_len=max(c["nodes"]),
                    workspace=ws, k_scale=c["cache"].get("k_scale"), v_scale=c["cache"].get("v_scale"))
        pa.pa_tree_attention(**args)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pa.pa_tree_attention(**args)
        graphs.append(graph)
        outs.append(args["out"])
        held.append(args)
    for out in outs:
        out.zero_()
    for i in (0, 1, 2, 1, 0, 2, 0):
        graphs[i].replay()
    torch.cuda.synchronize()
    for out, eager in zip(outs, want):
        assert torch.equal(out, eager)


@pytest.mark.parametrize("kv,D", [("bf16", 128), ("bf16", 64), ("int8", 64), ("fp8", 128)])
def test_tree_refused_then_valid_on_one_workspace(pa, kv, D):
    """A call all of whose sequences are left out (a bad parent behind a long context, no rows, too many
    rows), and at once a valid one with the same workspace: the bits that call gives alone."""
    good = _tree_case(kv, D, 16, 8, 2, [70, 700, 33], [9, 30, 16], 51)
    late = _tree_case(kv, D, 16, 8, 2, [40000], [30], 52)
    late["parents"][3] = 3
    none = _tree_case(kv, D, 16, 8, 2, [40000], [0], 53, behind=30)
    long = _tree_case(kv, D, 16, 8, 2, [40000], [31], 54)
    code = pa.kv_dtype_of(good["cache"]["k_cache"])
    n = max(pa.pa_tree_workspace_size(3, 55, 8, 2, D, 16, code, 700, 30), pa.pa_tree_workspace_size(1, 31, 8, 2, D, 16, code, 40000, 30))
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device=DEV)
    alone = _tree_call(pa, good, workspace=ws)
    _tree_check(alone, good)
    for bad, flagged in ((late, pa.PA_FLAG_TREE_PARENT), (none, 0), (long, pa.PA_FLAG_QUERY_OUT_OF_RANGE)):
        outs, held = [], torch.full_like(bad["q"], float("nan"))
        flag = _flag()
        for _ in range(20):
            _tree_call(pa, bad, out=held, max_q=30, flag=flag, workspace=ws)
            outs.append(_tree_call(pa, good, workspace=ws))
        torch.cuda.synchronize()
        assert flag.item() == flagged and torch.isnan(held.float()).all()
        assert all(torch.equal(out, alone) for out in outs)


class _Recorder:
    """The library with one call replaced: it notes its arguments and runs nothing."""

    def __init__(self, lib, name):
        self._lib, self._name, self.args = lib, name, None

    def __getattr__(self, name):
        if name != self._name:
            return getattr(self._lib, name)

        def call(*args):
            self.args = args
            return 0
        return call


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", ["pa_tree_attention", "pa_multi_token_attention", "pa_decode_shared_prefix"])
def test_default_workspace_belongs_to_the_calls_stream(pa, monkeypatch, name, handle):
    """A workspace allocated for a call on another stream than the current one is not given to the current
    stream's next allocation while that call may still run."""
    c = _tree_case("bf16", 128, 16, 8, 2, [6000, 700], [9, 30], 55)
    lib = pa.load_library()
    recorder, side, fresh = _Recorder(lib, name), torch.cuda.Stream(), torch.empty_like(c["q"])
    stream = side.cuda_stream if handle else side
    cache = (c["cache"]["k_cache"], c["cache"]["v_cache"], c["tables"], _i32(c["lens"]))
    q2 = torch.empty((2, 8, 128), dtype=torch.bfloat16, device=DEV)
    starts, parents, one, prefix = _i32(c["starts"]), _i32(c["parents"]), _i32([0, 2]), _i32([16])
    if name == "pa_tree_attention":
        n, at = pa.pa_tree_workspace_size(2, 39, 8, 2, 128, 16, 0, 6000, 30), -4
    elif name == "pa_multi_token_attention":
        n, at = pa.pa_multi_token_workspace_size(2, 39, 8, 2, 128, 16, 0, 6000, 30), -4
    else:
        n, at = pa.pa_decode_shared_prefix_workspace_size(2, 8, 2, 128, 16, 0, 6000, 2, 16), -4
    assert n > 0
    monkeypatch.setattr(pa, "_LIB", recorder)
    if name == "pa_tree_attention":
        pa.pa_tree_attention(fresh, c["q"], c["k"], c["v"], *cache, starts, parents, 0.1, 6000, 30, stream=stream)
    elif name == "pa_multi_token_attention":
        pa.pa_multi_token_attention(fresh, c["q"], *cache, starts, 0.1, 6000, 30, stream=stream)
    else:
        pa.pa_decode_shared_prefix(q2, q2, *cache, 0.1, 6000, one, prefix, 2, 16, stream=stream)
    monkeypatch.undo()
    start, size = recorder.args[at], recorder.args[at + 1]
    assert size >= n and recorder.args[-1] == side.cuda_stream
    others = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(4)]
    assert all(t.data_ptr() + n <= start or start + size <= t.data_ptr() for t in others)


def test_default_workspace_on_the_default_stream(pa, monkeypatch):
    """The default stream by its handle, 0, while another stream is current: the workspace is the default
    stream's, given back to it and to no other."""
    c = _tree_case("bf16", 128, 16, 8, 2, [6000, 700], [9, 30], 61)
    want, n = _tree_call(pa, c), pa.pa_tree_workspace_size(2, 39, 8, 2, 128, 16, 0, 6000, 30)
    torch.cuda.synchronize()
    recorder, out, side = _Recorder(pa.load_library(), "pa_tree_attention"), torch.empty_like(c["q"]), torch.cuda.Stream()
    with monkeypatch.context() as m, torch.cuda.stream(side):
        m.setattr(pa, "_LIB", recorder)
        _tree_call(pa, c, out=out, stream=0)
        start, size = recorder.args[-4], recorder.args[-3]
        others = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(4)]
        assert all(t.data_ptr() + n <= start or start + size <= t.data_ptr() for t in others)
    assert recorder.args[-1] in (0, None)
    assert torch.empty(size, dtype=torch.uint8, device=DEV).data_ptr() == start  # (the current stream is the default one again)
    assert torch.equal(_tree_call(pa, c, out=out, stream=0), want)


def test_default_workspace_on_a_side_stream(pa):
    """Calls that allocate their own workspace on a side stream, behind work there, while the main stream allocates
    and overwrites as much memory: the bits of a call on the main stream."""
    c = _tree_case("bf16", 128, 16, 8, 2, [9000, 700, 33], [9, 30, 16], 56)
    want, side = _tree_call(pa, c), torch.cuda.Stream()
    n = pa.pa_tree_workspace_size(3, 55, 8, 2, 128, 16, 0, 9000, 30)
    outs = [torch.full_like(c["q"], float("nan")) for _ in range(10)]
    lists = [_i32(c[x]) for x in ("lens", "starts", "parents")]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
    for out in outs:
        pa.pa_tree_attention(out, c["q"], c["k"], c["v"], c["cache"]["k_cache"], c["cache"]["v_cache"], c["tables"], *lists, c["scale"],
                             9000, 30, stream=side)
        for _ in range(4):
            torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0xff)
    for _ in range(200):
        torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0xff)
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for out in outs)


# ------------------------------------------------------------------------------ verify
def _verify_case(S, V, nodes, seed, kind="tree", drafter=True, probs="fp32", pad=0, sharp=2.0, near=0.7, before=0, behind=0):
    g = _gen(seed)
    T = before + sum(nodes) + behind
    starts = [before + sum(nodes[:s]) for s in range(S + 1)]
    dtype = torch.float32 if probs == "fp32" else torch.bfloat16
    x = torch.randn((T, V), generator=g) * sharp
    p = torch.softmax(x, -1).to(dtype)
    q = torch.softmax(x + torch.randn((T, V), generator=g) * near, -1).to(dtype)
    parents = [-7] * before + ref.random_parents(nodes, g, kind) + [-9] * behind
    tokens = [int(torch.multinomial(p[0].float(), 1, generator=g))] * T
    for s in range(S):
        for r in range(starts[s] + 1, starts[s + 1]):
            tokens[r] = int(torch.multinomial(q[starts[s] + max(parents[r], 0)].float(), 1, generator=g))

    def padded(t):
        wide = torch.full((T, V + pad), float("nan"), dtype=dtype, device=DEV)
        wide[:, :V] = t.to(DEV)
        return wide[:, :V]

    bs = 16
    lens = torch.randint(0, 50, (S,), generator=g).tolist()
    M = (50 + max([1, *nodes])) // bs + 1
    return dict(p=padded(p), q=padded(q) if drafter else None, tokens=tokens, parents=parents, starts=starts, nodes=nodes,
                u=torch.rand(T, generator=g), u_final=torch.rand(S, generator=g), lens=lens, bs=bs,
                tables=torch.randperm(S * M, generator=g).view(S, M).int(), S=S, V=V, W=max([1, *nodes]))


def _verify_call(pa, c, flag=None, slots=True):
    T = len(c["tokens"])
    o = dict(tokens_out=torch.full((c["S"], c["W"]), 99, dtype=torch.int32, device=DEV),
             path=torch.full((c["S"], c["W"]), 99, dtype=torch.int32, device=DEV),
             n_out=torch.full((c["S"],), 99, dtype=torch.int32, device=DEV),
             slots=torch.full((T,), 99, dtype=torch.int64, device=DEV))
    extra = dict(slot_mapping=o["slots"], block_tables=c["tables"].to(DEV), context_lens=_i32(c["lens"]), block_size=c["bs"],
                 num_blocks=c.get("N", c["tables"].numel())) if slots else {}
    pa.pa_verify_tree(o["tokens_out"], o["path"], o["n_out"], _i32(c["tokens"]), c["p"], _i32(c["starts"]), _i32(c["parents"]),
                      c["u"].to(DEV), c["u_final"].to(DEV), draft_probs=c["q"], err_flag=flag, **extra)
    torch.cuda.synchronize()
    return o


def _verify_check(o, c):
    tokens_out, path, n_out, slots = ref.verify_tree(c["tokens"], c["p"], c["q"], c["starts"], c["parents"], c["u"].tolist(),
                                                     c["u_final"].tolist(), c["W"], c["tables"].tolist(), c["lens"], c["bs"])
    assert o["n_out"].tolist() == n_out
    assert o["path"].tolist() == path
    assert o["tokens_out"].tolist() == tokens_out
    a, b = c["starts"][0], c["starts"][-1]
    assert o["slots"].tolist() == [99] * a + slots[a:b] + [99] * (len(slots) - b)
    return n_out


@pytest.mark.parametrize("probs", ["fp32", "bf16"])
@pytest.mark.parametrize("drafter", [True, False])
@pytest.mark.parametrize("V,pad", [(1, 0), (2, 0), (7, 1), (129, 0), (1000, 24), (5003, 0), (6007, 1), (32000, 0), (33333, 3)])
def test_verify_trees(pa, V, pad, drafter, probs):
    """Trees and chains of one row up, rows of no sequence, vocabularies on both sides of a vector and of
    a CTA's share, rows with padding behind the vocabulary (NaN there)."""
    kept = 0
    for seed, kind in ((1, "tree"), (2, "chain"), (3, "star")):
        c = _verify_case(5, V, [1, 6, 0, 25, 3], 100 * V + seed, kind=kind, drafter=drafter, probs=probs, pad=pad, before=2, behind=1)
        kept += sum(_verify_check(_verify_call(pa, c), c))
    # the 12 roots, and drafts (a fixed choice of little probability is rarely kept)
    assert kept > 15 or not drafter


@pytest.mark.parametrize("drafter", [True, False])
def test_verify_many_rejections(pa, drafter):
    """Flat, distant distributions and wide trees: a node rejects child after child, the same token among
    them more than once."""
    c = _verify_case(6, 40, [200, 100, 256, 2, 64, 33], 5, kind="star", drafter=drafter, sharp=1.0, near=3.0)
    c["u"] = 1 - (1 - c["u"]) * 1e-3  # hard to accept
    _verify_check(_verify_call(pa, c), c)
    c = _verify_case(3, 50001, [30, 12, 64], 6, kind="star", drafter=drafter, sharp=1.0, near=3.0)
    c["u"] = 1 - (1 - c["u"]) * 1e-3
    _verify_check(_verify_call(pa, c), c)


def test_verify_large_vocabulary(pa):
    """Vocabularies beyond what a launch keeps on chip, with and without an aligned row stride."""
    for V, pad, probs in ((300000, 0, "fp32"), (300001, 0, "fp32"), (600000, 8, "bf16"), (262144, 0, "fp32")):
        c = _verify_case(2, V, [4, 3], V, probs=probs, pad=pad, near=2.0)
        _verify_check(_verify_call(pa, c), c)


@pytest.mark.parametrize("probs", ["fp32", "bf16"])
@pytest.mark.parametrize("drafter", [True, False])
def test_verify_serving_batches_of_clusters(pa, drafter, probs):
    """More sequences than one wave of large blocks holds, each served by several blocks of threads: short and
    empty trees over vocabularies just above the smallest that is split, where one block's part of a
    sum is ready soonest; several rejections a sequence, some sequences refused."""
    for V, kind, pad in ((6001, "star", 0), (6016, "tree", 0), (9001, "chain", 7)):
        nodes = [(0, 1, 2, 4, 7, 12)[s % 6] for s in range(64)]
        c = _verify_case(64, V, nodes, V, kind=kind, drafter=drafter, probs=probs, pad=pad, near=1.5)
        c["u"][1::3] = 1 - (1 - c["u"][1::3]) * 1e-3  # hard to accept
        for _ in range(8):
            _verify_check(_verify_call(pa, c), c)
        bad = dict(c, parents=list(c["parents"]))
        refused = [s for s in range(64) if nodes[s] > 1 and s % 4 == 0]
        for s in refused:
            bad["parents"][c["starts"][s] + 1] = 1
        flag, good = _flag(), _verify_call(pa, c)
        o = _verify_call(pa, bad, flag=flag)
        assert flag.item() == pa.PA_FLAG_TREE_PARENT
        kept = [s for s in range(64) if s not in refused]
        assert (o["n_out"][refused] == 0).all() and (o["tokens_out"][refused] == -1).all()
        for name in ("tokens_out", "path", "n_out"):
            assert torch.equal(o[name][kept], good[name][kept])


def test_verify_draws_at_the_border_of_two_shares(pa):
    """Rows whose halves hold the same entries in another order, drawn at one half of their sum: the border of two
    blocks' shares exactly, so that the last bit of their sums decides.  The blocks of a sequence agree: one of
    the two neighbours is drawn, the same one every time.  (Eight blocks that each added the others' parts
    with roundings of their own left 3 of 38 such rows without a token.)"""
    g, S, half = _gen(50), 38, 4096
    for probs in (torch.float32, torch.bfloat16):
        a = torch.softmax(torch.randn((S, half), generator=g, dtype=torch.float64) * 4, -1).to(probs)
        p = torch.cat((a, torch.stack([row[torch.randperm(half, generator=g)] for row in a])), 1).to(DEV)
        assert (p > 0).all()
        said = []
        for _ in range(10):
            o = torch.full((S, 1), 99, dtype=torch.int32, device=DEV), torch.full((S, 1), 99, dtype=torch.int32, device=DEV)
            n = torch.empty(S, dtype=torch.int32, device=DEV)
            pa.pa_verify_tree(o[0], o[1], n, _i32([0] * S), p, _i32(range(S + 1)), _i32([-1] * S), torch.zeros(S, device=DEV),
                              torch.full((S,), 0.5, device=DEV))
            said.append(o[0][:, 0].tolist())
        assert all(x in (half - 1, half) for x in said[0]), said[0]
        assert all(x == said[0] for x in said)


def test_verify_one_hot_targets(pa):
    """Greedy targets: a draft is kept exactly where it is the target's token."""
    c = _verify_case(4, 300, [9, 9, 9, 9], 8, kind="chain", drafter=False)
    best = c["p"].argmax(-1)
    c["p"] = torch.nn.functional.one_hot(best, 300).float()
    for r in range(len(c["tokens"])):
        if r % 9 and r % 5:
            c["tokens"][r] = int(best[r - 1])
    n = _verify_check(_verify_call(pa, c), c)
    assert max(n) > 1


def test_verify_edges(pa):
    """u = 0, u just below 1, equal distributions (always kept), zero draft probability of a drafted token,
    tokens outside the vocabulary, a final number just below 1."""
    c = _verify_case(5, 100, [5] * 5, 9, kind="chain")
    below = float(np.nextafter(np.float32(1), np.float32(0)))
    c["u"][:10], c["u"][10:15] = 0.0, below
    c["u_final"][:] = torch.tensor([0.0, below, below, 0.5, 0.0])
    c["q"][10:15] = c["p"][10:15]
    c["q"][15, c["tokens"][16]] = 0.0
    n = _verify_check(_verify_call(pa, c), c)
    assert n[2] == 5
    for bad in (-1, 100, 2 ** 31 - 1):
        c["tokens"][6] = bad
        flag = _flag()
        o = _verify_call(pa, c, flag=flag)
        assert flag.item() == pa.PA_FLAG_TOKEN_OUT_OF_RANGE
        _verify_check(o, c)


def test_verify_draws_only_tokens_with_weight(pa):
    """Numbers at the ends of the range and rows that are zero nearly everywhere: never a token without weight."""
    S, V = 64, 3001
    c = _verify_case(S, V, [1] * S, 10)
    c["p"].zero_()
    g = _gen(11)
    for s in range(S):
        at = torch.randint(0, V, (1 + s % 3,), generator=g)
        c["p"][s, at.to(DEV)] = 0.3
    c["u_final"] = torch.tensor([[0.0, float(np.nextafter(np.float32(1), np.float32(0)))][s % 2] for s in range(S)])
    o = _verify_call(pa, c)
    _verify_check(o, c)


def test_verify_bad_probabilities(pa):
    """NaN and negative entries count as zero; a row without mass, or with an infinite one, gives -1 and the flag."""
    c = _verify_case(4, 200, [3] * 4, 12, kind="chain")
    c["p"][0, ::3], c["p"][4, ::5] = float("nan"), -1.0
    flag = _flag()
    o = _verify_call(pa, c, flag=flag)
    assert flag.item() == 0
    _verify_check(o, c)
    c["p"][6:9] = 0.0
    flag = _flag()
    o = _verify_call(pa, c, flag=flag)
    assert flag.item() == pa.PA_FLAG_PROBABILITY and o["tokens_out"][2].tolist() == [-1, -1, -1] and o["n_out"][2].item() == 1
    _verify_check(o, c)
    c["p"][6:9] = float("inf")
    c["u"][7] = 2.0
    flag = _flag()
    o = _verify_call(pa, dict(c, q=None), flag=flag)
    assert flag.item() & pa.PA_FLAG_PROBABILITY and (o["tokens_out"][2] == -1).any()


def test_verify_bad_trees_and_tables(pa):
    """Bad parents or too many rows leave a sequence out (n_out 0, slots -1); a missing table entry gives slot -1
    and the flag; without slot_mapping nothing of it is read."""
    for at, parent in ((7, 4), (8, -3), (6, 1)):
        c = _verify_case(3, 50, [4, 6, 5], 13)
        c["parents"][at] = parent
        flag = _flag()
        o = _verify_call(pa, c, flag=flag)
        ok = -1 <= parent < at - 4
        assert flag.item() == (0 if ok else pa.PA_FLAG_TREE_PARENT)
        if ok:
            _verify_check(o, c)
            continue
        assert o["n_out"][1].item() == 0 and (o["path"][1] == -1).all() and (o["slots"][4:10] == -1).all()
        solo = dict(c, parents=c["parents"][:4] + [-1] * 6 + c["parents"][10:])
        tokens_out, path, n_out, slots = ref.verify_tree(solo["tokens"], c["p"], c["q"], c["starts"], solo["parents"], c["u"].tolist(),
                                                         c["u_final"].tolist(), c["W"], c["tables"].tolist(), c["lens"], 16)
        for s in (0, 2):
            assert o["tokens_out"][s].tolist() == tokens_out[s] and o["path"][s].tolist() == path[s]
    c = _verify_case(3, 50, [4, 6, 5], 14)
    flag = _flag()
    o = _verify_call(pa, dict(c, W=5), flag=flag)
    assert flag.item() == pa.PA_FLAG_QUERY_OUT_OF_RANGE and o["n_out"][1].item() == 0
    flag = _flag()
    o = _verify_call(pa, dict(c, N=0x7fffffff, lens=[0, 10 ** 6, 3]), flag=flag)
    assert flag.item() == pa.PA_FLAG_BLOCK_OUT_OF_RANGE and (o["slots"][4:10] == -1).all() and (o["slots"][:4] >= 0).any()
    o = _verify_call(pa, c, slots=False)
    assert (o["slots"] == 99).all()
    _verify_check(dict(o, slots=_verify_call(pa, c)["slots"]), c)


@pytest.mark.parametrize("drafter", [True, False])
def test_verify_keeps_the_targets_law(pa, drafter):
    """The first token out follows the target's distribution whatever the drafter's: the frequencies over a
    grid of numbers and independent drafts.  S = 40000 draws: a frequency is off by sqrt(p (1 - p) / S) <= 0.0025
    at one standard deviation; six of them, 0.015, are asked for."""
    S, V, g = 40000, 6, _gen(15)
    p = torch.tensor([0.05, 0.4, 0.1, 0.25, 0.15, 0.05])
    q = torch.tensor([0.3, 0.1, 0.2, 0.2, 0.1, 0.1])
    nodes = 4  # a root and three children
    T = S * nodes
    tokens = torch.multinomial(q, T, replacement=True, generator=g) if drafter else torch.tensor([0, 1, 3, 4]).repeat(S)
    o = [torch.empty((S, nodes), dtype=torch.int32, device=DEV) for _ in range(2)]
    n = torch.empty(S, dtype=torch.int32, device=DEV)
    pa.pa_verify_tree(o[0], o[1], n, tokens.int().to(DEV), p.expand(T, V).contiguous().to(DEV),
                      torch.arange(0, T + 1, nodes, dtype=torch.int32, device=DEV), _i32([-1, 0, 0, 0]).repeat(S),
                      torch.rand(T, generator=g).to(DEV), torch.rand(S, generator=g).to(DEV),
                      draft_probs=q.expand(T, V).contiguous().to(DEV) if drafter else None)
    freq = torch.bincount(o[0][:, 0].long().cpu(), minlength=V) / S
    assert (freq - p).abs().max() < 0.015, freq


def test_verify_graph(pa):
    """Captured and replayed with other numbers."""
    c, d = (_verify_case(6, 9000, [7] * 6, s, near=2.0) for s in (21, 22))
    T = 42
    hold = [_i32(c["tokens"]), c["p"].clone(), c["q"].clone(), _i32(c["parents"]), c["u"].to(DEV), c["u_final"].to(DEV)]
    starts, o = _i32(c["starts"]), [torch.empty((6, 7), dtype=torch.int32, device=DEV) for _ in range(2)]
    n = torch.empty(6, dtype=torch.int32, device=DEV)

    def call():
        pa.pa_verify_tree(o[0], o[1], n, hold[0], hold[1], starts, hold[3], hold[4], hold[5], draft_probs=hold[2])

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for x, new in zip(hold, [_i32(d["tokens"]), d["p"], d["q"], _i32(d["parents"]), d["u"].to(DEV), d["u_final"].to(DEV)]):
        x.copy_(new)
    graph.replay()
    torch.cuda.synchronize()
    e = _verify_call(pa, d)
    assert torch.equal(o[0], e["tokens_out"]) and torch.equal(o[1], e["path"]) and torch.equal(n, e["n_out"])
    assert T == len(d["tokens"])


# -------------------------------------------------------------------------- the whole step
@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
def test_speculative_step(pa, kv):
    """Rotate and append a prompt, then two steps of: rotate a tree's rows, attend, verify, append the branch that
    was kept.  The cache then holds what appending the kept tokens one by one would have put there, and the kept
    rows' attention is what decoding them over that cache gives."""
    g, Hq, Hkv, D, bs, V = _gen(31), 8, 2, 128, 16, 500
    S, prompt = 3, [37, 5, 64]
    table = pa.pa_rotary_table(pa.pa_rotary_frequencies(D, 500000.0)[0], DEV)
    M, N = 8, 40
    tables = torch.randperm(N, generator=g)[: S * M].view(S, M).int().to(DEV)
    cache = _empty_cache(kv, N, Hkv, bs, D)
    lens = list(prompt)
    slot = lambda s, t: int(tables[s, t // bs]) * bs + t % bs  # noqa: E731
    T = sum(prompt)
    q, k, v = _randn(g, T, Hq, D), _randn(g, T, Hkv, D), _randn(g, T, Hkv, D)
    pos = torch.tensor([t for n in prompt for t in range(n)], device=DEV)
    slots = torch.tensor([slot(s, t) for s, n in enumerate(prompt) for t in range(n)], device=DEV)
    flag = _flag()
    pa.pa_rotary_and_cache(torch.empty_like(q), q, k, pos, table, value=v, slot_mapping=slots, err_flag=flag, **cache)
    other = {n: c.clone() for n, c in cache.items()}
    for step in range(2):
        nodes = [6, 9, 4]
        starts = [sum(nodes[:s]) for s in range(S + 1)]
        T, parents = sum(nodes), ref.random_parents(nodes, g)
        depth = [0] * T
        for s in range(S):
            for i in range(1, nodes[s]):
                depth[starts[s] + i] = depth[starts[s] + parents[starts[s] + i]] + 1
        q, k, v = _randn(g, T, Hq, D), _randn(g, T, Hkv, D), _randn(g, T, Hkv, D)
        row_seq = [s for s in range(S) for _ in range(nodes[s])]
        pos = torch.tensor([lens[row_seq[r]] + depth[r] for r in range(T)], device=DEV)
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        pa.pa_rotary_and_cache(qo, q, k, pos, table, key_out=ko)
        out = torch.empty_like(q)
        pa.pa_tree_attention(out, qo, ko, v, cache["k_cache"], cache["v_cache"], tables, _i32(lens), _i32(starts), _i32(parents),
                             D ** -0.5, M * bs, max(nodes), k_scale=cache.get("k_scale"), v_scale=cache.get("v_scale"), err_flag=flag)
        p = torch.softmax(torch.randn((T, V), generator=g) * 2, -1).to(DEV)
        tokens = torch.tensor([int(p[starts[row_seq[r]] + max(parents[r], 0)].argmax()) for r in range(T)])
        o = [torch.empty((S, max(nodes)), dtype=torch.int32, device=DEV) for _ in range(2)]
        n, rows_slots = torch.empty(S, dtype=torch.int32, device=DEV), torch.empty(T, dtype=torch.int64, device=DEV)
        pa.pa_verify_tree(o[0], o[1], n, _i32(tokens), p, _i32(starts), _i32(parents), torch.rand(T, generator=g).to(DEV) * 0.2,
                          torch.rand(S, generator=g).to(DEV), slot_mapping=rows_slots, block_tables=tables, context_lens=_i32(lens),
                          block_size=bs, num_blocks=N, err_flag=flag)
        append = {"bf16": pa.pa_reshape_and_cache, "int8": pa.pa_quantize_kv, "fp8": pa.pa_quantize_kv_fp8}[kv]
        append(ko, v, *cache.values(), rows_slots)
        torch.cuda.synchronize()
        assert flag.item() == 0
        assert max(n.tolist()) > 1
        for s in range(S):
            way = o[1][s, : n[s]].long()
            at = torch.tensor([slot(s, lens[s] + j) for j in range(len(way))], device=DEV)
            append(ko[way].contiguous(), v[way].contiguous(), *other.values(), at)
            if kv == "bf16":  # 8-bit caches hold the ancestors rounded; the tree saw them exact
                dec, m = torch.empty_like(qo[way]), len(way)
                ws = pa.pa_multi_token_workspace_size(1, m, Hq, Hkv, D, bs, 0, M * bs, m)
                pa.pa_multi_token_attention(dec, qo[way].contiguous(), other["k_cache"], other["v_cache"], tables[s:s + 1],
                                            _i32([lens[s] + m]), _i32([0, m]), D ** -0.5, M * bs, m,
                                            workspace=torch.empty(max(ws, 1), dtype=torch.uint8, device=DEV))
                # two results within 2^-8 of their size and of sum w |v| (at most max |v| < 5.5) each
                far = (dec.double() - out[way].double()).abs()
                assert (far <= 2 * (2.0 ** -8 * out[way].double().abs() + (2.0 ** -8 + 2.0 ** -12) * 5.5)).all()
            lens[s] += len(way)
        for name in cache:
            bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[cache[name].element_size()]
            assert torch.equal(cache[name].view(bits), other[name].view(bits)), name


def test_other_streams_and_devices(pa):
    """Calls on a side stream run there; tensors of another device than the first are refused."""
    c = _verify_case(2, 64, [3, 3], 40)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o = _verify_call(pa, c)
    _verify_check(o, c)
    q = _randn(_gen(1), 2, 2, 64)
    with pytest.raises(ValueError):
        pa.pa_rotary_and_cache(torch.empty_like(q), q, q.cpu(), torch.arange(2, device=DEV), pa.pa_rotary_table([1.0], DEV), key_out=q)
    assert math.isfinite(float(q.float().sum()))
