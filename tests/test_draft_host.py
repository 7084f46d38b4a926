"""Speculative-decoding calls without a GPU: the frequency rules and the 64-bit table against their
formulas, and every refusal that the host can give (nothing is queued, nothing dereferenced)."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

FAKE = 1 << 20  # never dereferenced: every refused call fails its host checks


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_197_gb300 import _build

    _build.build()
    import paged_kv_cache_197_gb300 as pa

    pa.load_library()
    return pa


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (20, 10000.0), (64, 500000.0), (128, 10000.0)])
def test_frequency_rules(pa, rot, base):
    """Each rule against its formula, to 1e-12 relative (pow and log are good to an ulp or two,
    2^-52, and a handful of products follow)."""
    n = rot // 2
    plain = [base ** (-2 * j / rot) for j in range(n)]

    def close(got, want):
        assert len(got) == len(want)
        assert all(abs(g - w) <= 1e-12 * abs(w) for g, w in zip(got.tolist(), want))

    inv, factor = pa.pa_rotary_frequencies(rot, base)
    close(inv, plain)
    assert factor == 1.0
    inv, factor = pa.pa_rotary_frequencies(rot, base, pa.PA_ROTARY_LINEAR, 4.0)
    close(inv, [f / 4 for f in plain])
    assert factor == 1.0
    if rot > 2:
        inv, _ = pa.pa_rotary_frequencies(rot, base, pa.PA_ROTARY_BASE, 8.0)
        close(inv, [(base * 8.0 ** (rot / (rot - 2))) ** (-2 * j / rot) for j in range(n)])
    # by parts: pairs above 32 turns in 4096 positions kept, below one turn stretched 16-fold
    inv, factor = pa.pa_rotary_frequencies(rot, base, pa.PA_ROTARY_RAMP, 16.0, 4096, 32, 1)
    assert abs(factor - (0.1 * math.log(16.0) + 1)) < 1e-12
    low = max(math.floor(rot * math.log(4096 / (32 * 2 * math.pi)) / (2 * math.log(base))), 0)
    high = min(math.ceil(rot * math.log(4096 / (2 * math.pi)) / (2 * math.log(base))), rot - 1)
    ramp = [min(max((j - low) / (high - low), 0), 1) for j in range(n)]
    close(inv, [f / 16 * r + f * (1 - r) for f, r in zip(plain, ramp)])
    # by wavelength
    inv, _ = pa.pa_rotary_frequencies(rot, base, pa.PA_ROTARY_WAVELENGTH, 8.0, 8192, 1, 4)
    want = []
    for f in plain:
        wave = 2 * math.pi / f
        if wave < 8192 / 4:
            want.append(f)
        elif wave > 8192:
            want.append(f / 8)
        else:
            r = (8192 / wave - 1) / 3
            want.append((1 - r) * f / 8 + r * f)
    close(inv, want)


def test_table_holds_turns(pa):
    """Entries are turns per position in units of 2^-64: off by the half unit of the rounding and
    the two roundings of the double quotient and its constant (3 * 2^-53 relative)."""
    inv = [1.0, 0.1234567, 1e-9, 6.5, -0.25, 0.0]
    two_pi = Fraction(6283185307179586476925286766559, 10 ** 30)
    table = pa.pa_rotary_table(inv)
    for f, t in zip(inv, table.tolist()):
        exact = Fraction(f) / two_pi % 1 * 2 ** 64
        off = (Fraction(t % 2 ** 64) - exact) % 2 ** 64
        off = min(off, 2 ** 64 - off)
        assert off <= Fraction(1, 2) + abs(Fraction(f)) / two_pi * 2 ** 64 * Fraction(3, 2 ** 53), (f, float(off))
    assert pa.pa_rotary_table([]).numel() == 0


def test_frequency_refusals(pa):
    def refused(*a, status=pa.PA_ERR_INVALID_ARG):
        with pytest.raises(pa.PagedAttentionError) as e:
            pa.pa_rotary_frequencies(*a)
        assert e.value.status == status

    refused(7)
    refused(0)
    refused(64, 1.0)
    refused(64, float("nan"))
    refused(64, 1e4, 9, status=pa.PA_ERR_UNSUPPORTED)
    refused(64, 1e4, pa.PA_ROTARY_LINEAR, 0.5)
    refused(2, 1e4, pa.PA_ROTARY_BASE, 2.0)
    refused(64, 1e4, pa.PA_ROTARY_RAMP, 2.0, 4096, 1, 32)
    refused(64, 1e4, pa.PA_ROTARY_WAVELENGTH, 2.0, 0, 1, 4)
    lib = pa.load_library()
    assert lib.pa_rotary_frequencies(64, 1e4, 0, 1, 0, 0, 0, None, None) == pa.PA_ERR_INVALID_ARG
    assert lib.pa_rotary_table(None, 3, None) == pa.PA_ERR_INVALID_ARG
    assert lib.pa_rotary_table(None, -1, None) == pa.PA_ERR_INVALID_ARG
    with pytest.raises(pa.PagedAttentionError):
        pa.pa_rotary_table([1.0, float("inf")])


def test_rotary_refusals(pa):
    lib = pa.load_library()

    def call(qo=FAKE, ko=None, q=2 * FAKE, qs=4 * 128, k=3 * FAKE, ks=2 * 128, v=4 * FAKE, vs=2 * 128, kc=5 * FAKE,
             vc=6 * FAKE, sc=None, kv=0, slots=FAKE, pos=FAKE, tab=FAKE, rot=128, f=1.0, T=3, Hq=4, Hkv=2, D=128,
             bs=16, N=4):
        return lib.pa_rotary_and_cache(qo, ko, q, qs, k, ks, v, vs, kc, vc, sc, sc, kv, slots, pos, tab, rot, 0, f,
                                       T, Hq, Hkv, D, bs, N, None, None)

    bad = pa.PA_ERR_INVALID_ARG
    assert call(T=0) == pa.PA_OK
    assert call(T=-1) == bad
    assert call(D=96) == pa.PA_ERR_UNSUPPORTED
    assert call(bs=8) == pa.PA_ERR_UNSUPPORTED
    assert call(kv=5) == pa.PA_ERR_UNSUPPORTED
    assert call(kv=pa.PA_KV_FP8) == bad            # scales missing
    assert call(rot=0) == bad and call(rot=130) == bad and call(rot=33) == bad
    assert call(f=float("inf")) == bad
    assert call(qs=4 * 128 - 8) == bad and call(qs=4 * 128 + 4) == bad and call(ks=0) == bad and call(vs=8) == bad
    assert call(qo=None) == bad and call(pos=None) == bad and call(tab=None) == bad and call(slots=None) == bad
    assert call(v=None) == bad and call(vc=None) == bad and call(kc=None) == bad
    assert call(kc=None, vc=None) == bad           # neither a cache nor key_out
    assert call(q=2 * FAKE + 2) == bad and call(kc=5 * FAKE + 8) == bad
    # overlaps that are not a whole dense tensor rotated in place
    assert call(qo=2 * FAKE, qs=5 * 128) == bad
    assert call(qo=2 * FAKE + 1024) == bad
    assert call(qo=3 * FAKE) == bad and call(qo=4 * FAKE) == bad
    assert call(ko=FAKE) == bad and call(ko=2 * FAKE) == bad and call(ko=4 * FAKE) == bad
    assert call(Hq=0) == bad and call(Hkv=0) == bad


def test_tree_refusals(pa):
    lib = pa.load_library()

    def call(out=FAKE, ks=2 * 128, vs=2 * 128, k=FAKE, par=FAKE, qs=FAKE, kv=0, M=4, S=2, T=8, Hq=8, Hkv=2, D=128, bs=16,
             N=4, scale=0.1, max_ctx=64, max_q=4, ws=FAKE, ws_bytes=1 << 40):
        return lib.pa_tree_attention(out, FAKE, k, ks, FAKE, vs, FAKE, FAKE, None, None, kv, FAKE, M, FAKE, qs, par, S,
                                     T, Hq, Hkv, D, bs, N, scale, max_ctx, max_q, ws, ws_bytes, None, None)

    bad = pa.PA_ERR_INVALID_ARG
    assert call(S=0) == pa.PA_OK and call(T=0) == pa.PA_OK
    assert call(D=80) == pa.PA_ERR_UNSUPPORTED and call(bs=64) == pa.PA_ERR_UNSUPPORTED and call(kv=4) == pa.PA_ERR_UNSUPPORTED
    assert call(Hq=7) == bad and call(max_q=0) == bad and call(max_q=9) == bad
    assert call(T=600, max_q=257) == bad            # more rows than a tree may have
    assert call(max_ctx=65) == pa.PA_ERR_OUT_OF_RANGE and call(max_ctx=-1) == bad
    assert call(par=None) == bad and call(qs=None) == bad and call(k=None) == bad
    assert call(kv=pa.PA_KV_INT8) == bad
    assert call(out=FAKE + 8) == bad and call(k=FAKE + 4) == bad
    assert call(ks=2 * 128 - 8) == bad and call(vs=2 * 128 + 4) == bad
    assert call(scale=float("nan")) == bad
    assert call(ws=None) == bad and call(ws_bytes=64) == bad and call(ws=FAKE + 16) == bad
    size = lambda **k: pa.pa_tree_workspace_size(**{**dict(  # noqa: E731
        S=2, T=8, Hq=8, Hkv=2, D=128, bs=16, kv_dtype=0, max_context_len=64, max_query_len=4), **k})
    assert size(D=80) == 0 and size(max_query_len=9) == 0 and size(kv_dtype=3) == 0
    assert size(max_context_len=0) > 0
    # more groups of four query heads than a grid has rows
    assert size(Hq=5 * 40000, Hkv=40000, max_query_len=1) == 0 and size(Hq=4 * 40000, Hkv=40000, max_query_len=1) > 0


def test_verify_refusals(pa):
    lib = pa.load_library()

    def call(out=FAKE, slots=FAKE, p=FAKE, ps=100, q=FAKE, qs=100, kind=0, par=FAKE, S=2, T=8, V=100, W=4, tab=FAKE, M=4,
             lens=FAKE, bs=16, N=4, u=FAKE):
        return lib.pa_verify_tree(out, FAKE, FAKE, slots, FAKE, p, ps, q, qs, kind, FAKE, par, u, FAKE, S, T, V, W, tab,
                                  M, lens, bs, N, None, None)

    bad = pa.PA_ERR_INVALID_ARG
    assert call(S=0) == pa.PA_OK
    assert call(S=-1) == bad and call(T=-1) == bad and call(T=0) == bad
    assert call(kind=2) == pa.PA_ERR_UNSUPPORTED
    assert call(V=0) == bad and call(V=(1 << 30) + 1, ps=1 << 31, qs=1 << 31) == bad
    assert call(W=0) == bad and call(W=9) == bad and call(T=600, W=257) == bad
    assert call(ps=99) == bad and call(qs=99) == bad
    assert call(out=None) == bad and call(p=None) == bad and call(par=None) == bad and call(u=None) == bad
    assert call(p=FAKE + 2) == bad and call(q=FAKE + 1, kind=1) == bad
    assert call(tab=None) == bad and call(lens=None) == bad and call(M=0) == bad and call(bs=8) == pa.PA_ERR_UNSUPPORTED
    assert call(S=70000, T=70000, W=1) == pa.PA_ERR_UNSUPPORTED


def test_bindings_refuse_host_tensors(pa):
    x = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.pa_rotary_and_cache(x, x, x, i.long(), i.long())
    with pytest.raises(ValueError):
        pa.pa_tree_attention(x, x, x, x, x[None], x[None], i[None], i, i, i, 0.1, 16, 1)
    with pytest.raises(ValueError):
        pa.pa_verify_tree(i[None], i[None], i, i, x[0].float(), i, i, i.float(), i.float())
    assert ctypes.sizeof(ctypes.c_uint64) == 8
