"""Host-side checks of the operators at a step's two ends: they answer without touching a GPU."""
import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_197_gb300 import _build

    _build.build()
    import paged_kv_cache_197_gb300 as pa

    return pa.load_library()


FAKE = 1 << 20  # never dereferenced: every call below fails its host checks
BIG = 1 << 40


def test_norm_rotary_host_checks(lib):
    import paged_kv_cache_197_gb300 as pa

    def call(D=128, rot=128, eps=1e-6, T=2, Hq=8, Hkv=2, qw=FAKE, kw=FAKE, kv=0, q_stride=1024, k_stride=256, v_stride=256, bs=16, N=4,
             q=FAKE, q_out=BIG, k_cache=None, factor=1.0):
        return lib.pa_norm_rotary_and_cache(q_out, 2 * BIG, q, q_stride, 3 * BIG, k_stride, 4 * BIG, v_stride, k_cache, k_cache,
                                            None, None, kv, 5 * BIG if k_cache else None, 6 * BIG, 7 * BIG, rot, 0, factor, qw, kw,
                                            eps, T, Hq, Hkv, D, bs, N, None, None)

    assert call(eps=0.0) == pa.PA_ERR_INVALID_ARG and b"eps" in lib.pa_last_error_string()
    assert b"pa_norm_rotary_and_cache" in lib.pa_last_error_string()
    for eps in (-1e-6, float("nan"), float("inf")):
        assert call(eps=eps) == pa.PA_ERR_INVALID_ARG
    assert call(qw=FAKE + 4) == pa.PA_ERR_INVALID_ARG and b"aligned" in lib.pa_last_error_string()
    assert call(kw=FAKE + 8) == pa.PA_ERR_INVALID_ARG
    assert call(D=96) == pa.PA_ERR_UNSUPPORTED
    assert call(rot=130) == pa.PA_ERR_INVALID_ARG
    assert call(q_stride=1020) == pa.PA_ERR_INVALID_ARG
    assert call(factor=float("inf")) == pa.PA_ERR_INVALID_ARG
    assert call(q_out=FAKE + 1024) == pa.PA_ERR_INVALID_ARG and b"overlaps" in lib.pa_last_error_string()
    assert call(k_cache=8 * BIG, kv=1) == pa.PA_ERR_INVALID_ARG  # scales missing
    assert call(k_cache=8 * BIG, bs=8) == pa.PA_ERR_UNSUPPORTED
    assert call(T=0) == pa.PA_OK and call(T=-1) == pa.PA_ERR_INVALID_ARG


def test_gather_host_checks(lib):
    import paged_kv_cache_197_gb300 as pa

    def call(k=FAKE, v=BIG, k_stride=256, v_stride=256, kc=2 * BIG, ks=None, kv=0, slots=3 * BIG, T=2, Hkv=2, D=128, bs=16, N=4):
        return lib.pa_gather_cache(k, k_stride, v, v_stride, kc, kc + (1 << 30) if kc else None, ks, ks, kv, slots, T, Hkv, D, bs, N, None,
                                   None)

    assert call(T=-1) == pa.PA_ERR_INVALID_ARG and b"pa_gather_cache" in lib.pa_last_error_string()
    assert call(D=96) == pa.PA_ERR_UNSUPPORTED and call(bs=8) == pa.PA_ERR_UNSUPPORTED and call(kv=3) == pa.PA_ERR_UNSUPPORTED
    assert call(N=0) == pa.PA_ERR_INVALID_ARG and call(Hkv=0) == pa.PA_ERR_INVALID_ARG
    assert call(k_stride=255) == pa.PA_ERR_INVALID_ARG and call(v_stride=260) == pa.PA_ERR_INVALID_ARG
    for name in ("k", "v", "kc", "slots"):
        assert call(**{name: None}) == pa.PA_ERR_INVALID_ARG, name
    assert call(kv=1) == pa.PA_ERR_INVALID_ARG and call(kv=2, ks=FAKE + 4) == pa.PA_ERR_INVALID_ARG
    assert call(k=FAKE + 8) == pa.PA_ERR_INVALID_ARG
    assert call(k=2 * BIG + 4096) == pa.PA_ERR_INVALID_ARG and b"overlaps" in lib.pa_last_error_string()
    assert call(v=2 * BIG - 512) == pa.PA_ERR_INVALID_ARG
    assert call(T=0) == pa.PA_OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that nothing lies at: only where nothing can be launched")
def test_gather_outputs_on_one_another(lib):
    """Rows of keys and values on one another are refused, at any distance and with strides that differ; rows in turn, slices of one
    tensor, are not."""
    import paged_kv_cache_197_gb300 as pa

    def refused(apart, k_stride=1024, v_stride=1024, T=3, row=256):
        """Values `apart` entries behind the keys."""
        status = lib.pa_gather_cache(BIG, k_stride, BIG + 2 * apart, v_stride, 4 * BIG, 4 * BIG + (1 << 30), None, None, 0, 5 * BIG, T,
                                     row // 128, 128, 16, 4, None, None)
        assert status != pa.PA_OK
        return status == pa.PA_ERR_INVALID_ARG and b"key_out overlaps value_out" in lib.pa_last_error_string()

    for apart in (0, 8, 248, 1024, 2048, -1024, -8, -248, 1024 - 248, 2048 - 8, -1024 + 8):
        assert refused(apart), apart
    assert refused(512, v_stride=512) and refused(0, T=1) and refused(-16, T=1)
    for apart in (256, 768, -256, 1024 + 256, 4096, -4096, 8192):
        assert not refused(apart), apart
    assert not refused(256, T=1) and not refused(8192, v_stride=512)


def test_sampling_host_checks(lib):
    import paged_kv_cache_197_gb300 as pa

    def draw(tokens=FAKE, x=BIG, stride=100, dtype=0, u=2 * BIG, R=2, V=100):
        return lib.pa_sample_tokens(tokens, None, x, stride, dtype, None, None, None, None, u, R, V, None, None)

    def rows(out=FAKE, out_stride=100, out_dtype=0, x=BIG, stride=100, dtype=0, R=2, V=100):
        return lib.pa_sampling_probs(out, out_stride, out_dtype, x, stride, dtype, None, None, None, None, R, V, None, None)

    for call, fn in ((draw, b"pa_sample_tokens"), (rows, b"pa_sampling_probs")):
        assert call(V=0) == pa.PA_ERR_INVALID_ARG and fn in lib.pa_last_error_string()
        big = pa.PA_SAMPLE_MAX_VOCABULARY + 1
        assert call(V=big, stride=big) == pa.PA_ERR_UNSUPPORTED
        assert call(R=-1) == pa.PA_ERR_INVALID_ARG and call(R=(1 << 20) + 1) == pa.PA_ERR_UNSUPPORTED
        assert call(dtype=2) == pa.PA_ERR_UNSUPPORTED
        assert call(stride=99) == pa.PA_ERR_INVALID_ARG and call(x=None) == pa.PA_ERR_INVALID_ARG
        assert call(x=BIG + 2) == pa.PA_ERR_INVALID_ARG and call(x=BIG + 1, dtype=1) == pa.PA_ERR_INVALID_ARG
        assert call(R=0, x=None) == pa.PA_OK
    assert draw(tokens=None) == pa.PA_ERR_INVALID_ARG and draw(u=None) == pa.PA_ERR_INVALID_ARG
    assert rows(out=None) == pa.PA_ERR_INVALID_ARG and rows(out_stride=99) == pa.PA_ERR_INVALID_ARG
    assert rows(out_dtype=7) == pa.PA_ERR_UNSUPPORTED and rows(out=FAKE + 2) == pa.PA_ERR_INVALID_ARG
    assert rows(out=BIG) == pa.PA_ERR_INVALID_ARG and b"overlaps" in lib.pa_last_error_string()
    assert rows(out=BIG + 4 * 199) == pa.PA_ERR_INVALID_ARG  # the last entry


def test_bindings_refuse_host_tensors(lib):
    import paged_kv_cache_197_gb300 as pa

    x, i = torch.zeros((2, 8)), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_sample_tokens(i, x, torch.zeros(2))
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_sampling_probs(x, x)
    heads = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_norm_rotary_and_cache(heads, heads, heads, torch.zeros(2, dtype=torch.int64), torch.zeros(32, dtype=torch.int64), 1e-6)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_gather_cache(heads, heads, torch.zeros((1, 2, 16, 64), dtype=torch.bfloat16), torch.zeros((1, 2, 16, 64), dtype=torch.bfloat16),
                           torch.zeros(2, dtype=torch.int64))
