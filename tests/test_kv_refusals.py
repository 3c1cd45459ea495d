"""What the cache calls refuse beyond the ends of single fields, on the CPU:
every argument is checked before any GPU call, and none is made here."""
import ctypes

import pytest

import verify_nvfp4_w4a16_amd as nv

torch = pytest.importorskip("torch")
from tests.test_kv_capi_cpu import A, _cache, _queries, _seqs  # noqa: E402
from verify_nvfp4_w4a16_amd import serving  # noqa: E402


@pytest.mark.parametrize("scale,k_scale,ok", [(1e30, 1e30, False), (-3e38, 2.0, False), (3e38, 1.0, True), (1e30, 1e-30, True),
                                              (1e-30, 1e-30, True), (0.0, 3e38, True)])
def test_refusal_of_scales_whose_product_is_infinite(scale, k_scale, ok):
    lib = serving._kv()
    c, s, q = _cache(k_scale=k_scale), _seqs(), _queries(scale=scale)
    assert (lib.nvfp4_kv_attention_workspace(c, s, q, ctypes.c_int64()) == nv.OK) == ok
    if not ok:
        assert lib.nvfp4_kv_attention(c, s, q, A, A, A, 1 << 40, None) == nv.ERR_SHAPE
        assert lib.nvfp4_kv_weights(c, s, q, A, A, A, None) == nv.ERR_SHAPE


@pytest.mark.parametrize("scales", [dict(k_scale=0.5), dict(v_scale=2.0), dict(k_scale=3.0, v_scale=0.25)])
def test_refusal_of_eviction_into_a_cache_of_other_scales(scales):
    # codes are copied as they are: read at another scale they would stand for other values
    lib = serving._kv()
    for c, dst in ((_cache(), _cache(**scales)), (_cache(**scales), _cache())):
        assert lib.nvfp4_kv_evict(c, _seqs(), A, 100, 64, 1, 2, dst, A, 1, A, A, A, None) == nv.ERR_SHAPE
    # equal ones pass on to the checks that follow
    assert lib.nvfp4_kv_evict(_cache(**scales), _seqs(), A, 100, 64, 1, 2, _cache(**scales), A, 1, A, A, None, None) == nv.ERR_NULL
