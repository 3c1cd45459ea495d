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


def _host_cache(device="cpu"):
    """A cache object over host memory, for checks that come before any call of the library."""
    cache = object.__new__(serving.KvCache)
    cache.data = torch.zeros(4, 1, 72 * 64, dtype=torch.uint8)
    cache.kv_heads, cache.head_dim, cache.pages, cache.device = 1, 64, 4, torch.device(device)
    cache._c = serving._Cache(cache.data.data_ptr(), 4, 1, 64, 1.0, 1.0)
    return cache


def test_python_refuses_a_workspace_elsewhere_or_in_pieces():
    cache = _host_cache()
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    table, lens, starts = (torch.tensor(x, dtype=torch.int32) for x in ([[0]], [1], [0, 1]))
    for bad in (torch.zeros(1 << 20, dtype=torch.uint8, device="meta"), torch.zeros(1 << 20, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            serving.kv_attention(q, cache, table, lens, starts, 1, 1, workspace=bad)


def test_python_refuses_eviction_into_a_cache_on_another_device():
    cache, other = _host_cache(), _host_cache("meta")
    table, lens = torch.tensor([[0]], dtype=torch.int32), torch.tensor([1], dtype=torch.int32)
    with pytest.raises(ValueError, match="dst"):
        serving.kv_evict(torch.zeros(1, 1, 1), cache, table, lens, torch.tensor([[1]], dtype=torch.int32), 1, dst=other)
