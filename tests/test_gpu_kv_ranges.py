"""The paged NVFP4 cache on the GPU (gpu) at the ends of what its calls accept:
windows, scales, caps and bounds of any size, against the float64 oracle.

Tolerances are test_gpu_kv.py's where not said otherwise."""
import numpy as np
import pytest
import torch

import verify_nvfp4_w4a16_amd as nv
import workload
from oracle import bf16_bits_to_f64
from oracle import kv as okv
from tests._kv import DEV, PAGE, Paged, bf16, int32, starts, stored
from tests.test_gpu_kv import _attend, _check, _query_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,group", [(1, 4), (12, 4), (40, 4)])
@pytest.mark.parametrize("window", [1500, 1 << 31, (1 << 63) - 1])
def test_attention_with_a_window_that_no_sequence_fills(new, group, window):
    # few, 33 to 64 and more rows a kv head; parts of pages among them
    lens = [1500, 70, 1]
    news = [new, min(new, 70), 1]
    c = Paged(lens, 1, 64, 201)
    qb = _query_bits(sum(news), group, 64, 202)
    none = _attend(c, qb, news)
    wide = _attend(c, qb, news, window=window)
    _check(c, qb, news, *wide)
    assert np.array_equal(none[0], wide[0]) and np.array_equal(none[1], wide[1])


def _pool_of(address):
    """The stream whose pool of torch's allocator the address lies in."""
    for segment in torch.cuda.memory_snapshot():
        if segment["address"] <= address < segment["address"] + segment["total_size"]:
            return segment["stream"]
    raise AssertionError("not an address of the allocator")


def test_what_a_call_makes_belongs_to_its_stream(monkeypatch):
    """A block that the current stream's pool hands out may be in use by work queued there, so
    results and workspaces for another stream come from that stream's pool."""
    from verify_nvfp4_w4a16_amd import serving
    lib, scratch = serving._kv(), []
    for name, place in (("nvfp4_kv_attention", 5), ("nvfp4_sample", 12)):
        def spy(*args, real=getattr(lib, name), place=place):
            scratch.append(args[place])
            return real(*args)
        monkeypatch.setattr(lib, name, spy)
    c = Paged([3000, 70], 1, 64, 211, extra=2)
    q, st = bf16(_query_bits(2, 2, 64, 212)), starts([1, 1])
    logits, u = torch.zeros(2, 500, device=DEV), torch.full((2,), 0.5, device=DEV)
    dst = int32([[c.free[0]], [c.free[1]]])
    args = (c.cache, c.table_t, c.lens_t, st)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def calls(stream):
        out, lse = nv.kv_attention(q, *args, 1, 3000, stream=stream)
        w = nv.kv_weights(q, lse, *args, 1, 3000, stream=stream)
        return [out, lse, w, *nv.kv_read(*args, 2, stream=stream), *nv.sample(logits, u, stream=stream),
                *nv.kv_evict(w, c.cache, c.table_t, c.lens_t, dst, 64, stream=stream)]

    here, first = calls(None), scratch[:]
    there, second = calls(side), scratch[2:]
    side.synchronize()
    torch.cuda.synchronize()
    assert len(first) == len(second) == 2 and all(first) and all(second)
    assert set(first).isdisjoint(second)
    for x in [t.data_ptr() for t in there] + second:
        assert _pool_of(x) == side.cuda_stream
    for x in [t.data_ptr() for t in here] + first:
        assert _pool_of(x) == torch.cuda.current_stream().cuda_stream
    for a, b in zip(here, there):
        assert torch.equal(a, b)


class Guarded:
    """A tensor inside a larger one whose other elements hold a pattern of their own."""

    def __init__(self, shape, dtype, fill=None):
        self.n, self.pad = int(np.prod(shape)), 4096
        size = torch.empty((), dtype=dtype).element_size()
        self.all = torch.full(((self.n + 2 * self.pad) * size,), 0xA5, dtype=torch.uint8, device=DEV)
        self.t = self.all.view(dtype)[self.pad:self.pad + self.n].view(shape)
        self.untouched = self.t.clone()
        if fill is not None:
            self.t.copy_(fill)
        self.edge = self.pad * size

    def check(self):
        assert bool((self.all[:self.edge] == 0xA5).all()) and bool((self.all[-self.edge:] == 0xA5).all())
        return self.t


@pytest.mark.parametrize("new", [[5, 9], [40, 30]])
def test_descending_starts_touch_nothing_beyond_the_arrays(new):
    """Which rows are computed is not defined, but guards around every array stay as they were."""
    d, heads = 64, 4
    c = Paged([3000, 90, 500], 2, d, 221)
    total = sum(new) + 20
    for order in ([total, 0, new[0], new[0] + new[1]], [7, 3, total, 0], [new[0] + 1, new[0] + 2, 0, new[0]]):
        data = Guarded(c.data.shape, torch.uint8, c.data)
        cache = nv.KvCache(data.t, 2, d, c.k_scale, c.v_scale)
        before = data.t.clone()
        rows = bf16(workload.activations_bf16(total, 4 * d, 222).reshape(total, 4, d))
        st = int32(order)
        q = bf16(_query_bits(total, heads, d, 223))
        args = (cache, c.table_t, c.lens_t, st)
        out, lse = Guarded((total, heads, d), torch.bfloat16), Guarded((total, heads), torch.float32)
        k, v = (Guarded((total, 2, d), torch.bfloat16) for _ in range(2))
        w = Guarded((3, 2, 3000), torch.float32)
        ws = nv.kv_attention_workspace(cache, q, c.table_t, c.lens_t, st, max(new), 3000)
        ws = Guarded((ws,), torch.uint8) if ws else None
        nv.kv_attention(q, *args, max(new), 3000, out=out.t, lse=lse.t, workspace=ws and ws.t)
        nv.kv_read(*args, total, k=k.t, v=v.t)
        nv.kv_weights(q, torch.zeros_like(lse.t), *args, max(new), 3000, out=w.t)
        assert torch.equal(data.t, before)
        nv.kv_append(cache, rows[:, :2], rows[:, 2:], c.table_t, c.lens_t, st)
        torch.cuda.synchronize()
        for x in (data, out, lse, k, v, w, ws):
            if x is not None:
                x.check()


# few, 33 to 64 and more rows a kv head
ROWS = [(1, 4), (12, 4), (40, 4)]


@pytest.mark.parametrize("new,group", ROWS)
@pytest.mark.parametrize("kw", [{}, dict(window=100), dict(causal=False), dict(softcap=3.0)])
def test_attention_at_scale_zero(new, group, kw):
    # all slots that a query sees weigh alike
    lens = [3000, 90, 5]
    news = [new, new, 1]
    c = Paged(lens, 1, 64, 231)
    qb = _query_bits(sum(news), group, 64, 232)
    _check(c, qb, news, *_attend(c, qb, news, scale=0.0, **kw), scale=0.0, **kw)


@pytest.mark.parametrize("new,group", ROWS)
def test_attention_of_zero_queries_over_small_keys(new, group):
    lens, news = [700, 90], [new, new]
    c = Paged(lens, 1, 128, 233, k_scale=2.0 ** -100)
    qb = _query_bits(sum(news), group, 128, 234)
    qb[::2, 1:] = 0
    _check(c, qb, news, *_attend(c, qb, news))


@pytest.mark.parametrize("t", [2.0 ** -149, 1e-40, 4.8e-40, 5e-40, 2.0 ** -126, 2.0 ** -115, 5.6e37, 5.8e37, 1e38, 3.4e38])
def test_append_at_the_ends_of_the_tensor_scale(t):
    """Codes, scales and read values at tensor scales whose sixfold, or its inverse, fp32 does not hold."""
    d, n = 64, 192
    t = float(np.float32(t))
    g = workload.rng(241)
    # magnitudes from far below the scale's smallest step to beyond its largest
    size = np.exp(g.uniform(-9, 10, (n, 2, d // 16, 1))) * t
    x = np.clip(g.standard_normal((n, 2, d // 16, 16)) * size, -3.3e38, 3.3e38).astype(np.float32)
    x[0] = 0.0
    x[1, :, 0] = 0.0
    x[2, :, 1, 3] = np.inf
    bits = workload.f32_to_bf16_bits(x.reshape(n, 2, d))
    rows = bf16(bits)
    cache = nv.KvCache.empty(3, 1, d, t, t)
    where = (int32([[2, 0, 1]]), int32([n]), int32([0, n]))
    nv.kv_append(cache, rows[:, :1], rows[:, 1:], *where)
    read = nv.kv_read(cache, *where, n)
    torch.cuda.synchronize()
    got = stored(cache.data.cpu().numpy(), [2, 0, 1], n, 0, d)
    for which in (0, 1):
        codes, scales = okv.quantise_rows(bits[:, which], t)
        assert np.array_equal(got[2 * which + 1], scales)
        assert np.array_equal(got[2 * which], codes)
        with np.errstate(over="ignore"):
            val = okv.values(codes, scales, 1.0).astype(np.float32) * np.float32(t)
        back = read[which][:, 0].view(torch.int16).cpu().numpy().view(np.uint16)
        assert np.array_equal(workload.bf16_bits_to_f32(back), workload.bf16_bits_to_f32(workload.f32_to_bf16_bits(val)))


@pytest.mark.parametrize("new,group", ROWS)
@pytest.mark.parametrize("cap", [1e-40, 0.02, 50.0, 1e3, 1e4, 1e6, 1e8, 1e30, 3.4e38])
def test_attention_with_a_cap_of_any_size(new, group, cap):
    """A capped score is off by a relative 2^-20 beside its sum's own error, whatever the cap."""
    lens, news, d = [300, 70], [new, new], 64
    c = Paged(lens, 1, d, 251)
    qb = _query_bits(sum(news), group, d, 252)
    out, lse = _attend(c, qb, news, softcap=cap)
    q, at = bf16_bits_to_f64(qb), 0
    for s, n in enumerate(lens):
        for h in range(group):
            k, v = c.k[s][0], c.v[s][0]
            o, l, spread, size = okv.attention(q[at:at + new, h], k, v, d ** -0.5, softcap=cap)
            # both scores of a difference, and the exponential's own 2^-20
            eps = (2 * (d + 8) * 2.0 ** -24 + 2 * 2.0 ** -20) * size[:, None] + 2.0 ** -20
            tol = 2.0 ** -8 * np.abs(o) + (eps + 2.0 ** -10) * spread + (n + 1) * 2.0 ** -24 * np.abs(v).max()
            assert np.all(np.abs(out[at:at + new, h] - o) <= tol), (s, h)
            lim = eps[:, 0] + n * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(l))
            assert np.all(np.abs(lse[at:at + new, h] - l) <= lim), (s, h, float((np.abs(lse[at:at + new, h] - l) / lim).max()))
        at += new


@pytest.mark.parametrize("cap", [0.02, 50.0, 1e4, 1e8])
def test_slot_weights_with_a_cap_of_any_size(cap):
    n, new, group, d = 200, 9, 4, 64
    c = Paged([n], 1, d, 253)
    qb = _query_bits(new, group, d, 254)
    q64 = bf16_bits_to_f64(qb)
    lses = np.stack([okv.attention(q64[:, h], c.k[0][0], c.v[0][0], d ** -0.5, softcap=cap)[1] for h in range(group)], 1).astype(np.float32)
    got = nv.kv_weights(bf16(qb), torch.from_numpy(lses).to(DEV), c.cache, c.table_t, c.lens_t, starts([new]), new, n, softcap=cap)
    got = got.cpu().numpy()[0, 0].astype(np.float64)
    want, size = np.zeros(n), np.zeros(n)
    for h in range(group):
        w, z = okv.slot_weights(q64[:, h], c.k[0][0], lses[:, h].astype(np.float64), d ** -0.5, softcap=cap)
        want, size = want + w, size + z
    # as test_slot_weights has it, with the cap's relative 2^-20 of a score in place of a part of the cap
    tol = (2 * (d + 8) * 2.0 ** -24 + 2.0 ** -20) * size + (2.0 ** -20 + (new * group + 2) * 2.0 ** -24 + np.abs(lses).max() * 2.0 ** -22) * want
    assert np.all(np.abs(got - want) <= tol + 1e-30), float((np.abs(got - want) / tol).max())


@pytest.mark.parametrize("new,group", ROWS)
def test_attention_where_the_scales_product_is_too_small_for_fp32(new, group):
    """A product that has five bits in fp32, between the largest keys and the largest queries, whose scores are ordinary."""
    n, d = 90, 256
    k_scale, scale = float(np.float32(2.0 ** -70)), float(np.float32(16.5 * 2.0 ** -79))
    g = workload.rng(261)
    kv = np.where(g.random((n, 2, d)) < 0.5, -1.0, 1.0).astype(np.float32) * np.float32(2688 * 2.0 ** -70)
    kv[::9, 0] = abs(kv[::9, 0])                                # scores near the largest, the others' near 0
    bits = workload.f32_to_bf16_bits(kv)
    rows = bf16(bits)
    c = Paged([n], 1, d, 262, k_scale=k_scale, v_scale=k_scale)
    nv.kv_append(c.cache, rows[:, :1], rows[:, 1:], c.table_t, c.lens_t, int32([0, n]))
    for x, col in ((c.k, 0), (c.v, 1)):
        codes, scales = okv.quantise_rows(bits[:, col], k_scale)
        x[0] = okv.values(codes, scales, k_scale)[None]
    qb = workload.f32_to_bf16_bits(np.full((new, group, d), 1.5 * 2.0 ** 126, np.float32))
    out, lse = _attend(c, qb, [new], scale=scale)
    _check(c, qb, [new], out, lse, scale=scale)
    w = nv.kv_weights(bf16(qb), torch.from_numpy(lse).float().to(DEV), c.cache, c.table_t, c.lens_t, starts([new]), new, n, scale=scale)
    # each query's weights over what it sees sum to 1, but for lse's rounding and the scores' errors
    assert abs(float(w.double().sum()) - new * group) <= 1e-4 * new * group


@pytest.mark.parametrize("new,group", ROWS)
@pytest.mark.parametrize("v_scale", [2.0 ** -126, 2.0 ** -100, 2.0 ** 100])
def test_attention_of_one_value_at_the_ends_of_v_s_tensor_scale(new, group, v_scale):
    # weights that sum to one give the value itself, whatever the sum was before
    n, d = 207126, 64
    cache = nv.KvCache.empty(-(-n // PAGE), 1, d, 2.0 ** -6, v_scale)
    where = (int32(np.arange(-(-n // PAGE))[None]), int32([n]))
    rows = torch.randn(n, 2, d, generator=torch.Generator(device=DEV).manual_seed(271), device=DEV).bfloat16()
    rows[:, 1] = 6.0 * v_scale
    nv.kv_append(cache, rows[:, :1], rows[:, 1:], *where, int32([0, n]))
    q = bf16(_query_bits(new, group, d, 272))
    for scale in (None, 0.0):
        out, lse = nv.kv_attention(q, cache, *where, int32([0, new]), new, n, scale=scale)
        got = out.float().cpu().numpy().astype(np.float64) / (6.0 * v_scale)
        # f16 weights against the fp32 sum of the same weights, and the output's rounding
        assert np.all(np.abs(got - 1) <= 2.0 ** -8 + 2.0 ** -10), float(np.abs(got - 1).max())
        if scale == 0.0:
            seen = n - new + 1 + np.arange(new)[:, None]
            assert np.all(np.abs(lse.cpu().numpy() - np.log(seen)) <= n * 2.0 ** -24 + 1e-5)


@pytest.mark.parametrize("new,group", ROWS)
def test_attention_keeps_the_mass_of_many_small_weights(new, group):
    """Every 32nd slot, whose value is zero, has 2^26 times the weight of each other.

    A weight enters the second product as f16 times 2^7, so it is off by half of f16's
    smallest step, 2^-32 of the largest weight, at most; twice that is allowed."""
    n, d = 4000, 64
    large = np.arange(n) % 32 == 0
    kv = np.zeros((n, 2, d), np.float32)
    kv[large, 0, 0] = 6.0
    kv[~large, 1] = 6.0
    kv[1::2, 1, ::2] = 3.0
    rows = bf16(workload.f32_to_bf16_bits(kv))
    c = Paged([n], 1, d, 281, k_scale=2.0 ** -3, v_scale=2.0 ** -3)
    nv.kv_append(c.cache, rows[:, :1], rows[:, 1:], c.table_t, c.lens_t, int32([0, n]))
    q = np.zeros((new, group, d), np.float32)
    q[..., 0] = 3.0
    scale = 26 * np.log(2.0) / 18                              # those slots' score is 26 log 2, all others' 0
    out, lse = _attend(c, workload.f32_to_bf16_bits(q), [new], scale=scale)
    v, top = kv[:, 1].astype(np.float64), np.exp(18 * float(np.float32(scale)))
    for i in range(new):
        seen = n - new + i + 1
        many, few = int((~large[:seen]).sum()), int(large[:seen].sum())
        mass = few * top + many
        ref = v[:seen].sum(0) / mass
        tol = (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -13) * ref + 2 * many * 2.0 ** -32 * 6.0 / few
        assert np.all(np.abs(out[i] - ref) <= tol), (i, float((np.abs(out[i] - ref) / tol).max()))
        assert np.all(np.abs(lse[i] - np.log(mass)) <= 1e-5)


def test_workspaces_elsewhere_or_in_pieces_are_refused():
    c = Paged([200], 1, 64, 301)
    q, logits, u = bf16(_query_bits(1, 2, 64, 302)), torch.zeros(1, 500, device=DEV), torch.zeros(1, device=DEV)
    for bad in (torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            nv.kv_attention(q, c.cache, c.table_t, c.lens_t, starts([1]), 1, 200, workspace=bad)
        with pytest.raises(ValueError, match="workspace"):
            nv.sample(logits, u, workspace=bad)


@pytest.mark.parametrize("max_q,max_kv", [(8, 128), (8, 1100), (20, 128), (70, 1100)])
def test_sequences_beyond_the_bounds_count_as_ones_of_that_size(max_q, max_kv):
    """A sequence with more slots or new tokens than the call's bounds is taken for one that ends
    there: its first max_q rows are those of max_kv slots, and nothing else is written."""
    lens, new, d, heads = [1500, 40], [90, 1], 64, 4
    c = Paged(lens, 1, d, 291)
    total = sum(new)
    qb = _query_bits(total, heads, d, 292)
    q, st = bf16(qb), starts(new)
    args = (c.cache, c.table_t, c.lens_t, st, max_q, max_kv)
    out, lse, w = Guarded((total, heads, d), torch.bfloat16), Guarded((total, heads), torch.float32), Guarded((2, 1, max_kv), torch.float32)
    n = nv.kv_attention_workspace(c.cache, q, c.table_t, c.lens_t, st, max_q, max_kv)
    ws = Guarded((n,), torch.uint8) if n else None
    nv.kv_attention(q, *args, out=out.t, lse=lse.t, workspace=ws and ws.t)
    nv.kv_weights(q, lse.t, *args, out=w.t)
    torch.cuda.synchronize()
    if ws:
        ws.check()
    got, got_lse = out.check().float().cpu().numpy().astype(np.float64), lse.check().cpu().numpy().astype(np.float64)
    # rows past max_q are as they were
    assert torch.equal(out.t[max_q:90].view(torch.int16), out.untouched[max_q:90].view(torch.int16))
    assert torch.equal(lse.t[max_q:90].view(torch.int32), lse.untouched[max_q:90].view(torch.int32))
    kept = np.r_[0:max_q, 90]
    c.k, c.v = [x[:, :max_kv] for x in c.k], [x[:, :max_kv] for x in c.v]
    c.lens = [min(x, max_kv) for x in lens]
    _check(c, qb[kept], [max_q, 1], got[kept], got_lse[kept])
    got_w, q64 = w.check().cpu().numpy().astype(np.float64), bf16_bits_to_f64(qb)
    for s, rows in enumerate((range(0, max_q), [90])):
        want, size = np.zeros(c.lens[s]), np.zeros(c.lens[s])
        for h in range(heads):
            x, z = okv.slot_weights(q64[rows, h], c.k[s][0], got_lse[rows, h], d ** -0.5)
            want, size = want + x, size + z
        tol = 2 * (d + 8) * 2.0 ** -24 * size + (2.0 ** -20 + (len(rows) * heads + 2) * 2.0 ** -24 + np.abs(got_lse[rows]).max() * 2.0 ** -22) * want
        assert np.all(np.abs(got_w[s, 0, :c.lens[s]] - want) <= tol + 1e-30), s
        assert not got_w[s, 0, c.lens[s]:].any()
