"""Penalties, biases and grammar masks on logits (gpu) against the float64 oracle.

Tolerance: each of at most five fp32 operations (a division or product, two
subtractions and a product, an addition) rounds its result once, by 2^-24 of its size at
most, and the oracle sums those sizes: |out - ref| <= 2^-24 size (1 + 2^-20), the
last factor for what the earlier roundings add to a later result's size; where
out is bf16 another 2^-8 of the value."""
import numpy as np
import pytest
import torch

import verify_nvfp4_w4a16_amd as nv
import workload
from oracle import draft as odraft
from tests._kv import DEV, int32
from tests.test_gpu_draft import _parents
from tests.test_gpu_kv_ranges import Guarded

pytestmark = pytest.mark.gpu


def _f32(x):
    return torch.tensor(np.asarray(x, np.float32), device=DEV)


class Case:
    """Inputs of both sides: sequences with a history, rows, and whatever the options add."""

    def __init__(self, seed, vocab, new, said, bias=0, states=0, tree=False, kind=torch.float32, strided=False, penalties=True):
        g = workload.rng(seed)
        self.vocab, self.new, self.rows = vocab, list(new), sum(new)
        self.starts = np.concatenate([[0], np.cumsum(new)])
        seqs = len(new)
        self.lens = [said] * seqs if np.isscalar(said) else list(said)
        self.history = g.integers(0, max(1, min(vocab, 50)), (seqs, max(self.lens + [1]))).astype(np.int32)
        self.history[:, 1::3] = g.integers(0, vocab, self.history[:, 1::3].shape)
        self.history[:, 2::7] = g.choice([-1, vocab, vocab - 1, 2 ** 31 - 1, -(2 ** 31)], self.history[:, 2::7].shape)
        self.prompt = [int(g.integers(0, n + 1)) for n in self.lens]
        self.r = g.choice([1.0, 1.2, 0.7, -3.0], seqs).astype(np.float32)
        self.p = g.choice([0.0, 0.6, -0.3], seqs).astype(np.float32)
        self.f = g.choice([0.0, 0.25, -0.1], seqs).astype(np.float32)
        if not penalties:
            self.r[:], self.p[:], self.f[:] = 1.0, 0.0, 0.0
        pitch = vocab + (3 if strided else 0)
        x = g.standard_normal((self.rows, pitch)).astype(np.float32) * 4
        x[:, ::11] = 0.0
        if self.rows:
            x[0, :min(4, vocab)] = [np.nan, np.inf, -np.inf, -0.0][:min(4, vocab)]
        self.wide = torch.tensor(x, device=DEV).to(kind)
        self.logits = self.wide[:, :vocab]
        self.x = self.logits.float().cpu().numpy().astype(np.float64)
        self.kw = dict(prompt_lens=int32(self.prompt), q_starts=int32(self.starts), repetition=_f32(self.r), presence=_f32(self.p),
                       frequency=_f32(self.f))
        self.bias = None
        if bias:
            self.bias = g.integers(0, vocab, (seqs, bias)).astype(np.int32)
            self.bias[:, ::4] = g.choice([-1, vocab, int(self.history[0, 0]) % vocab], self.bias[:, ::4].shape)
            self.values = g.standard_normal((seqs, bias)).astype(np.float32)
            self.kw.update(bias_tokens=int32(self.bias), bias_values=_f32(self.values))
        self.allowed = None
        if states:
            self.allowed = g.integers(0, 2 ** 32, (states, -(-vocab // 32)), dtype=np.uint32)
            self.state = g.integers(-1, states + 1, self.rows)               # both ends are no state
            self.kw.update(allowed=torch.from_numpy(self.allowed.view(np.int32)).to(DEV), allowed_rows=int32(self.state))
        self.drafted = None
        if tree:
            self.drafted = g.integers(0, min(vocab, 30), self.rows).astype(np.int32)
            self.drafted[::5] = g.choice([-1, vocab, vocab - 1])
            self.ways = [w for n in new for w in odraft.ways(_parents(g, n))]
            words = -(-max(new) // 64)
            bits = np.array([odraft.mask_words(w, words) for w in self.ways], np.uint64)
            self.kw.update(drafted=int32(self.drafted), masks=torch.from_numpy(bits.view(np.int64)).to(DEV))

    def call(self, **kw):
        return nv.adjust_logits(self.logits, int32(self.history), int32(self.lens), **{**self.kw, **kw})

    def expected(self, row):
        s = int(np.searchsorted(self.starts[1:], row, side="right"))
        text = self.history[s, :max(self.lens[s], 0)].tolist()
        said = text[self.prompt[s]:]
        if self.drafted is not None:
            said = said + [int(self.drafted[self.starts[s] + a]) for a in self.ways[row]]
        bias = list(zip(self.bias[s].tolist(), self.values[s].astype(np.float64).tolist())) if self.bias is not None else ()
        allowed = None
        if self.allowed is not None and 0 <= self.state[row] < len(self.allowed):
            v = np.arange(self.vocab)
            allowed = (self.allowed[self.state[row], v // 32] >> (v % 32).astype(np.uint32) & 1).astype(bool)
        return odraft.adjust(self.x[row], text[:self.prompt[s]], said, float(self.r[s]), float(self.p[s]), float(self.f[s]), bias, allowed)

    def check(self, out):
        got = out.float().cpu().numpy().astype(np.float64)
        half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 0.0
        for row in range(self.rows):
            want, size = self.expected(row)
            fine = np.isfinite(want)
            assert np.array_equal(np.isnan(got[row]), np.isnan(want)) and np.array_equal(got[row][np.isinf(want)], want[np.isinf(want)]), row
            want, size, value = want[fine], size[fine], got[row][fine]
            off = np.abs(value - want) - (2.0 ** -24 * size * (1 + 2.0 ** -20) + half * np.abs(want))
            assert (off <= 0).all(), (row, off.max(initial=0.0), np.flatnonzero(fine)[off.argmax()])


CASES = [
    dict(vocab=1, new=[1], said=3),
    dict(vocab=7, new=[1, 1], said=[0, 5], bias=2),
    dict(vocab=1000, new=[1] * 5, said=[0, 1, 100, 999, 64], bias=30, states=3),
    dict(vocab=8191, new=[1, 1], said=2000),
    dict(vocab=8192, new=[1, 1], said=2000, bias=1024, states=2),
    dict(vocab=8193, new=[1, 1], said=[2001, 3], strided=True, bias=7),
    dict(vocab=20001, new=[9, 0, 16], said=[500, 3, 0], tree=True, bias=3, states=5),
    dict(vocab=3001, new=[64, 65, 256], said=[50, 0, 333], tree=True),
    dict(vocab=50021, new=[3, 8, 1], said=777, bias=100, states=4),          # several rows a sequence without a tree
    dict(vocab=4097, new=[1, 1, 1], said=100, penalties=False),               # a copy
    dict(vocab=4097, new=[1, 1, 1], said=100, penalties=False, bias=50, states=2),
    dict(vocab=151552, new=[1], said=40000, bias=300),
]


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", CASES)
def test_adjust(case, kind):
    c = Case(seed=case["vocab"], kind=kind, **case)
    out = c.call()
    assert out.dtype == kind and out.is_contiguous()
    c.check(out)
    assert torch.equal(torch.nan_to_num(out.float()), torch.nan_to_num(c.call().float()))


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_out_of_the_other_type_in_place_and_strided(kind):
    c = Case(1, 5003, [2, 5], 300, bias=9, states=3, kind=kind, strided=True)
    other = torch.bfloat16 if kind == torch.float32 else torch.float32
    guarded = Guarded((7, 5010), other)
    untouched = guarded.t[:, 5003:].clone()
    got = c.call(out=guarded.t[:, :5003])
    torch.cuda.synchronize()
    guarded.check()
    c.check(got)
    assert torch.equal(guarded.t[:, 5003:].contiguous().view(torch.uint8), untouched.contiguous().view(torch.uint8))
    want = c.call()
    edge = c.wide[:, 5003:].clone()
    c.call(out=c.logits)                                      # in place: what lies between the rows stays
    assert torch.equal(c.logits.contiguous().view(torch.uint8), want.view(torch.uint8)) and torch.equal(c.wide[:, 5003:], edge)


def test_rows_are_their_own_sequences_without_starts():
    c = Case(2, 2000, [1, 1, 1], [5, 0, 900], bias=4)
    a = c.call()
    b = c.call(q_starts=None)
    assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))
    # without a list of states row r has state r
    states = torch.randint(-2 ** 31, 2 ** 31, (3, 63), device=DEV).int()
    a = nv.adjust_logits(c.logits, allowed=states)
    b = nv.adjust_logits(c.logits, allowed=states, allowed_rows=int32([0, 1, 2]))
    assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)) and bool(torch.isinf(a).any())


def test_only_what_is_given_is_applied():
    c = Case(3, 3000, [1, 1], 200)
    plain = nv.adjust_logits(c.logits)
    assert torch.equal(torch.nan_to_num(plain), torch.nan_to_num(c.logits))
    history = (int32(c.history), int32(c.lens))
    assert torch.equal(torch.nan_to_num(nv.adjust_logits(c.logits, *history)), torch.nan_to_num(plain))
    # without prompt lengths all of the history was said
    got = nv.adjust_logits(c.logits, *history, presence=_f32([0.5, 0.5])).cpu().numpy()
    for row in range(2):
        want, _ = odraft.adjust(c.x[row], [], c.history[row, :c.lens[row]].tolist(), 1.0, 0.5)
        fine = np.isfinite(want)
        assert np.allclose(got[row][fine], want[fine], rtol=0, atol=2.0 ** -24 * 32)


def test_lengths_are_taken_into_their_ranges():
    c = Case(4, 999, [1, 1, 1, 1], 64)
    c.lens, c.prompt = [10 ** 9, -5, 64, 30], [-3, 10, 10 ** 9, 31]
    c.kw["prompt_lens"] = int32(c.prompt)
    out = c.call()
    c.lens, c.prompt = [64, 0, 64, 30], [0, 0, 64, 30]
    c.check(out)


def test_rows_of_no_sequence_and_descending_starts():
    c = Case(5, 9000, [3, 4], 100, bias=5, tree=True)
    out = Guarded((7, 9000), torch.float32)
    out.t.fill_(7.5)
    c.call(q_starts=int32([1, 3, 6]), out=out.t)
    torch.cuda.synchronize()
    out.check()
    assert bool((out.t[0] == 7.5).all()) and bool((out.t[6] == 7.5).all()) and not bool((out.t[1:6] == 7.5).all())
    for order in ([7, 0, 3], [5, 2, 7], [-4, 10 ** 9, 2]):
        out = Guarded((7, 9000), torch.float32)
        c.call(q_starts=int32(order), out=out.t)
        torch.cuda.synchronize()
        out.check()


def test_on_another_stream_and_in_a_graph():
    c = Case(6, 30011, [9, 20], 500, bias=20, states=4, tree=True)
    want = c.call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c.call(stream=side)
    side.synchronize()
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
    out, args = torch.empty_like(want), (int32(c.history), int32(c.lens))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.adjust_logits(c.logits, *args, **c.kw, out=out)
    for _ in range(4):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(want))


def test_refusals_that_need_a_gpu_tensor():
    x = torch.zeros(2, 10, device=DEV)
    for kw in (dict(history=int32([[1], [2]])), dict(history_lens=int32([1, 1])), dict(prompt_lens=int32([1, 1])),
               dict(bias_tokens=int32([[1], [2]])), dict(drafted=int32([1, 2])), dict(allowed_rows=int32([1, 2])),
               dict(repetition=_f32([1.0])), dict(presence=_f32([1.0, 1.0]).double()), dict(frequency=torch.zeros(2)),
               dict(allowed=int32([1, 2])), dict(q_starts=_f32([0, 1, 2])), dict(q_starts=int32([])), dict(out=x[:, :9]), dict(out=x.half()),
               dict(allowed=int32([[1], [2]])[:, :0])):
        with pytest.raises(ValueError):
            nv.adjust_logits(x, **kw)
    # lists of no entries are as none
    for kw in (dict(history=torch.zeros(2, 0, dtype=torch.int32, device=DEV), history_lens=int32([0, 5]), presence=_f32([1.0, 1.0])),
               dict(bias_tokens=torch.zeros(2, 0, dtype=torch.int32, device=DEV), bias_values=torch.zeros(2, 0, device=DEV)),
               dict(allowed=torch.zeros(0, 1, dtype=torch.int32, device=DEV))):
        assert torch.equal(nv.adjust_logits(x, **kw), x)


def test_repetition_at_the_ends_of_its_range():
    # x / r as a product with 1 / r, whose error goes back in: half a step of the result, also where 1 / r is subnormal or
    # has no number; below 2^-126 steps are 2^-149
    r = np.array([1e-40, 2e-39, 1.2e-38, 1e-20, 3.0, 1e20, 1e38, 3e38], np.float32)
    x = np.array([1e-5, 0.3, 7.0, 80.0, -1e-5, -80.0, 3e38, np.inf, 0.0], np.float32)
    logits = _f32(np.tile(x, (len(r), 1)))
    said = int32(np.tile(np.arange(len(x)), (len(r), 1)))
    out = nv.adjust_logits(logits, said, int32([len(x)] * len(r)), repetition=_f32(r)).cpu().numpy().astype(np.float64)
    with np.errstate(over="ignore"):
        want = np.where(x > 0, x.astype(np.float64) / r[:, None].astype(np.float64), x.astype(np.float64) * r[:, None].astype(np.float64))
    most = float(np.finfo(np.float32).max)
    far = np.abs(want) >= most * (1 + 2.0 ** -25)
    assert np.array_equal(out[far], np.sign(want[far]) * np.inf)
    near = ~far
    assert np.all(np.abs(out[near] - want[near]) <= 2.0 ** -24 * (1 + 2.0 ** -20) * np.abs(want[near]) + 2.0 ** -149)


def test_more_logits_than_a_launch_takes():
    rows, vocab = 8200, 1 << 22
    if torch.cuda.mem_get_info()[0] < 90e9:
        pytest.skip("70 GB of logits")
    logits = torch.zeros((rows, vocab), dtype=torch.bfloat16, device=DEV)
    tokens = int32(np.stack([np.arange(rows) * 511, np.full(rows, vocab - 1)], 1))
    values = _f32(np.stack([1.0 + np.arange(rows) % 128, np.full(rows, -3.0)], 1))
    nv.adjust_logits(logits, bias_tokens=tokens, bias_values=values, out=logits)
    for row in (0, 1, 4095, 8190, 8191, 8192, 8199):
        at = logits[row].nonzero().flatten().tolist()
        assert at == [row * 511, vocab - 1], (row, at)
        assert logits[row, at].tolist() == [1.0 + row % 128, -3.0]
    del logits
    torch.cuda.empty_cache()


def test_repetition_is_a_rounded_quotient():
    g = workload.rng(31)
    rows, vocab = 64, 20000
    x = (g.standard_normal((rows, vocab)) * 8).astype(np.float32)
    r = g.uniform(0.5, 2.0, rows).astype(np.float32)
    r[:3] = [1.1, 1.0 + 2.0 ** -23, 2.0 - 2.0 ** -23]
    said = int32(np.tile(np.arange(vocab), (rows, 1)))
    out = nv.adjust_logits(_f32(x), said, int32([vocab] * rows), repetition=_f32(r)).cpu().numpy()
    assert np.array_equal(out, np.where(x > 0, x / r[:, None], x * r[:, None]))
