"""Token sampling on the GPU (gpu) against exact integer masses in Python.

A token's mass is floor(2^30 exp d) with the exponential in fp32 there and in
float64 here: at most 2^-22 of the value and one unit apart.  The masses
compared are sums of such, so decisions that fall by a relative margin of more
than 1e-5 (2^-22 with a wide factor, and a unit each for up to 2^12 of tokens)
are the same; rows where the oracle's margin is smaller are left out, and the
test asserts that few are."""
import numpy as np
import pytest
import torch

import verify_nvfp4_w4a16_amd as nv
import workload
from oracle.sample import sample as sample_ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")

PARAMS = [(1.0, 0, 1.0, 0.0), (0.7, 50, 0.95, 0.0), (1.3, 0, 0.9, 0.0), (0.9, 0, 1.0, 0.05), (0.0, 0, 1.0, 0.0),
          (1.0, 1, 1.0, 0.0), (0.6, 20, 0.5, 0.2), (2.0, 7, 1.0, 0.0), (1.0, 0, 0.0, 0.0), (1.0, 0, 1.0, 2.0),
          (1.0, 3, 0.999, 0.0), (5.0, 0, 0.3, 0.0), (1e-6, 0, 0.9, 0.0), (1.0, 10 ** 9, 0.8, 0.0)]


def _run(x, u, params, dtype):
    cols = list(zip(*params))
    t = [torch.tensor(c, dtype=torch.int32 if i == 1 else torch.float32, device=DEV) for i, c in enumerate(cols)]
    logits = torch.from_numpy(x).to(DEV).to(dtype)
    tok, lp = nv.sample(logits, torch.tensor(u, dtype=torch.float32, device=DEV), *t)
    tok2, lp2 = nv.sample(logits, torch.tensor(u, dtype=torch.float32, device=DEV), *t)
    torch.cuda.synchronize()
    assert torch.equal(tok, tok2) and torch.equal(lp, lp2)
    return logits.float().cpu().numpy(), tok.cpu().numpy(), lp.cpu().numpy()


def _compare(x, u, params, dtype, most_left_out):
    x, tok, lp = _run(x, u, params, dtype)
    left = 0
    for r, (t, k, p, m) in enumerate(params):
        want, want_lp, margin = sample_ref(x[r], u[r], t, k, p, m)
        if margin < 1e-5:
            left += 1
            continue
        assert tok[r] == want, (r, params[r], margin)
        assert abs(lp[r] - want_lp) <= 1e-5 + 2.0 ** -22 * abs(want_lp) or lp[r] == want_lp, (r, params[r])
    assert left <= most_left_out, left


@pytest.mark.parametrize("vocab", [1, 2, 63, 64, 65, 1000, 4097])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sample(vocab, dtype):
    g = workload.rng(90 + vocab)
    rows = len(PARAMS) * 3
    x = (g.standard_normal((rows, vocab)) * 3).astype(np.float32)
    u = g.random(rows).astype(np.float32).tolist()
    _compare(x, u, PARAMS * 3, dtype, rows // 6)


def test_sample_a_large_vocabulary():
    g = workload.rng(95)
    x = (g.standard_normal((len(PARAMS), 151552)) * 2).astype(np.float32)
    x[:, g.integers(0, 151552, 30)] += 9
    u = g.random(len(PARAMS)).astype(np.float32).tolist()
    _compare(x, u, PARAMS, torch.float32, 6)     # a broad tail has a boundary every 1e-5 or so


def test_sample_equal_logits_take_the_lowest_index():
    x = np.zeros((6, 300), np.float32)
    x[4] = 1.0
    x[4, 7] = x[4, 200] = 3.0
    params = [(1.0, 0, 1.0, 0.0), (1.0, 10, 1.0, 0.0), (1.0, 0, 0.25, 0.0), (0.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0), (1.0, 10, 0.5, 0.0)]
    u = [0.5, 0.95, 0.9999, 0.7, 0.7, 0.9999]
    _, tok, lp = _run(x, u, params, torch.float32)
    # all weights are 2^30: 300 stay; the first 10; the first 75; the first maximum; the first of the two; 5 of 10
    assert tok.tolist() == [150, 9, 74, 0, 7, 4]
    assert np.allclose(lp, [-np.log(300), -np.log(10), -np.log(75), 0, 0, -np.log(5)], rtol=2.0 ** -20, atol=0)


@pytest.mark.parametrize("vocab,step", [(3000, 0.5), (20000, 0.125), (20001, 2.0), (60000, 1.0)])
def test_sample_many_equal_logits(vocab, step):
    """Cuts among hundreds to tens of thousands of tokens of one weight: only the index decides."""
    g = workload.rng(96)
    ks = [1, 5, 64, 65, 200, 257, 1000, 2999, 9000, 15000]
    x = np.round(g.standard_normal((2 * len(ks), vocab)) / step).astype(np.float32) * np.float32(step)
    params = [(1.0, k, 1.0, 0.0) for k in ks] + [(0.7, k, 0.9, 0.0) for k in ks]
    u = g.random(2 * len(ks)).astype(np.float32).tolist()
    _compare(x, u, params, torch.float32, 6)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [3, 8, 9, 1003, 16384, 16391, 33001])
def test_sample_rows_at_any_address(vocab, dtype):
    # rows read 16 bytes at a time from wherever they begin give what whole ones give
    g = workload.rng(97)
    n = len(PARAMS)
    wide = torch.from_numpy((g.standard_normal((n, vocab + 11)) * 3).astype(np.float32)).to(DEV).to(dtype)
    wide[:, 5 + vocab:] = 100.0                               # beyond a row lies what would win
    wide[:, :5] = 100.0
    u = torch.from_numpy(g.random(n).astype(np.float32)).to(DEV)
    t = [torch.tensor(c, dtype=torch.int32 if i == 1 else torch.float32, device=DEV) for i, c in enumerate(zip(*PARAMS))]
    rows = wide[:, 5:5 + vocab]
    padded = torch.full((n, (vocab + 15) // 8 * 8), float("-inf"), device=DEV, dtype=dtype)
    padded[:, :vocab] = rows
    got, lp = nv.sample(rows, u, *t)
    want, want_lp = nv.sample(padded, u, *t)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(lp, want_lp)


def test_sample_a_temperature_whose_inverse_is_infinite():
    x = np.full((4, 1000), -3.0, np.float32)
    x[:, [10, 500, 999]] = 2.0                                # below the maximum nothing has a weight, and all of it stays
    x[3, 500] = np.nan
    _, tok, lp = _run(x, [0.0, 0.5, 0.9, 0.6], [(1e-40, 0, 1.0, 0.0), (1e-40, 0, 1.0, 0.0), (1e-40, 3, 1.0, 0.0), (1e-40, 0, 1.0, 0.0)], torch.float32)
    assert tok.tolist() == [10, 500, 999, 999]
    assert np.allclose(lp, np.log([1 / 3, 1 / 3, 1 / 3, 1 / 2]), atol=1e-6)


def test_sample_ends_of_the_random_number():
    x = np.zeros((4, 5), np.float32)
    x[:, 0] = x[:, 4] = -np.inf
    _, tok, _ = _run(x, [0.0, float(np.nextafter(np.float32(1), np.float32(0))), 1.0, 1 / 3], [(1.0, 0, 1.0, 0.0)] * 4, torch.float32)
    assert tok[0] == 1 and tok[1] == 3 and tok[2] == 3 and tok[3] in (1, 2)


def test_sample_rows_without_finite_logits():
    x = np.zeros((6, 70), np.float32)
    x[0] = -np.inf
    x[1] = np.nan
    x[2, ::2] = np.nan
    x[3] = -np.inf
    x[3, 69] = -1e30
    x[4, 5] = np.inf
    x[5, :] = -np.inf
    x[5, 3] = np.nan
    _, tok, lp = _run(x, [0.0] * 6, [(1.0, 0, 0.9, 0.0)] * 6, torch.float32)
    assert tok.tolist() == [-1, -1, 1, 69, 5, -1]
    assert np.isneginf(lp[[0, 1, 5]]).all() and lp[3] == 0 and lp[4] == 0


def test_sample_defaults_strided_rows_and_another_stream():
    g = workload.rng(97)
    wide = torch.from_numpy(g.standard_normal((9, 700)).astype(np.float32)).to(DEV)
    u = torch.from_numpy(g.random(9).astype(np.float32)).to(DEV)
    view = wide[:, :333]
    a = nv.sample(view, u)
    b = nv.sample(view.contiguous(), u, *(torch.full((9,), v, dtype=d, device=DEV) for v, d in
                                          ((1.0, torch.float32), (0, torch.int32), (1.0, torch.float32), (0.0, torch.float32))))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = nv.sample(view, u, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_sample_in_a_graph():
    g = workload.rng(98)
    x = torch.from_numpy((g.standard_normal((3, 5000)) * 3).astype(np.float32)).to(DEV)
    u = torch.from_numpy(g.random(3).astype(np.float32)).to(DEV)
    p = torch.full((3,), 0.9, device=DEV)
    tok = torch.empty(3, dtype=torch.int32, device=DEV)
    lp = torch.empty(3, device=DEV)
    nv.sample(x, u, top_p=p, token=tok, logprob=lp)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.sample(x, u, top_p=p, token=tok, logprob=lp)
    for i in range(4):
        x.copy_(torch.from_numpy((g.standard_normal((3, 5000)) * 3).astype(np.float32)))
        graph.replay()
        torch.cuda.synchronize()
        got = tok.clone(), lp.clone()
        want = nv.sample(x, u, top_p=p)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
