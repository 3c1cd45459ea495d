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
