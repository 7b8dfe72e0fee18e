"""Hand-worked pins of the key/value cache oracle (no GPU)."""
import math

import numpy as np
import pytest
import torch

from oracle.kv import PAGE, KvError, KvOracle, e4m3_round, scale_for


def test_e4m3_round_agrees_with_torch_on_every_code_and_between():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    vals = codes[~torch.isnan(codes)].double().numpy()
    assert np.array_equal(e4m3_round(vals), vals)
    u = np.unique(np.abs(vals))
    mids = (u[1:] + u[:-1]) / 2
    x = np.concatenate([mids, np.nextafter(mids, 0), np.nextafter(mids, 1e9), -mids]).astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(e4m3_round(x), want)
    assert e4m3_round(np.array(1e9)) == 448 and np.isnan(e4m3_round(np.array(np.nan)))


def test_scale_is_the_smallest_power_of_two():
    assert scale_for(448.0) == 1.0 and scale_for(np.nextafter(448.0, 1e9)) == 2.0 and scale_for(224.0) == 0.5
    assert scale_for(0.0) == 2.0 ** -40 and scale_for(math.inf) == 2.0 ** 40


def test_reserve_takes_lowest_pages_in_list_order_and_copies_shared_ones():
    o = KvOracle(1, 8, 1, 4, 3, 3)
    o.reserve([70, 10], [2, 0])                     # row 2: pages 0, 1; row 0: page 2
    assert o.table[2, :2].tolist() == [0, 1] and o.table[0, 0] == 2
    o.fork([2], [1])
    assert o.refs[:3].tolist() == [2, 2, 1]
    o.reserve([1, 1], [1, 2])                       # both write page 1: row 1 copies, row 2 keeps it
    assert o.table[1, :2].tolist() == [0, 3] and o.table[2, :2].tolist() == [0, 1]
    assert o.refs[:4].tolist() == [2, 1, 1, 1] and o.len.tolist() == [10, 71, 71]
    with pytest.raises(KvError):
        o.reserve([3 * PAGE], [0])
    assert o.len[0] == 10


def test_release_under_a_window_and_compact():
    o = KvOracle(1, 6, 1, 4, 2, 5)
    o.reserve([64 * 4], [0])
    o.reserve([5], [1])
    o.release([0], window=65, sinks=1)              # later queries see j > 256 - 65 = 191 and j < 1
    assert o.table[0, :4].tolist() == [0, -1, -1, 3]
    o.k[0, 3, 0] = 3.0
    o.compact()                                      # used 0, 3, 4 -> 4 into 1 ... the ascending pairing
    assert o.table[0, :4].tolist() == [0, -1, -1, 1] and o.table[1, 0] == 2
    assert (o.k[0, 1, 0] == 3.0).all() and o.refs.tolist() == [1, 1, 1, 0, 0, 0]


def test_append_grows_the_scale_and_rescales():
    o = KvOracle(1, 1, 1, 2, 1, 1)
    o.reserve([1])
    o.append(0, np.array([[[1.0, 448.0]]]), np.array([[[0.5, 0.25]]]), [1])
    assert o.ks[0, 0, 0] == 1.0 and o.k[0, 0, 0, 0].tolist() == [1.0, 448.0]
    o.reserve([1])
    o.append(0, np.array([[[900.0, 0.0]]]), np.array([[[0.5, np.nan]]]), [1])
    assert o.ks[0, 0, 0] == 4.0 and o.k[0, 0, 0, 0].tolist() == [0.25, 112.0]
    assert np.isnan(o.k[0, 0, 0, 1, 0]) and o.k[0, 0, 0, 1, 1] == 0.0 and o.v[0, 0, 0, 1, 1] == 0.0


def test_attend_by_hand():
    o = KvOracle(1, 2, 1, 1, 1, 2)
    o.reserve([3])
    o.append(0, np.array([[[0.0]], [[1.0]], [[2.0]]]), np.array([[[1.0]], [[2.0]], [[4.0]]]), [3])
    y, _, _ = o.attend(0, np.ones((3, 1, 1)), [3], 1.0)
    e = math.e
    assert np.allclose(y[:, 0, 0], [1.0, (1 + 2 * e) / (1 + e), (1 + 2 * e + 4 * e * e) / (1 + e + e * e)])
    y, _, _ = o.attend(0, np.ones((3, 1, 1)), [3], 1.0, window=1, sinks=1)
    assert np.allclose(y[:, 0, 0], [1.0, (1 + 2 * e) / (1 + e), (1 + 4 * e * e) / (1 + e * e)])
    y, _, _ = o.attend(0, np.ones((5, 1, 1)), [5], 1.0)   # two queries before the first key see nothing
    assert (y[:2] == 0).all() and y[2, 0, 0] == 1.0
