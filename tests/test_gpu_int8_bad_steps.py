"""Steps of the 8-bit cache whose numbers do not fit together: what is wrong of one sequence leaves the others as they are.
Bounds and definitions as in test_gpu_int8.py."""
import numpy as np
import pytest

from oracle import int8
from test_gpu_int8 import BF16, F32, Setup, dev, tq, wide  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def runs(starts, lengths, n):
    """Sequences with tokens."""
    return [b for b in range(len(lengths)) if 0 <= starts[b] < starts[b + 1] <= n and lengths[b] >= 0]


def check_rows(tq, s, starts, lengths, served):
    """append and read: the rows of the sequences `served` and of no other, and the fault bit."""
    cache, t, table, _, _ = s.device(tq)
    st, le = dev(starts), dev(lengths)
    tq.append_int8(s.K.cuda(), s.V.cuda(), st, cache, table, le)
    assert tq.device_faults() == 32
    host = [x.copy() for x in s.cache]
    for b in served:
        int8.append(*host, wide(s.K), wide(s.V), starts[b:b + 2], lengths[b:b + 1], s.table[b:b + 1])
    for got, want in zip(t, host):
        assert np.array_equal(got.cpu().numpy(), want)
    out = tuple(torch.full((s.n, s.H, s.D), 7.0, dtype=s.dtype, device="cuda") for _ in range(2))
    tq.read_int8(cache, table, st, le, s.n, s.dtype, out=out)
    assert tq.device_faults() == 32
    hit = np.zeros((s.n, s.H, s.D), bool)
    for b in served:                                  # a token of two sequences has one's value or the other's
        rows, slot = slice(starts[b], starts[b + 1]), lengths[b] + np.arange(starts[b + 1] - starts[b])
        want = [int8.values(host[of], host[2], of, s.table[b, slot // s.page], slot % s.page) for of in range(2)]
        hit[rows] |= (wide(out[0])[rows] == want[0]) & (wide(out[1])[rows] == want[1])
    for b in served:
        assert hit[starts[b]:starts[b + 1]].all()
    other = np.ones(s.n, bool)
    for b in served:
        other[starts[b]:starts[b + 1]] = False
    assert all((wide(x)[other] == 7.0).all() for x in out)


LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("counts,at,value", [([5, 6, 7, 8], 2, -1000000), ([5, 6, 7, 8], 1, HIGH), ([5, 6, 7, 8], 3, LOW), ([5, 6, 7, 8], 0, -1),
                                             ([5, 6, 7, 8], 0, HIGH), ([40, 1, 0, 17, 33], 4, LOW), ([40, 1, 0, 17, 33], 3, LOW),
                                             ([40, 1, 0, 17, 33], 3, 1000), ([40, 1, 0, 17, 33], 5, -1)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_start_out_of_range(tq, counts, at, value, dtype):
    s = Setup(counts, [3, 10, 0, 20, 31][:len(counts)], 2, 64, 16, dtype, seed=at, padding=40)
    starts = s.starts.copy()
    starts[at] = value
    check_rows(tq, s, starts, s.lengths, runs(starts, s.lengths, s.n))


@pytest.mark.parametrize("at", [0, 1, 31, 32, 33, 50, 64, 99, 100])
@pytest.mark.parametrize("value", [LOW, -1, HIGH, 10 ** 6])
def test_a_start_out_of_range_among_many(tq, at, value):
    s = Setup([1 + 5 * i % 23 for i in range(100)], [7 * i % 40 for i in range(100)], 1, 64, 16, BF16, seed=at)
    starts = s.starts.copy()
    starts[at] = value
    check_rows(tq, s, starts, s.lengths, runs(starts, s.lengths, s.n))


def test_several_bad_numbers(tq):
    s = Setup([9] * 70, [5 * i % 33 for i in range(70)], 2, 128, 32, BF16, seed=3)
    starts, lengths = s.starts.copy(), s.lengths.copy()
    starts[[5, 20, 21, 64]], lengths[[0, 40, 69]] = [HIGH, LOW, 10 ** 6, -7], [-1, LOW, -5]
    check_rows(tq, s, starts, lengths, runs(starts, lengths, s.n))


def test_a_start_that_descends(tq):
    """[0, 100), nothing, [50, 150): two sequences may have tokens in common, as long as they write to pages of their own."""
    s = Setup([100, 0, 100], [0, 0, 0], 2, 128, 16, BF16, seed=8)
    starts = np.array([0, 100, 50, 150], np.int32)
    check_rows(tq, s, starts, s.lengths, [0, 2])

