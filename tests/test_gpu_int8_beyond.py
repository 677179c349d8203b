"""attend_int8 for tokens whose slots lie beyond the page table: what is there of their window and of the first slots is seen.
Bounds and definitions as in test_gpu_int8.py."""
import pytest

from test_gpu_int8 import BF16, F32, Setup, check_attend, tq  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,sinks", [(8, 44), (8, 48), (1, 33), (5, 32), (8, 3), (8, 0), (30, 40), (8, 2 ** 31 - 1)])
@pytest.mark.parametrize("count,dtype", [(2, BF16), (2, F32), (40, BF16), (40, F32)])
def test_first_slots_of_tokens_beyond_the_table(tq, window, sinks, count, dtype):
    """48 slots are there; the tokens' slots lie behind them, the window's with them or across the end."""
    for before in (60, 49, 30):
        s = Setup([count, 3], [48 - count, 20], 2, 128, 16, dtype, seed=count)
        s.append()
        assert s.table.shape[1] == 3 and (s.table[0] >= 0).all()
        s.lengths[0] = before
        check_attend(tq, s, 1, window=window, sinks=sinks, faults=32 if before + count > 48 else 0)
