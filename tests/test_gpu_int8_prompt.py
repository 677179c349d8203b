"""attend_int8 for pieces of prompts: more than 32 columns a sequence, which take the tcgen05 form with bf16 queries and the
warp-wide form in blocks of 32 columns with fp32 ones.  Bounds as in test_gpu_int8.py."""
import numpy as np
import pytest

from test_gpu_int8 import BF16, F32, HALF, Setup, bounds, check_attend, dev, tq, wide  # noqa: F401
from oracle import int8

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,before,G", [([64], [0], 1), ([128], [0], 1), ([33], [95], 4), ([64], [64], 4), ([65], [300], 4), ([257], [3], 1),
                                             ([100], [1000], 3), ([40, 1, 90, 0, 33], [5, 700, 0, 9, 250], 4), ([300], [0], 7), ([17], [2000], 8)])
@pytest.mark.parametrize("D,page", [(128, 16), (64, 256), (128, 64)])
def test_prompt(tq, counts, before, G, D, page):
    s = Setup(counts, before, 2, D, page, BF16, seed=sum(counts) + D, padding=3)
    s.append()
    check_attend(tq, s, G)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 2), (37, 0), (100, 33), (128, 16), (5, 2 ** 31 - 1), (2 ** 31 - 1, 3), (300, 200)])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_window(tq, window, sinks, D):
    s = Setup([150, 60], [90, 700], 1, D, 32, BF16, seed=window % 97)
    s.append()
    check_attend(tq, s, 3, window=window, sinks=sinks)


@pytest.mark.parametrize("H,T,before", [(1, 40, 6000), (3, 33, 3000)])
def test_prompt_split_over_the_length(tq, H, T, before):
    """Few columns over many slots: every block of the device has a part of the length."""
    s = Setup([T], [before], H, 128, 64, BF16, seed=T)
    s.append()
    check_attend(tq, s, 1)


def test_prompt_many_units(tq):
    """More units than blocks: each block goes through several, of all lengths."""
    s = Setup([37] * 60, [(97 * i) % 400 for i in range(60)], 4, 64, 16, BF16, seed=3)
    s.append()
    check_attend(tq, s, 2)


def test_prompt_of_one_slot_each(tq):
    """Units of a single tile: the infos of several are alive at once."""
    s = Setup([40] * 40, [0] * 40, 4, 128, 64, BF16, seed=4)
    s.append()
    check_attend(tq, s, 1)


def test_prompt_absent_pages(tq):
    s = Setup([40, 50], [100, 20], 2, 128, 16, BF16)
    s.append()
    s.table[0, 2], s.table[1, :] = -5, s.cache[0].shape[0]
    got = check_attend(tq, s, 4, faults=32)
    assert not got[40:].any() and got[:40].any()


@pytest.mark.parametrize("shift", [-50, 60, -115, 115])
def test_prompt_values_far_apart(tq, shift):
    s = Setup([40], [300], 2, 128, 16, BF16, spread=0)
    s.append()
    up = np.arange(s.cache[2].shape[0]) % 3 == 0
    s.cache[2][up, :, :, 1] = np.clip(s.cache[2][up, :, :, 1].astype(int) + shift, -120, 121)
    check_attend(tq, s, 4, size=20.0)


def test_prompt_scale_and_nan_queries(tq):
    s = Setup([60, 50], [40, 170], 2, 128, 32, BF16)
    s.append()
    for scale in (0.0, -0.3, 1.5):
        check_attend(tq, s, 2, scale=scale)
    Q = s.queries(2)
    good = check_attend(tq, s, 2, Q=Q)
    Q[1, 3, 5], Q[70, 0, 2], Q[2, 1] = float("nan"), float("inf"), 0.0
    cache, _, table, starts, lengths = s.device(tq)
    out = wide(tq.attend_int8(Q.cuda(), starts, cache, table, lengths))
    hit = np.zeros(out.shape[:2], bool)
    hit[1, 3] = hit[70, 0] = True
    assert np.isnan(out[hit]).all()
    hit[2, 1] = True
    assert np.array_equal(out[~hit], good[~hit])


def test_prompt_repeats_and_in_a_graph(tq):
    s = Setup([90, 33], [600, 70], 2, 128, 64, BF16, seed=9)
    s.append()
    cache, _, table, starts, lengths = s.device(tq)
    Q = s.queries(4).cuda()
    ws = torch.empty(tq.attend_int8_workspace_bytes(s.n, 2, 2, 4, 128), dtype=torch.uint8, device="cuda")
    first = tq.attend_int8(Q, starts, cache, table, lengths, workspace=ws)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        out = tq.attend_int8(Q, starts, cache, table, lengths, workspace=ws)
    for _ in range(3):
        ws.random_(0, 256)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)


@pytest.mark.parametrize("counts,before,G", [([33], [95], 4), ([100], [200], 3), ([40, 1, 90], [5, 300, 0], 4)])
def test_prompt_f32(tq, counts, before, G):
    s = Setup(counts, before, 2, 128, 32, F32, seed=sum(counts), padding=1)
    s.append()
    check_attend(tq, s, G)
    check_attend(tq, s, G, window=50, sinks=3)
