"""attend_int8 for pieces of prompts where units of up to 128 columns (one half of a block's columns) and larger ones follow each
other: the half without columns has to keep up with the block's other warps.  Against the definition in 64 bits, computed
sequence by sequence on the device; bounds as in test_gpu_int8.py."""
import numpy as np
import pytest

from oracle import int8
from test_gpu_int8 import BF16, HALF, Setup, bounds, dev, tq, wide  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def attend(Q, kc, vc, ex, starts, lengths, table, scale, window, sinks, logit_eps, value_eps, least):
    """oracle.int8.attend, a head of a sequence at a time; every page present."""
    n, Hq, D = Q.shape
    H, page = kc.shape[1:3]
    G = Hq // H
    out, bound = (torch.full((n, Hq, D), float("nan"), dtype=torch.float64, device="cuda") for _ in range(2))
    for b in range(len(lengths)):
        first, count, end = int(starts[b]), int(starts[b + 1] - starts[b]), int(lengths[b] + starts[b + 1] - starts[b])
        if count == 0:
            continue
        s = torch.arange(end, device="cuda")
        pg = table[b].long()[s // page]
        at = torch.arange(end - count, end, device="cuda").view(-1, 1, 1)
        seen = s <= at
        if window:
            seen &= (s > at - window) | (s < sinks)
        for h in range(H):
            e = ex[pg, h, s % page // 16].double()
            k, v = ((x[pg, h, s % page].double() - 127.5) * torch.exp2(e[:, i, None]) for i, x in enumerate((kc, vc)))
            q = Q[first:first + count, h * G:(h + 1) * G].double()
            z = (scale * (q @ k.T)).masked_fill(~seen, -float("inf"))
            p = torch.softmax(z, -1)
            t = logit_eps * abs(scale) * (q.abs() @ k.abs().T).masked_fill(~seen, 0).amax(-1, keepdim=True)
            out[first:first + count, h * G:(h + 1) * G] = p @ v
            bound[first:first + count, h * G:(h + 1) * G] = ((torch.expm1(2 * t) + value_eps) * (p @ v.abs())
                                                            + least * seen.sum(-1, keepdim=True) * 128 * (p * torch.exp2(e[:, 1])).amax(-1, keepdim=True))
    return out, bound


@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3)])
def test_the_definition_by_sequence(tq, window, sinks):
    s = Setup([5, 0, 40], [33, 7, 90], 2, 64, 16, BF16, seed=1)
    s.append()
    Q = s.queries(3)
    want = int8.attend(wide(Q), *s.cache, s.starts, s.lengths, s.table, 0.125, window, sinks, *bounds(BF16))
    got = attend(Q.cuda(), *(dev(x) for x in s.cache), s.starts, s.lengths, dev(s.table), 0.125, window, sinks, *bounds(BF16))
    for g, w in zip(got, want):
        assert np.allclose(wide(g), w, rtol=1e-12, atol=1e-14)


RAGGED = np.random.default_rng(5).integers(1, 51, 64).tolist()


@pytest.mark.parametrize("counts,before,H,G,D,page,window,sinks", [
    ([52, 67] * 80, [1300, 1100] * 80, 8, 2, 128, 64, 300, 0),        # one half, two halves in turn
    ([52, 67] * 80, [1300, 1100] * 80, 8, 2, 64, 32, 300, 5),
    ([40, 40, 40, 40, 40, 200] * 10, [0] * 60, 16, 1, 128, 16, 0, 0),  # fresh prompts: a tile or two a unit
    ([40] * 50 + [200] * 10, [0] * 60, 32, 1, 64, 16, 0, 0),
    ([40, 40, 40, 40, 40, 200] * 10, [2000, 3000, 5000, 2500, 0, 1500] * 10, 8, 1, 128, 64, 1200, 4),
    (RAGGED, [12000] * 64, 8, 4, 128, 256, 4096, 4),
    ([1056, 1056], [20000, 20000], 8, 4, 128, 256, 9000, 0),          # the last of a head's units has 128 columns
    ([90] * 16, [8192] * 16, 8, 3, 128, 64, 0, 0),
])
def test_units_of_one_half_and_of_two(tq, counts, before, H, G, D, page, window, sinks):
    g = torch.Generator(device="cuda").manual_seed(len(counts) + D)
    used = [-(-(c + n) // page) for c, n in zip(counts, before)]
    N = sum(used) + 3
    order = torch.randperm(N, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(counts), max(used)), -1, dtype=torch.int32, device="cuda")
    for b, (u, z) in enumerate(zip(used, np.cumsum(used))):
        table[b, :u] = order[z - u:z]
    kc, vc = (torch.randint(0, 256, (N, H, page, D), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2))
    ex = torch.randint(-8, -4, (N, H, page // 16, 2), generator=g, device="cuda", dtype=torch.int8)
    cache = tq.Int8Cache(kc, vc, ex)
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    n = int(starts[-1])
    assert n * G > 32 * len(counts)                                   # the form for prompts
    Q = torch.randn(n, H * G, D, generator=g, device="cuda").to(BF16)
    a = Q, dev(starts), cache, table, dev(np.array(before, np.int32))
    got = tq.attend_int8(*a, window=window or None, sinks=sinks)
    again = [tq.attend_int8(*a, window=window or None, sinks=sinks) for _ in range(5)]
    assert all(torch.equal(x, got) for x in again) and tq.device_faults() == 0
    want, bound = attend(Q, kc, vc, ex, starts, before, table, D ** -0.5, window, sinks, *bounds(BF16))
    err, allowed = (got.double() - want).abs(), bound + HALF[BF16] * want.abs() + 1e-30
    assert (err <= allowed).all(), (float((err / allowed).max()), (err > allowed).sum())
