"""GPU parity of the paged cache's append where a CTA has whole rotations and several tiles: sizes
follow the device (a tile is 128 rows of one KV head's keys or values; with few of them a CTA takes
a quarter of the rotation).  Tolerances are those of test_gpu_paged.py."""
import numpy as np
import pytest

from test_gpu_paged import D, Pages, check_append, dev, tq  # noqa: F401  (tq: the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def some_rows(rng, n, B, S):
    """n (sequence, slot, position) of different slots, one in ten to be skipped."""
    at = rng.permutation(B * S)[:n]
    rows = np.stack([at // S, at % S, rng.integers(0, 10 ** 6, n)], 1).astype(np.int32)
    skip = np.flatnonzero(rng.random(n) < 0.1)
    rows[skip, rng.integers(0, 2, skip.size)] = -1
    return rows


def some_vectors(rng, n, H):
    x = rng.standard_normal((n, H, D)) * np.exp(2 * rng.standard_normal((n, H, 1)))
    x[..., [3, 17]] *= 15
    x[rng.random((n, H)) < 0.01] = 0
    return x.astype(np.float32)


@pytest.mark.parametrize("kb,vb", [(2, 4), (3, 3), (4, 2)])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("size", ["one", "some", "many"])
def test_append_whole_rotations(tq, size, bf16, kb, vb):
    """One tile a CTA; up to two; six and more, in runs that go on from keys to values and from
    head to head.  Odd tails, skipped and zero rows, heads that share rotations."""
    H = 5
    tiles = {"one": sms() // (2 * H) - 1, "some": 15 * sms() // (20 * H), "many": -(-6 * sms() // (2 * H)) + 1}[size]
    n = 128 * (tiles - 1) + 77
    items = tiles * H * 2
    assert 4 * items > sms() and {"one": items <= sms(), "some": sms() < items < 2 * sms(), "many": items > 6 * sms()}[size]
    rng = np.random.default_rng(n + kb)
    B, S = 3, -(-n // 2)
    p = Pages(tq, B, H, S, 64, kb, vb, rot=2, seed=n + vb)
    rows, K, V = some_rows(rng, n, B, S), some_vectors(rng, n, H), some_vectors(rng, n, H)
    k, v = (dev(x).bfloat16() if bf16 else dev(x) for x in (K, V))
    before = p.host()
    mass, pos = rng.random((B, H, S)).astype(np.float32), np.full((B, H, S), -5, np.int32)
    m, q = dev(mass), dev(pos)
    tq.append_paged(k, v, dev(rows), p.cache, p.t, mass=m, positions=q)
    torch.cuda.synchronize()
    check_append(p, before, k.double().cpu().numpy(), v.double().cpu().numpy(), rows)
    for b, s, at in rows:
        if b >= 0 and s >= 0:
            mass[b, :, s], pos[b, :, s] = 0.0, at
    assert np.array_equal(m.cpu().numpy(), mass) and np.array_equal(q.cpu().numpy(), pos)
    # once more to the same places: the same bits
    once = p.host()
    tq.append_paged(k, v, dev(rows), p.cache, p.t)
    assert all(np.array_equal(x.view(np.uint8), y.view(np.uint8)) for x, y in zip(once, p.host()))
    assert tq.device_faults() == 0
