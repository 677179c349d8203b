"""GPU parity of the paged cache's operators where their order or their arithmetic is decided by
little: windows of protected tokens longer than the budget, coordinates next to a midpoint.
Tolerances are those of test_gpu_paged.py."""
import numpy as np
import pytest

from conftest import codebook
from test_gpu_paged import D, Pages, check_append, dev, run_evict, some_positions, tq  # noqa: F401  (tq: the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


# ---- evict: more protected slots than are kept --------------------------------

def test_evict_window_by_hand(tq):
    """32 tokens in order, the newest 8 protected, room for 4: the heaviest of the 8."""
    p = Pages(tq, 1, 1, 32, 16, seed=1)
    mass = np.full((1, 1, 32), 9.0, np.float32)
    mass[0, 0, 24:] = [1, 2, 5, 6, 4, 2, 3, 0]
    pos = np.arange(32, dtype=np.int32).reshape(1, 1, 32)
    _, got = tq.evict_paged(p.cache, p.t, p.n, p.n, dev(mass), dev(pos), 4, 8)
    assert got[0, 0, :4].tolist() == [26, 27, 28, 30]


@pytest.mark.parametrize("S,budget,recent", [(40, 1, 40), (600, 100, 101), (600, 100, 99), (600, 100, 100), (600, 599, 600), (5000, 700, 3000),
                                             (70001, 300, 5000), (393300, 1000, 200000)])
def test_evict_windows(tq, S, budget, recent):
    """Windows as long as the budget, shorter and longer by one, and much longer; one CTA,
    clusters, keys in device memory; weights all different and in ties."""
    rng = np.random.default_rng(S + recent)
    B, lengths = (3, [S, S - 7, S // 2]) if S < 10000 else (1, [S])
    p = Pages(tq, B, 2 if B > 1 else 1, S, 16 if S < 10000 else 256, 2, 2, rot=1, seed=3, lengths=lengths)
    pos = some_positions(rng, B, p.H, S, lengths)
    for mass in (np.exp(2 * rng.standard_normal(pos.shape)), rng.integers(0, 3, pos.shape), -rng.random(pos.shape)):
        run_evict(tq, p, mass.astype(np.float32), pos, np.asarray(lengths, np.int32) + 5, budget, recent)


# ---- append: coordinates next to midpoints ------------------------------------

def append_and_check(tq, p, K, V, bf16):
    n = len(K)
    k, v = (dev(x.astype(np.float32)).bfloat16() if bf16 else dev(x.astype(np.float32)) for x in (K, V))
    rows = np.stack([np.zeros(n), np.arange(n), np.arange(n)], 1).astype(np.int32)
    before = p.host()
    tq.append_paged(k, v, dev(rows), p.cache, p.t)
    check_append(p, before, k.double().cpu().numpy(), v.double().cpu().numpy(), rows)


def with_coordinate(rng, Pi, d, y):
    """Vectors [n,128] of any length whose unit vectors' coordinate d[i] along Pi is y[i]."""
    P = Pi.astype(np.float64)[d]
    x = rng.standard_normal(P.shape)
    x -= (x * P).sum(1, keepdims=True) * P
    x *= np.sqrt(1 - y * y)[:, None] / np.linalg.norm(x, axis=1, keepdims=True)
    return (x + y[:, None] * P) * np.exp(rng.standard_normal((len(d), 1)))


@pytest.mark.parametrize("n", [128, 6000])
@pytest.mark.parametrize("bits", [2, 3, 4])
def test_append_at_the_bounds_of_the_second_sums(tq, n, bits):
    """Coordinates at the distances from a midpoint where a code is taken from the first product,
    from its second sum or from the pairs (5e-6, 2^-19), a few ulp to either side, and on it."""
    rng = np.random.default_rng(n + bits)
    p = Pages(tq, 1, 1, n, 256, bits, bits, seed=bits)
    out = []
    for Pi, cb in ((p.Pk, p.kc), (p.Pv, p.vc)):
        mid = 0.5 * (cb[1:].astype(np.float64) + cb[:-1])
        off = np.array([0.0, 1e-9, 2.0 ** -19, 2.0 ** -19 + 4e-9, 2.0 ** -19 - 4e-9, 2.0 ** -19 + 1e-8, 5e-6, 5e-6 + 4e-9, 5e-6 - 4e-9, 6e-6])
        y = rng.choice(mid, n) + rng.choice(off, n) * rng.choice((-1.0, 1.0), n)
        out.append(with_coordinate(rng, Pi[0], rng.integers(0, D, n), y)[:, None])
    append_and_check(tq, p, out[0], out[1], False)


@pytest.mark.parametrize("w", [1e-6, 2e-6, 3.4e-6, 5e-6, 9e-6, 1.1e-5, 4e-5])
@pytest.mark.parametrize("n", [128, 6000])
def test_append_midpoints_two_cells_apart(tq, n, w):
    """Three midpoints at m, m + 2w and m + 124w, so that cells are w wide and the first two as
    near one another as the cells allow; coordinates between and about them."""
    rng = np.random.default_rng(n)
    p = Pages(tq, 1, 1, n, 256, 2, 2, seed=5)
    out = []
    for name, Pi, m in (("kc", p.Pk, 0.05), ("vc", p.Pv, -0.031)):
        c = np.array([m - w, m + w, m + 3 * w, m + 245 * w]).astype(np.float32)
        setattr(p, name, c)
        mid = 0.5 * (c[1:].astype(np.float64) + c[:-1])
        y = rng.choice(mid, n) + rng.choice([0.5, 0.7, 1.0, 1.3, 1.5, 1e-3, 0.0], n) * w * rng.choice((-1.0, 1.0), n)
        out.append(with_coordinate(rng, Pi[0], rng.integers(0, D, n), y)[:, None])
    p.upload(tq)
    append_and_check(tq, p, out[0], out[1], False)


@pytest.mark.parametrize("n", [128, 6000])
@pytest.mark.parametrize("bf16", [False, True])
def test_append_rows_along_the_rotation(tq, n, bf16):
    """Rows that are sums of one, two or five rows of the rotation: all products of a coordinate
    point one way, so that the tensor core's errors do.  Midpoints 1e-8 to 2e-5 about it."""
    rng = np.random.default_rng(n)
    p = Pages(tq, 1, 1, n, 256, 4, 4, seed=6)
    for m in (1, 2, 5):
        off = np.logspace(-8, -4.7, 4)
        c = np.sort(np.concatenate([m ** -0.5 + s * off + e for s in (-1, 1) for e in (-2e-9, 2e-9)])).astype(np.float32)
        p.kc = p.vc = c
        p.upload(tq)
        out = []
        for Pi in (p.Pk[0], p.Pv[0]):
            d, sign = np.stack([rng.permutation(D)[:m] for _ in range(n)]), rng.choice((-1.0, 1.0), (n, m))
            sign[:, 0] = 1
            x = (Pi.astype(np.float64)[d] * sign[..., None]).sum(1) * np.exp(rng.standard_normal((n, 1)))
            out.append((x * (1 + 1e-6 * rng.standard_normal(x.shape)))[:, None])
        append_and_check(tq, p, out[0], out[1], bf16)


# ---- append: lengths ----------------------------------------------------------

def lengths_of(tq, K):
    n = K.shape[0]
    p = Pages(tq, 1, 1, n, 256, 3, 3, seed=8)
    rows = np.stack([np.zeros(n), np.arange(n), np.arange(n)], 1).astype(np.int32)
    tq.append_paged(K, K, dev(rows), p.cache, p.t)
    kn, vn = (x[p.table[0, rows[:, 1] // 256], 0, rows[:, 1] % 256] for x in (p.host()[1], p.host()[3]))
    assert np.array_equal(kn, vn)
    return kn


@pytest.mark.parametrize("bf16", [False, True])
def test_append_lengths_are_the_nearest(tq, bf16):
    """fp16 lengths of random rows of all sizes are those of the 64-bit ones."""
    rng = np.random.default_rng(1)
    K = rng.standard_normal((20000, 1, D)) * np.exp(3 * rng.standard_normal((20000, 1, 1)))
    K[::3, :, 1:] *= 1e-3
    k = dev(K.astype(np.float32)).bfloat16() if bf16 else dev(K.astype(np.float32))
    got = lengths_of(tq, k)
    with np.errstate(over="ignore"):
        want = np.sqrt((k[:, 0].double().cpu().numpy() ** 2).sum(-1)).astype(np.float16)
    assert np.array_equal(got, want), f"{(got != want).sum()} lengths differ"


def test_append_lengths_between_two_steps(tq):
    """Lengths on the middle of two fp16 numbers (to the even one), and 2^-25 of it to either
    side; about the largest number, among the subnormal ones, and about the smallest."""
    steps = np.arange(0x7c00, dtype=np.uint16).view(np.float16).astype(np.float64)
    rng = np.random.default_rng(2)
    i = np.concatenate([rng.integers(0, 0x7bff, 400), np.arange(6), np.arange(0x3fa, 0x405), [0x7bfe, 0x7bff]])
    lo, hi = steps[i], np.append(steps, 65536.0)[i + 1]
    mid = 0.5 * (lo + hi)
    K = np.zeros((3 * i.size, 1, D), np.float32)
    for j, d in enumerate((0, 1, -1)):
        K[j * i.size:(j + 1) * i.size, 0, 70] = np.nextafter(mid.astype(np.float32), np.float32(np.inf * d)) if d else mid
    K[i.size:2 * i.size:2, 0, 70] = mid[::2]                   # above it by another coordinate
    K[i.size:2 * i.size:2, 0, 3] = mid[::2] * 2.0 ** -12
    got = lengths_of(tq, dev(K))
    with np.errstate(over="ignore"):
        want = np.sqrt((K[:, 0].astype(np.float64) ** 2).sum(-1)).astype(np.float16)
    assert np.array_equal(got, want), np.flatnonzero(got != want)
