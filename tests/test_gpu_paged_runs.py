"""GPU parity of the paged decode where a warp's run is long: many tiles of one unit, and many
units one after another.  Sizes follow the device: the split cuts the line of all units'
tiles (32 slots) into 12 runs an SM.

Tolerances are those of test_gpu_paged.py."""
import numpy as np
import pytest

import oracle
from oracle import paged
from test_gpu_paged import D, Pages, check_mass, check_out, dev, run_decode, tq  # noqa: F401  (tq: the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TILE = 32


def runs():
    return 12 * min(192, torch.cuda.get_device_properties(0).multi_processor_count)


def tiles_of(lengths):
    return sum(-(-int(n) // TILE) for n in lengths)


KINDS = {"f32": (False, False, 5), "f32_mass": (False, True, 4), "bf16": (True, False, 9), "mass4": (True, True, 3),
         "mass8": (True, True, 8)}


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("kind", KINDS)
def test_runs_of_several_units(tq, kind, many, page):
    """Every warp goes through several units, most of them shorter than its ring of stages, some
    sequences empty; up to 32 sequences and more.  The same call gives the same bits."""
    bf16, mass, G = KINDS[kind]
    rng = np.random.default_rng(page + many)
    B = 300 if many else 32
    lengths = rng.integers(0, 130, B)
    lengths[rng.random(B) < 0.1] = 0
    lengths[B // 2], lengths[-1] = 129, 0
    H = -(-5 * runs() // tiles_of(lengths))
    p = Pages(tq, B, H, 130, page, 3, 3 if many else 2, rot=1, seed=B + page, lengths=lengths)
    assert tiles_of(lengths) * H >= 5 * runs() and B * H > 2 * runs()
    a, ma = run_decode(tq, p, G, bf16, mass)
    b, mb = run_decode(tq, p, G, bf16, mass)
    assert torch.equal(a, b) and (not mass or torch.equal(ma, mb))


def chunked(p, Q, scale, ke, ve, chunk=1 << 15):
    """`paged.decode_paged` of one sequence and one head, by chunks of slots in 64 bits."""
    n, Pk, Pv = int(p.lengths[0]), p.Pk[0].astype(np.float64), p.Pv[0].astype(np.float64)
    a = Q[0].astype(np.float64) @ Pk.T
    kc, vc = p.kc.astype(np.float64), p.vc.astype(np.float64)
    pg, r = paged.slot_rows(p.table, 0, n, p.page)
    s, t = np.empty((len(a), n)), np.zeros((len(a), 1))
    for i in range(0, n, chunk):
        at = pg[i:i + chunk], 0, r[i:i + chunk]
        c, nk = kc[oracle.unpack_indices(p.kp[at], p.kb, D)], p.kn[at].astype(np.float64)
        s[:, i:i + chunk] = scale * (a @ c.T) * nk
        t = np.maximum(t, (abs(scale) * nk * (np.abs(a) @ np.abs(c).T)).max(1, keepdims=True))
    w = np.exp(s - s.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    acc, big = np.zeros((len(a), D)), np.zeros((len(a), D))
    for i in range(0, n, chunk):
        at = pg[i:i + chunk], 0, r[i:i + chunk]
        c = vc[oracle.unpack_indices(p.vp[at], p.vb, D)]
        x = w[:, i:i + chunk] * p.vn[at].astype(np.float64)
        acc += x @ c
        big += x @ np.abs(c)
    grow = np.expm1(2 * t * (2 * ke + ke ** 2))
    return (acc @ Pv)[None], w[None, None], ((grow + 2 * ve + ve ** 2) * (big @ np.abs(Pv)))[None], grow.T[None]


@pytest.mark.parametrize("page", [16, 256])
@pytest.mark.parametrize("kind", ["f32", "f32_mass", "bf16", "mass4", "mass8"])
def test_long_runs_rise(tq, kind, page):
    """Ten tiles a warp and more, in which logits (up to 7 a tile, for some queries downwards)
    and values' lengths rise, so that sums and scales are taken along from tile to tile."""
    bf16, mass, _ = KINDS[kind]
    G = 8 if kind == "mass8" else 4
    n = TILE * runs() * 10 + 45
    p = Pages(tq, 1, 1, n, page, 3, 3, seed=7)
    rng = np.random.default_rng(8)
    tile = np.arange(n) // TILE
    at = p.table[0, np.arange(n) // page], 0, np.arange(n) % page
    p.kp[at] = p.kp[0, 0, 0]                                   # one direction: the lengths make the logits
    p.kn[at] = (2.0 + tile % 9 + 0.3 * rng.random(n)).astype(np.float16)
    p.vn[at] = (rng.uniform(0.5, 1, n) * 2.0 ** (tile % 7 - 3)).astype(np.float16)
    p.upload(tq)
    c = p.kc.astype(np.float64)[oracle.unpack_indices(p.kp[0, 0, 0][None], 3, D)[0]] @ p.Pk[0]
    Q = np.stack([x * c / (c @ c) for x in (7.0, 6.0, -4.0, 0.01, 1.0, -7.0, 3.0, 6.5)[:G]])[None].astype(np.float32)
    q = dev(Q).bfloat16() if bf16 else dev(Q)
    qf = q.float().cpu().numpy()
    S = p.table.shape[1] * page
    m = torch.ones(1, 1, S, device="cuda") if mass else None
    got = tq.decode_paged(q, p.cache, p.t, p.n, mass=m, scale=1.0)
    ke = 2.0 ** -18 if (mass or not bf16) else 2.0 ** -11 + 2.0 ** -18
    want, w, bound, _ = chunked(p, qf, 1.0, ke, 2.0 ** -11 if bf16 else 2.0 ** -18)
    # values of lengths up to 8: the sums' share of the tolerance goes by the largest
    err = np.abs(got.double().cpu().numpy() - want)
    tol = bound + 8e-5 + 1e-5 * np.abs(want) + (2.0 ** -8 * np.abs(want) if bf16 else 0)
    assert (err <= tol).all(), np.max(err / tol)
    if mass:
        check_mass(m[..., :n], np.ones((1, 1, n)), w, chunked(p, qf, 1.0, 2.0 ** -18, 2.0 ** -18)[3])
        assert (m[..., n:] == 1).all()
    again = tq.decode_paged(q, p.cache, p.t, p.n, scale=1.0, mass=None if m is None else torch.ones_like(m))
    assert torch.equal(got, again)
