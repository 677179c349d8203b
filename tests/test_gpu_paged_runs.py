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


@pytest.mark.parametrize("kind,S", [(k, 1 << 17) for k in KINDS] + [("f32", 1 << 20), ("bf16", 1 << 20)])   # with mass, 2^20 slots of logits take 8 GB
@pytest.mark.parametrize("values", ["one", "some"])
def test_sums_of_long_runs(tq, kind, values, S):
    """Hundreds and thousands of tiles a warp with equal or nearly equal weights, over values
    that are all the same row or 256 rows in turn: the errors of a sum's additions all point one
    way.  Every slot of a sequence lies on one page, so the result is that of 256 slots."""
    bf16, mass, _ = KINDS[kind]
    G, B, H, page = 8 if kind == "mass8" else 4, 16 if mass else 64, 8, 256
    p = Pages(tq, B, H, page, page, 3, 3, rot=1, seed=17)
    p.kn[:] = 0.0 if values == "one" else 0.01
    p.vn[:] = 1.0
    if values == "one":
        p.vp[:] = p.vp[:, :, :1]
    p.upload(tq)
    Q = np.random.default_rng(18).standard_normal((B, H * G, D)).astype(np.float32)
    q = dev(Q).bfloat16() if bf16 else dev(Q)
    ke = 2.0 ** -18 if (mass or not bf16) else 2.0 ** -11 + 2.0 ** -18
    want, w, bound, wrel = p.want(q.float().cpu().numpy(), None, ke, 2.0 ** -11 if bf16 else 2.0 ** -18)
    t = dev(np.repeat(p.table, S // page, axis=1))
    n = torch.full((B,), S, dtype=torch.int32, device="cuda")
    assert B * H * S // TILE > 200 * runs()
    m = torch.zeros(B, H, S, device="cuda") if mass else None
    out = tq.decode_paged(q, p.cache, t, n, mass=m)
    check_out(out, want, bound, bf16)
    if mass:
        check_mass(m.view(B, H, S // page, page)[:, :, ::37].reshape(B, H, -1), np.zeros(1),
                   np.tile(w / (S // page), len(range(0, S // page, 37))), wrel)


@pytest.mark.parametrize("kind", ["f32", "f32_mass", "bf16", "mass4", "mass8"])
def test_long_runs_of_rising_and_falling_pages(tq, kind):
    """600 tiles a warp and more of 40 pages in changing order: logits that rise and fall by up
    to 60 over a run, values whose lengths do.  A page that occurs k times counts k times."""
    bf16, mass, _ = KINDS[kind]
    G, B, page, U = 8 if kind == "mass8" else 4, 4, 256, 40
    rng = np.random.default_rng(41)
    p = Pages(tq, 1, 1, U * page, page, 3, 3, seed=42, spare=0)
    p.kp[:] = p.kp[0, 0, 0]                                    # one direction: the lengths make the logits
    level = rng.permutation(U)
    p.kn[:] = (1.0 + 0.2 * level[:, None, None] + 0.3 * rng.random(p.kn.shape)).astype(np.float16)
    p.vn[:] = (rng.uniform(0.5, 1, p.vn.shape) * 2.0 ** rng.integers(-3, 4, (U, 1, 1))).astype(np.float16)
    p.upload(tq)
    M = -(-600 * TILE * runs() // (B * page)) + 1
    byl = np.argsort(level)
    i = np.arange(B * M).reshape(B, M)
    table = byl[np.where((i // 200) % 2, (i // 5) % U, U - 1 - (i // 7) % U)].astype(np.int32)
    lengths = M * page - np.array([0, 1, 77, 255])
    assert sum(-(-lengths // TILE)) >= 600 * runs()
    count = np.zeros((B, U, page))
    for b in range(B):
        np.add.at(count[b], table[b], 1)
        count[b, table[b, -1], page - (M * page - lengths[b]):] -= 1
    c = p.kc.astype(np.float64)[oracle.unpack_indices(p.kp[0, 0, 0][None], 3, D)[0]]
    k = c @ p.Pk[0]
    Q = np.stack([x * k / (c @ c) for x in (6.0, -6.0, 0.01, 1.0, -1.0, 3.0, -2.0, 5.0)[:G]])[None].repeat(B, 0).astype(np.float32)
    q = dev(Q).bfloat16() if bf16 else dev(Q)
    qf = q.float().cpu().numpy().astype(np.float64)
    m = torch.zeros(B, 1, M * page, device="cuda") if mass else None
    got = tq.decode_paged(q, p.cache, dev(table), dev(lengths.astype(np.int32)), mass=m, scale=1.0).double().cpu().numpy()
    ke, ve = 2.0 ** -18 if (mass or not bf16) else 2.0 ** -11 + 2.0 ** -18, 2.0 ** -11 if bf16 else 2.0 ** -18
    Pv = p.Pv[0].astype(np.float64)
    cv = p.vc.astype(np.float64)[oracle.unpack_indices(p.vp.reshape(-1, 48), 3, D)]
    nk, nv = p.kn.reshape(-1).astype(np.float64), p.vn.reshape(-1).astype(np.float64)
    for b in range(B):
        a = qf[b] @ p.Pk[0].astype(np.float64).T
        s = (a @ c)[:, None] * nk
        e = np.exp(s - s.max(1, keepdims=True))
        w = e / (e * count[b].reshape(-1)).sum(1, keepdims=True)        # of one slot
        x = w * count[b].reshape(-1) * nv
        want = (x @ cv) @ Pv
        t = (nk.max() * (np.abs(a) @ np.abs(c)))[:, None]
        grow = np.expm1(2 * t * (2 * ke + ke ** 2))
        bound = (grow + 2 * ve + ve ** 2) * ((x @ np.abs(cv)) @ np.abs(Pv))
        tol = bound + 8e-5 + 1e-5 * np.abs(want) + (2.0 ** -8 * np.abs(want) if bf16 else 0)
        err = np.abs(got[b] - want)
        assert (err <= tol).all(), np.max(err / tol)
        if mass:
            at = np.r_[0:M - 1:97]
            wrel = np.expm1(2 * t[:, 0] * (2 * 2.0 ** -18 + 2.0 ** -36))
            ww = w.reshape(G, U, page)[:, table[b, at]].reshape(1, 1, G, -1)
            check_mass(m[b, 0].view(M, page)[dev(at)].view(1, 1, -1), np.zeros(1), ww, wrel[None, None])
            assert not m[b, 0, lengths[b]:].any()
