"""GPU parity of the paged cache's operators (append, decode, evict) with their float64
definitions, at the sizes and orders where they can go wrong.

Tolerances, all derived from the arithmetic:
- cells and fp16 lengths of append: equal; a cell may differ only where the float64
  coordinate lies within 1e-13 of a midpoint (128 products in 64 bits), a length by half a
  step of fp16 plus fp32 summation, that is one step.
- decode: `oracle.paged.decode_paged` turns a relative error per operand into a bound on the
  output.  fp32 queries: 2^-18 per operand covers the 128 fp32 additions of a logit, and the
  ABI's 1e-5 (1 + |out|) is asked for on top.  bf16 queries: operands rounded to fp16 (2^-11,
  beside the 2^-18), half a step of bf16 for the output (2^-8 |out|), 1e-5 (1 + |out|) for
  the fp32 sums.
- mass: the weights' bound with 2^-18 per operand, a factor 1 + 2^-18 for exp and the sum, and
  half a step of fp32 (2^-24) for each of the addition and the product.
"""
import numpy as np
import pytest

import oracle
from oracle import paged
from conftest import codebook

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module")
def tq():
    from compressed_kv_cache_gb300 import build as tqbuild
    tqbuild.build()
    from compressed_kv_cache_gb300 import tq as mod
    assert torch.cuda.is_available()
    mod.device_faults()
    return mod


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def rotations(rng, h):
    return np.stack([oracle.haar_rotation(rng.standard_normal((D, D))) for _ in range(h)]).astype(np.float32)


class Pages:
    """A cache of random rows on the host and the device, with B sequences on scattered pages."""

    def __init__(self, tq, B, H, S, page=16, kb=3, vb=3, rot=None, seed=0, spare=2, lengths=None):
        rng = self.rng = np.random.default_rng(seed)
        self.B, self.H, self.page, self.kb, self.vb = B, H, page, kb, vb
        M = -(-S // page)
        N = B * M + spare
        self.kp = rng.integers(0, 256, (N, H, page, 16 * kb), dtype=np.uint8)
        self.vp = rng.integers(0, 256, (N, H, page, 16 * vb), dtype=np.uint8)
        self.kn = rng.uniform(0.5, 3, (N, H, page)).astype(np.float16)
        self.vn = rng.uniform(0.5, 3, (N, H, page)).astype(np.float16)
        self.Pk, self.Pv = rotations(rng, rot or H), rotations(rng, rot or H)
        self.kc, self.vc = (codebook(D, b)[0].astype(np.float32) for b in (kb, vb))
        self.table = rng.permutation(N)[:B * M].reshape(B, M).astype(np.int32)
        self.lengths = np.asarray([S] * B if lengths is None else lengths, dtype=np.int32)
        for b, n in enumerate(self.lengths):
            self.table[b, -(-int(n) // page):] = -1
        self.upload(tq)

    def upload(self, tq):
        self.cache = tq.PagedCache(*(dev(x) for x in (self.kp, self.kn, self.vp, self.vn, self.Pk, self.kc, self.Pv, self.vc)))
        self.t = dev(self.table)
        self.n = dev(self.lengths)

    def host(self):
        c = self.cache
        return tuple(x.cpu().numpy() for x in (c.k_plane, c.k_norm, c.v_plane, c.v_norm))

    def want(self, Q, scale=None, ke=2.0 ** -18, ve=2.0 ** -18):
        return paged.decode_paged(Q, self.kp, self.kn, self.vp, self.vn, self.table, self.lengths, self.Pk, self.kc,
                                  self.Pv, self.vc, D ** -0.5 if scale is None else scale, ke, ve)


def check_out(got, want, bound, bf16):
    got = got.float().cpu().numpy().astype(np.float64)
    tol = 1e-5 * (1 + np.abs(want))
    if bf16:
        tol = tol + bound + 2.0 ** -8 * np.abs(want)
    err = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), f"{(err > tol).sum()} of {err.size} off, worst {np.max(err / tol):.3g} of the tolerance"


def check_mass(got, before, w, wrel):
    add = (w * (1 + wrel[..., None] + 2.0 ** -18)).sum(2) - w.sum(2)
    want = before + w.sum(2)
    err = np.abs(got.cpu().numpy().astype(np.float64) - want)
    tol = add + 2.0 ** -23 * np.abs(want)
    assert (err <= tol).all(), f"worst {np.max(err / np.maximum(tol, 1e-30)):.3g} of the tolerance"


def run_decode(tq, p, G, bf16=False, mass=False, scale=None, seed=5, big=1.0):
    rng = np.random.default_rng(seed)
    Q = (big * rng.standard_normal((p.B, p.H * G, D))).astype(np.float32)
    q = dev(Q).bfloat16() if bf16 else dev(Q)
    S = int(p.table.shape[1]) * p.page
    before = rng.random((p.B, p.H, S)).astype(np.float32) if mass else None
    m = dev(before) if mass else None
    ws = torch.full((tq.decode_paged_workspace_bytes(p.B, p.H, G, S if mass else 0, mass),), 255, dtype=torch.uint8, device="cuda")
    out = tq.decode_paged(q, p.cache, p.t, p.n, mass=m, scale=scale, workspace=ws)
    torch.cuda.synchronize()
    ke = 2.0 ** -18 if (mass or not bf16) else 2.0 ** -11 + 2.0 ** -18
    want, w, bound, _ = p.want(q.float().cpu().numpy(), scale, ke, 2.0 ** -11 if bf16 else 2.0 ** -18)
    check_out(out, want, bound, bf16)
    if mass:
        wrel = p.want(q.float().cpu().numpy(), scale)[3]
        check_mass(m, before, w, wrel)
    return out, m


# ---- decode -------------------------------------------------------------------

RAGGED = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 255, 300]


@pytest.mark.parametrize("kb", [2, 3, 4])
@pytest.mark.parametrize("vb", [2, 3, 4])
@pytest.mark.parametrize("kind", ["f32", "bf16", "mass", "f32_mass"])
def test_decode_bits(tq, kb, vb, kind):
    p = Pages(tq, 3, 2, 200, 16, kb, vb, seed=10 * kb + vb, lengths=[200, 77, 0])
    run_decode(tq, p, 4, bf16=not kind.startswith("f32"), mass="mass" in kind)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("kind", ["f32", "bf16", "mass"])
def test_decode_lengths_and_pages(tq, page, kind):
    p = Pages(tq, len(RAGGED), 2, 300, page, seed=page, lengths=RAGGED)
    run_decode(tq, p, 2, bf16=kind != "f32", mass=kind == "mass")


@pytest.mark.parametrize("G", [1, 3, 4, 5, 7, 8, 9, 17])
@pytest.mark.parametrize("kind", ["f32", "bf16", "mass"])
def test_decode_groups(tq, G, kind):
    p = Pages(tq, 2, 3, 500, 32, 3, 2, rot=2 if G % 2 else 1, seed=G, lengths=[500, 91])
    run_decode(tq, p, G, bf16=kind != "f32", mass=kind == "mass")


@pytest.mark.parametrize("kind", ["f32", "bf16", "mass"])
def test_decode_long_and_many(tq, kind):
    """One long sequence of an odd length; many short ones; scales other than 1/sqrt(D)."""
    bf16, mass = kind != "f32", kind == "mass"
    run_decode(tq, Pages(tq, 1, 1, 70001, 64, 3, 3, seed=21), 2, bf16, mass)
    run_decode(tq, Pages(tq, 200, 2, 90, 16, 3, 3, rot=1, seed=22, lengths=np.arange(200) % 91), 2, bf16, mass)
    run_decode(tq, Pages(tq, 2, 2, 333, 16, 4, 3, seed=23), 4, bf16, mass, scale=0.02)
    run_decode(tq, Pages(tq, 2, 2, 333, 16, 4, 3, seed=24), 4, bf16, mass, scale=-0.05)
    run_decode(tq, Pages(tq, 2, 2, 333, 16, 4, 3, seed=25), 4, bf16, mass, scale=0.0)


@pytest.mark.parametrize("bf16", [False, True])
def test_decode_peaked_and_rising(tq, bf16):
    """Logits that rise along the sequence (the running maximum changes all the time) and
    span more than fp32's exponents can hold."""
    p = Pages(tq, 1, 1, 2000, 16, 3, 3, seed=31)
    s = np.arange(2000)
    p.kn[p.table[0, s // 16], 0, s % 16] = np.linspace(0.01, 300, 2000).astype(np.float16)
    p.upload(tq)
    if bf16:     # the bound of fp16 operands is empty for logits of this size: weights must still be finite and one
        p.vc[:] = 0.25
        p.upload(tq)
        q = torch.randn(1, 4, D, device="cuda").bfloat16()
        out = tq.decode_paged(q, p.cache, p.t, p.n)
        # every value row is nv/4 in each rotated coordinate: the output is a mean of nv times one vector
        v = 0.25 * p.Pv[0].astype(np.float64).sum(0)
        ratio = (out[0].float().cpu().numpy() @ v) / (v @ v)
        assert ((ratio > 0.49) & (ratio < 3.02)).all()
    else:
        rng = np.random.default_rng(5)
        Q = rng.standard_normal((1, 4, D)).astype(np.float32)
        want, _, bound, _ = p.want(Q)
        got = tq.decode_paged(dev(Q), p.cache, p.t, p.n).cpu().numpy()
        assert (np.abs(got - want) <= bound + 1e-5 * (1 + np.abs(want))).all()


def test_decode_ignores_what_lies_behind_a_length(tq):
    """Slots behind a length on the last page hold NaN and infinity lengths, other pages too."""
    for bf16, mass in ((False, False), (True, False), (True, True)):
        p = Pages(tq, 2, 2, 100, 64, seed=41, lengths=[70, 33])
        used = np.zeros(p.kn.shape, bool)
        for b, n in enumerate(p.lengths):
            pg, r = paged.slot_rows(p.table, b, int(n), p.page)
            used[pg, :, r] = True
        for x in (p.kn, p.vn):
            x[~used] = np.where(np.arange((~used).sum()) % 2, np.nan, np.inf)
        p.upload(tq)
        out, m = run_decode(tq, p, 4, bf16, mass)
        if mass:
            assert torch.isfinite(m).all()


def test_decode_magnitudes(tq):
    """Queries, centroids and lengths far from one: nothing overflows or vanishes on the way."""
    for big, nv, cs in ((1e6, 1.0, 1.0), (1e-6, 1.0, 1.0), (1.0, 3e-5, 1.0), (1.0, 2e4, 1.0), (1.0, 1.0, 1e-4)):
        p = Pages(tq, 1, 2, 150, 16, 3, 3, seed=51)
        p.vn = np.float16(nv) * p.vn
        p.kc, p.vc = (np.float32(cs) * c for c in (p.kc, p.vc))
        p.upload(tq)
        Q = (big * np.random.default_rng(6).standard_normal((1, 8, D))).astype(np.float32)
        for bf16 in (False, True):
            q = dev(Q).bfloat16() if bf16 else dev(Q)
            scale = D ** -0.5 / big / cs
            want, _, bound, _ = p.want(q.float().cpu().numpy(), scale, 2.0 ** -11 if bf16 else 2.0 ** -18, 2.0 ** -11 if bf16 else 2.0 ** -18)
            got = tq.decode_paged(q, p.cache, p.t, p.n, scale=scale).float().cpu().numpy()
            size = nv * cs
            tol = 1e-5 * (size + np.abs(want)) + (bound + 2.0 ** -8 * np.abs(want) if bf16 else 0)
            assert (np.abs(got - want) <= tol).all(), (big, nv, cs, bf16)


def test_decode_out_of_range_pages_and_lengths(tq):
    """A page number out of range makes its slots absent, a length out of range is cut; both
    are recorded, nothing out of range is read."""
    tq.device_faults()
    p = Pages(tq, 4, 2, 96, 16, seed=61)
    p.table[0, 2], p.table[1, 0], p.table[1, 5] = -7, p.kp.shape[0], 2 ** 31 - 1
    p.table[2, :] = -1
    p.upload(tq)
    p.n = dev(np.array([96, 96, 96, 96], np.int32))
    for bf16, mass in ((False, True), (True, False), (True, True)):
        run_decode(tq, p, 2, bf16, mass)
        assert tq.device_faults() == 32
    p = Pages(tq, 2, 2, 96, 16, seed=62)
    p.n = dev(np.array([-5, 2 ** 31 - 1], np.int32))
    p.lengths = np.array([0, 96], np.int32)
    run_decode(tq, p, 2)
    assert tq.device_faults() == 32
    run_decode(tq, Pages(tq, 1, 1, 40, 16, seed=63), 1)
    assert tq.device_faults() == 0


def test_decode_mass_shorter_than_the_pages(tq):
    """mass of 50 slots for pages of 64: a length of 50 fits it, one of 60 is cut to it."""
    tq.device_faults()
    p = Pages(tq, 2, 1, 64, 16, seed=65, lengths=[50, 64])
    m = torch.zeros(2, 1, 50, device="cuda")
    q = torch.randn(2, 2, D, device="cuda")
    out = tq.decode_paged(q, p.cache, p.t, p.n, mass=m)
    p.lengths = np.array([50, 50], np.int32)
    want, w, bound, wrel = p.want(q.cpu().numpy())
    check_out(out, want, bound, False)
    check_mass(m, np.zeros((2, 1, 50)), w[..., :50], wrel)
    assert tq.device_faults() == 32


def test_decode_shared_pages_and_repeats(tq):
    """Two sequences on the same pages (a shared prefix) with masses of their own; the same
    call gives the same bits."""
    p = Pages(tq, 3, 2, 160, 32, seed=71)
    p.table[1, :3], p.table[2] = p.table[0, :3], p.table[0]
    p.upload(tq)
    for bf16 in (False, True):
        a, ma = run_decode(tq, p, 4, bf16, True)
        b, mb = run_decode(tq, p, 4, bf16, True)
        assert torch.equal(a, b) and torch.equal(ma, mb)


def test_decode_offsets_past_32_bits(tq):
    """Planes of more than 2^32 bytes: the pages of one sequence lie at their end."""
    N, H, page = 180_000, 8, 64                                # 4.4e9 bytes of 3-bit rows a plane
    p = Pages(tq, 1, H, 200, page, seed=81)
    kp, vp = (torch.zeros(N, H, page, 48, dtype=torch.uint8, device="cuda") for _ in range(2))
    kn, vn = (torch.zeros(N, H, page, dtype=torch.float16, device="cuda") for _ in range(2))
    assert kp.numel() > 2 ** 32
    src = torch.from_numpy(p.table[0].astype(np.int64)).cuda()
    at = torch.tensor([N - 1, N - 3, 5, N - 2], device="cuda")
    for big, x in ((kp, p.kp), (vp, p.vp), (kn, p.kn), (vn, p.vn)):
        big[at] = dev(x)[src]
    q = torch.randn(1, H * 2, D, device="cuda")
    big = tq.PagedCache(kp, kn, vp, vn, p.cache.Pi_k, p.cache.k_codebook, p.cache.Pi_v, p.cache.v_codebook)
    for x in (q, q.bfloat16()):
        got = tq.decode_paged(x, big, at.int()[None].contiguous(), p.n)
        assert torch.equal(got, tq.decode_paged(x, p.cache, p.t, p.n))
    # append and evict at the same places
    K, V = torch.randn(1, H, D, device="cuda"), torch.randn(1, H, D, device="cuda")
    rows = torch.tensor([[0, 3, 9]], dtype=torch.int32, device="cuda")
    t = at.int()[None].contiguous()
    for cache, table in ((big, t), (p.cache, p.t)):
        tq.append_paged(K, V, rows, cache, table)
    mass = torch.arange(200, 0, -1, device="cuda", dtype=torch.float32).expand(1, H, 200).flip(-1).contiguous()
    pos = torch.zeros(1, H, 200, dtype=torch.int32, device="cuda")
    seen = torch.tensor([200], dtype=torch.int32, device="cuda")
    outs = [tq.evict_paged(c, tab, p.n, seen, mass, pos, 70, 0) for c, tab in ((big, t), (p.cache, p.t))]
    assert torch.equal(outs[0][0], outs[1][0])
    for x, y in ((kp, p.cache.k_plane), (vp, p.cache.v_plane), (kn, p.cache.k_norm), (vn, p.cache.v_norm)):
        assert torch.equal(x[at], y[src])


# ---- append -------------------------------------------------------------------

def check_append(p, before, K, V, rows, skipped=()):
    """Rows written as the definition says, everything else left as it was."""
    got = p.host()
    want = [x.copy() for x in before]
    for x, plane, norm, Pi, cb, bits in ((K, 0, 1, p.Pk, p.kc, p.kb), (V, 2, 3, p.Pv, p.vc, p.vb)):
        planes, norms = paged.append_rows(x, Pi, cb, bits)
        gap = paged.border_gap(x, Pi, cb)
        for i, (b, s, _) in enumerate(rows):
            if i in skipped or b < 0 or s < 0:
                continue
            pg, r = p.table[b, s // p.page], s % p.page
            gp = got[plane][pg, :, r]
            differ = oracle.unpack_indices(gp, bits, D) != oracle.unpack_indices(planes[i], bits, D)
            assert not (differ & (gap[i] > 1e-13)).any(), f"row {i}: {(differ & (gap[i] > 1e-13)).sum()} cells"
            step = np.spacing(norms[i].astype(np.float16)).astype(np.float64)
            gn = got[norm][pg, :, r]
            assert (np.abs(gn.astype(np.float64) - norms[i].astype(np.float64)) <= step).all() or (gn == norms[i]).all()
            want[plane][pg, :, r], want[norm][pg, :, r] = gp, gn
    for x, y in zip(got, want):
        assert np.array_equal(x.view(np.uint8), y.view(np.uint8)), "a row that was not named has changed"


@pytest.mark.parametrize("kb,vb", [(2, 2), (3, 3), (4, 4), (2, 4), (4, 3), (3, 2)])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("n", [1, 5, 127, 128, 129, 300])
def test_append(tq, kb, vb, bf16, n):
    H = 3 if n < 10 else 2
    p = Pages(tq, 2, H, 320, 32 if n % 2 else 16, kb, vb, rot=2 if n % 2 else 1, seed=n + kb)
    rng = np.random.default_rng(n)
    at = rng.permutation(640)[:n]
    rows = np.stack([at // 320, at % 320, rng.integers(0, 10 ** 6, n)], 1).astype(np.int32)
    skip = rng.random(n) < 0.1
    rows[skip, rng.integers(0, 2)] = -1
    K, V = (rng.standard_normal((n, H, D)) * np.exp(rng.standard_normal((n, H, 1))) for _ in range(2))
    K[..., [3, 17]] *= 15
    k, v = (dev(x.astype(np.float32)) for x in (K, V))
    if bf16:
        k, v = k.bfloat16(), v.bfloat16()
    before = p.host()
    mass = rng.random((2, H, 320)).astype(np.float32)
    pos = np.full((2, H, 320), -5, np.int32)
    m, q = dev(mass), dev(pos)
    tq.append_paged(k, v, dev(rows), p.cache, p.t, mass=m, positions=q)
    torch.cuda.synchronize()
    check_append(p, before, k.double().cpu().numpy(), v.double().cpu().numpy(), rows)
    for b, s, at in rows:
        if b >= 0 and s >= 0:
            mass[b, :, s], pos[b, :, s] = 0.0, at
    assert np.array_equal(m.cpu().numpy(), mass) and np.array_equal(q.cpu().numpy(), pos)


@pytest.mark.parametrize("kind", ["tight", "wide", "uneven", "same", "zero"])
@pytest.mark.parametrize("bf16", [False, True])
def test_append_codebooks(tq, kind, bf16):
    """Codebooks whose midpoints lie together, outside the coordinates' range, at very uneven
    distances, on one another, or all at 0."""
    for kb, vb in ((2, 3), (3, 4), (4, 2)):
        p = Pages(tq, 1, 2, 160, 16, kb, vb, seed=7 * kb)
        for name, b in (("kc", kb), ("vc", vb)):
            c = getattr(p, name).astype(np.float64)
            c = {"tight": 1e-3 * c, "wide": 8 * c, "uneven": np.sign(c) * (np.abs(c) + 0.02) ** 3 * 30, "same": np.full(c.size, 0.03),
                 "zero": np.zeros(c.size)}[kind]
            setattr(p, name, np.sort(c).astype(np.float32))
        p.upload(tq)
        rng = np.random.default_rng(kb)
        K, V = (dev(rng.standard_normal((150, 2, D)).astype(np.float32)) for _ in range(2))
        if bf16:
            K, V = K.bfloat16(), V.bfloat16()
        rows = np.stack([np.zeros(150), np.arange(150), np.arange(150)], 1).astype(np.int32)
        before = p.host()
        tq.append_paged(K, V, dev(rows), p.cache, p.t)
        check_append(p, before, K.double().cpu().numpy(), V.double().cpu().numpy(), rows)


def test_append_special_rows(tq):
    """Zero, one-hot, huge, tiny and subnormal rows; rows with NaN or infinity; coordinates
    that lie exactly on a midpoint."""
    rng = np.random.default_rng(3)
    n, H = 12, 2
    p = Pages(tq, 1, H, 64, 16, 3, 4, seed=91)
    had = np.stack([oracle.hadamard_rotation(np.where(np.arange(D) % (2 + h), 1.0, -1.0)) for h in range(H)]).astype(np.float32)
    p.Pk, p.Pv = had, had
    p.upload(tq)
    K = rng.standard_normal((n, H, D))
    K[0] = 0
    K[1] = 0
    K[1, :, 5] = 3.0
    K[2] *= 1e36
    K[3] *= 1e-37
    K[4] *= 1e-41
    K[5] = 0
    K[5, :, :2] = 0.7                                          # half of the Hadamard coordinates are exactly 0: a midpoint
    K[6] = 0
    K[6, :, 64:68] = -0.3
    K[7] *= 2e4
    K = K.astype(np.float32)
    rows = np.stack([np.zeros(n), np.arange(n) * 5, np.arange(n)], 1).astype(np.int32)
    for V in (K[::-1].copy(), K.copy()):
        before = p.host()
        tq.append_paged(dev(K), dev(V), dev(rows), p.cache, p.t)
        with np.errstate(over="ignore"):
            check_append(p, before, K.astype(np.float64), V.astype(np.float64), rows)
    bad = K.copy()
    bad[0, 0, 9], bad[1, 1, 0], bad[2, 0, 127] = np.nan, np.inf, -np.inf
    tq.append_paged(dev(bad), dev(K), dev(rows), p.cache, p.t)
    kp, kn, _, _ = p.host()
    for i, h in ((0, 0), (1, 1), (2, 0)):
        pg, r = p.table[0, rows[i, 1] // 16], rows[i, 1] % 16
        assert not kp[pg, h, r].any()
        assert np.isnan(kn[pg, h, r]) if i == 0 else np.isinf(kn[pg, h, r])
    # the other heads of those rows and the other rows are as ever
    want, _ = paged.append_rows(K.astype(np.float64)[:, ::-1], had[::-1], p.kc, 3)
    pg, r = p.table[0, 0], 0
    assert np.array_equal(kp[pg, 1, r], want[0, 0])


def test_append_out_of_range_rows(tq):
    tq.device_faults()
    p = Pages(tq, 2, 2, 64, 16, seed=95)
    p.table[1, 2] = -1
    p.table[0, 3] = p.kp.shape[0]
    p.upload(tq)
    rows = np.array([[2, 0, 0], [0, 64, 0], [1, 33, 0], [0, 50, 0], [2 ** 31 - 1, 2 ** 31 - 1, 0], [0, 7, 7], [-1, 3, 0], [1, -9, 0]], np.int32)
    K = np.random.default_rng(1).standard_normal((8, 2, D)).astype(np.float32)
    before = p.host()
    m, q = torch.ones(2, 2, 64, device="cuda"), torch.ones(2, 2, 64, dtype=torch.int32, device="cuda")
    tq.append_paged(dev(K), dev(K), dev(rows), p.cache, p.t, mass=m, positions=q)
    check_append(p, before, K.astype(np.float64), K.astype(np.float64), rows, skipped={0, 1, 2, 3, 4})
    assert tq.device_faults() == 32
    assert int((q != 1).sum()) == 2 and int((m != 1).sum()) == 2
    tq.append_paged(dev(K[:0]), dev(K[:0]), dev(rows[:0]), p.cache, p.t)
    tq.append_paged(dev(K[6:]), dev(K[6:]), dev(rows[6:]), p.cache, p.t)
    assert tq.device_faults() == 0


# ---- evict --------------------------------------------------------------------

def run_evict(tq, p, mass, pos, seen, budget, recent):
    before = p.host()
    S = mass.shape[-1]
    out = torch.full(mass.shape, -3.0, device="cuda"), torch.full(mass.shape, -7, dtype=torch.int32, device="cuda")
    ws = torch.full((tq.evict_paged_workspace_bytes(p.B, p.H, S, min(budget, S)),), 255, dtype=torch.uint8, device="cuda")
    got = tq.evict_paged(p.cache, p.t, p.n, dev(seen), dev(mass), dev(pos), budget, recent, workspace=ws, out=out)
    torch.cuda.synchronize()
    assert got[0] is out[0] and got[1] is out[1]
    want_m, want_p = np.full(mass.shape, -3.0, np.float32), np.full(mass.shape, -7, np.int32)
    want = [x.copy() for x in before]
    plan = paged.evict_paged(mass, pos, p.lengths, seen, budget, recent)
    for (b, h), (kept, to, fro) in plan.items():
        keep = kept.size
        m, q = mass[b, h].copy(), pos[b, h].copy()
        m[to], q[to] = m[fro], q[fro]
        want_m[b, h, :keep], want_p[b, h, :keep] = m[:keep], q[:keep]
        t = p.table[b]
        for x in want:
            x[t[to // p.page], h, to % p.page] = x[t[fro // p.page], h, fro % p.page]
    assert np.array_equal(got[0].cpu().numpy(), want_m, equal_nan=True)
    assert np.array_equal(got[1].cpu().numpy(), want_p)
    for x, y in zip(p.host(), want):
        assert np.array_equal(x.view(np.uint8), y.view(np.uint8))


def some_positions(rng, B, H, S, lengths):
    pos = np.full((B, H, S), -1, np.int32)
    for b in range(B):
        for h in range(H):
            pos[b, h, :lengths[b]] = rng.permutation(int(lengths[b]) + 5)[:lengths[b]]
    return pos


@pytest.mark.parametrize("S,budget,recent", [(1, 1, 0), (40, 1, 0), (40, 39, 3), (40, 40, 10), (40, 100, 0), (300, 16, 16),
                                             (300, 17, 5), (300, 150, 40), (1023, 512, 0), (1025, 900, 900), (2500, 700, 64),
                                             (5000, 4096, 128)])
def test_evict(tq, S, budget, recent):
    rng = np.random.default_rng(S + budget)
    lengths = [S, max(0, S - 13), 0, S // 2]
    for kb, vb, page in ((3, 3, 16), (2, 4, 64)):
        p = Pages(tq, 4, 2, S, page, kb, vb, rot=1, seed=S, lengths=lengths)
        mass = np.exp(2 * rng.standard_normal((4, 2, S))).astype(np.float32)
        run_evict(tq, p, mass, some_positions(rng, 4, 2, S, lengths), np.asarray(lengths, np.int32) + 5, budget, recent)


def test_evict_long(tq):
    """Longer than one CTA, and than a cluster, keeps in shared memory."""
    rng = np.random.default_rng(7)
    for S, budget in ((70001, 20000), (262147, 1000), (393216, 100), (700003, 350000)):
        p = Pages(tq, 1, 1, S, 256, 2, 2, seed=9)
        mass = np.exp(rng.standard_normal((1, 1, S))).astype(np.float32)
        pos = rng.permutation(S).astype(np.int32).reshape(1, 1, S)
        run_evict(tq, p, mass, pos, np.array([S], np.int32), budget, 100)


def test_evict_ties_and_special_weights(tq):
    """All equal; few values; zeros of both signs; NaN, infinities, negative; more protected
    slots than the budget; none protected; extreme positions."""
    rng = np.random.default_rng(8)
    S = 1500
    base = Pages(tq, 3, 2, S, 32, seed=11, lengths=[S, 1100, 700])
    special = np.array([0.0, -0.0, np.nan, np.inf, -np.inf, -1.0, 1e-45, 3e38, 1.0], np.float32)
    for mass in (np.zeros((3, 2, S), np.float32), rng.integers(0, 3, (3, 2, S)).astype(np.float32),
                 special[rng.integers(0, special.size, (3, 2, S))], np.full((3, 2, S), np.nan, np.float32)):
        for pos, seen, recent in ((some_positions(rng, 3, 2, S, base.lengths), base.lengths + 5, 50),
                                  (np.zeros((3, 2, S), np.int32), np.zeros(3, np.int32), 5),          # all protected
                                  (np.full((3, 2, S), -2 ** 31, np.int32), np.full(3, 2 ** 31 - 1, np.int32), 0),
                                  (np.full((3, 2, S), -2 ** 31, np.int32), np.full(3, -2 ** 31, np.int32), 2 ** 31 - 1)):
            for budget in (1, 333, 1100):
                run_evict(tq, base, mass, pos, seen.astype(np.int32), budget, recent)


def test_evict_out_of_range(tq):
    """A move whose page number is out of range is left out; lengths out of range are cut."""
    tq.device_faults()
    p = Pages(tq, 1, 1, 64, 16, seed=13)
    p.table[0, 0], p.table[0, 3] = -1, 2 ** 30
    p.upload(tq)
    before = p.host()
    mass = np.arange(64, dtype=np.float32).reshape(1, 1, 64)     # the last 32 are kept: 32..63 -> 0..31
    pos = np.zeros((1, 1, 64), np.int32)
    p.n = dev(np.array([2 ** 31 - 1], np.int32))
    tq.evict_paged(p.cache, p.t, p.n, dev(np.array([64], np.int32)), dev(mass), dev(pos), 32, 0)
    assert tq.device_faults() == 32
    got = p.host()
    # 32..47 -> 0..15 goes to an absent page, 48..63 -> 16..31 comes from one
    assert all(np.array_equal(x.view(np.uint8), y.view(np.uint8)) for x, y in zip(got, before))


# ---- together -----------------------------------------------------------------

def test_a_run_of_them_together(tq):
    """Prompt, decode steps with their weights, eviction, more decode steps, as a server runs
    them; every step against the definitions on the rows that are then in the cache."""
    rng = np.random.default_rng(99)
    B, H, G, S, budget, recent = 3, 2, 4, 160, 96, 16
    p = Pages(tq, B, H, S, 32, 3, 3, seed=100)
    p.lengths = np.zeros(B, np.int32)
    mass, pos = torch.full((B, H, S), 9.0, device="cuda"), torch.full((B, H, S), -1, dtype=torch.int32, device="cuda")
    other = torch.zeros_like(mass), torch.full_like(pos, -1)
    seen = np.zeros(B, np.int32)

    def append(counts):
        rows = np.concatenate([np.stack([np.full(c, b), p.lengths[b] + np.arange(c), seen[b] + np.arange(c)], 1)
                               for b, c in enumerate(counts)] + [np.full((2, 3), -1)]).astype(np.int32)
        x = torch.randn(2, len(rows), H, D, device="cuda").bfloat16()
        before = p.host()
        tq.append_paged(x[0], x[1], dev(rows), p.cache, p.t, mass=mass, positions=pos)
        check_append(p, before, x[0].double().cpu().numpy(), x[1].double().cpu().numpy(), rows)
        p.lengths += np.asarray(counts, np.int32)
        seen[:] += np.asarray(counts, np.int32)
        p.n = dev(p.lengths)
        p.kp, p.kn, p.vp, p.vn = p.host()

    append([130, 100, 5])
    for step in range(3):
        q = torch.randn(B, H * G, D, device="cuda").bfloat16()
        before = mass.cpu().numpy().astype(np.float64)
        out = tq.decode_paged(q, p.cache, p.t, p.n, mass=mass)
        qf = q.float().cpu().numpy()
        want, w, bound, wrel = p.want(qf, None, 2.0 ** -18, 2.0 ** -11)
        check_out(out, want, bound, True)
        check_mass(mass, before, w, wrel)
        if step == 1:
            m, ps = mass.cpu().numpy(), pos.cpu().numpy()
            plan = paged.evict_paged(m, ps, p.lengths, seen, budget, recent)
            tq.evict_paged(p.cache, p.t, p.n, dev(seen), mass, pos, budget, recent, out=other)
            mass, pos, other = other[0], other[1], (mass, pos)
            p.lengths = np.minimum(p.lengths, budget)
            p.n = dev(p.lengths)
            p.kp, p.kn, p.vp, p.vn = p.host()
            for (b, h), (kept, _, _) in plan.items():
                # the same tokens are there, whatever their order
                assert sorted(pos[b, h, :kept.size].tolist()) == sorted(ps[b, h, kept].tolist())
        append([1, 1, 1])
    assert tq.device_faults() == 0


def test_streams_and_graphs(tq):
    """The three calls on a side stream, captured into one graph each with workspaces of their
    own, replayed after the inputs changed."""
    B, H, G, S = 2, 2, 4, 200
    p = Pages(tq, B, H, S, 16, seed=111, lengths=[200, 150])
    q = torch.randn(B, H * G, D, device="cuda").bfloat16()
    K = torch.randn(2, B, H, D, device="cuda")
    rows = torch.tensor([[0, 3, 3], [1, 140, 140]], dtype=torch.int32, device="cuda")
    mass, pos = torch.rand(B, H, S, device="cuda"), torch.zeros(B, H, S, dtype=torch.int32, device="cuda")
    seen = torch.tensor([200, 150], dtype=torch.int32, device="cuda")
    mass0 = mass.clone()
    planes = (p.cache.k_plane, p.cache.k_norm, p.cache.v_plane, p.cache.v_norm)
    save = [x.clone() for x in planes]

    def step(ws1, ws2, out, eo):
        tq.append_paged(K[0], K[1], rows, p.cache, p.t, mass=mass, positions=pos)
        tq.decode_paged(q, p.cache, p.t, p.n, mass=mass, workspace=ws1, out=out)
        tq.evict_paged(p.cache, p.t, p.n, seen, mass, pos, 100, 0, workspace=ws2, out=eo)

    def fresh():
        return (torch.empty(tq.decode_paged_workspace_bytes(B, H, G, S, True), dtype=torch.uint8, device="cuda"),
                torch.empty(tq.evict_paged_workspace_bytes(B, H, S, 100), dtype=torch.uint8, device="cuda"),
                torch.empty_like(q), (torch.zeros_like(mass), torch.zeros_like(pos)))

    def reset():
        mass.copy_(mass0)
        pos.zero_()
        for x, y in zip(planes, save):
            x.copy_(y)

    first = fresh()
    step(*first)                                               # eager
    torch.cuda.synchronize()
    reset()
    side, graphs = torch.cuda.Stream(), []
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        g, bufs = torch.cuda.CUDAGraph(), fresh()
        with torch.cuda.stream(side):
            with torch.cuda.graph(g, stream=side):
                step(*bufs)
        graphs.append((g, bufs))
    for g, bufs in graphs:
        reset()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs[2], first[2])
        assert torch.equal(bufs[3][0][..., :100], first[3][0][..., :100]) and torch.equal(bufs[3][1][..., :100], first[3][1][..., :100])
    # other lengths and queries in the same buffers
    reset()
    p.n.copy_(torch.tensor([77, 3], dtype=torch.int32))
    q.copy_(torch.randn(B, H * G, D, device="cuda").bfloat16())
    graphs[0][0].replay()
    torch.cuda.synchronize()
    got = [graphs[0][1][2].clone(), mass.clone()]
    reset()
    step(*first)
    torch.cuda.synchronize()
    assert torch.equal(got[0], first[2]) and torch.equal(got[1], mass)
    # a side stream of its own, behind work that is still under way there
    reset()
    with torch.cuda.stream(side):
        junk = torch.randn(4096, 4096, device="cuda")
        for _ in range(20):
            junk = junk @ junk * 1e-4
        step(*first)
    side.synchronize()
    assert torch.equal(got[0], first[2])


def test_binding_refusals(tq):
    p = Pages(tq, 2, 2, 64, 16, seed=121)
    q = torch.randn(2, 4, D, device="cuda")
    bad = [dict(Q=q.half()), dict(Q=q[:1]), dict(Q=q[:, :3]), dict(Q=q[:, :1]), dict(Q=q.transpose(0, 1)), dict(Q=q.cpu()),
           dict(Q=q[..., :64].contiguous()), dict(Q=None),
           dict(page_table=p.t.long()), dict(page_table=p.t[0]), dict(page_table=p.t.cpu()), dict(page_table=p.t.t()),
           dict(lengths=p.n[:1]), dict(lengths=p.n.long()), dict(mass=torch.zeros(2, 2, 64, device="cuda").double()),
           dict(mass=torch.zeros(2, 1, 64, device="cuda")), dict(out=q.bfloat16()), dict(out=q[:1]),
           dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), dict(scale=float("inf"))]
    for kw in bad:
        args = dict(Q=q, cache=p.cache, page_table=p.t, lengths=p.n)
        args.update(kw)
        with pytest.raises((TypeError, ValueError, tq.TQError)):
            tq.decode_paged(**args)
    K, rows = torch.randn(3, 2, D, device="cuda"), torch.zeros(3, 3, dtype=torch.int32, device="cuda")
    for kw in (dict(K=K.double()), dict(V=K[:2]), dict(V=K.bfloat16()), dict(rows=rows.long()), dict(rows=rows[:, :2]),
               dict(K=K[:, :1]), dict(mass=torch.zeros(2, 2, 0, device="cuda")), dict(positions=torch.zeros(2, 2, 64, device="cuda"))):
        args = dict(K=K, V=K, rows=rows, cache=p.cache, page_table=p.t)
        args.update(kw)
        with pytest.raises((TypeError, ValueError, tq.TQError)):
            tq.append_paged(**args)
    mass, pos = torch.zeros(2, 2, 64, device="cuda"), torch.zeros(2, 2, 64, dtype=torch.int32, device="cuda")
    for kw in (dict(budget=0), dict(budget=-2 ** 40), dict(recent=-1), dict(mass=mass[0]), dict(positions=pos.long()),
               dict(out=(mass, pos)), dict(seen=p.n.cpu()), dict(mass=mass[..., :63])):
        args = dict(cache=p.cache, page_table=p.t, lengths=p.n, seen=p.n, mass=mass, positions=pos, budget=32, recent=0)
        args.update(kw)
        with pytest.raises((TypeError, ValueError, tq.TQError)):
            tq.evict_paged(**args)
    c = p.cache
    good = dict(k_plane=c.k_plane, k_norm=c.k_norm, v_plane=c.v_plane, v_norm=c.v_norm, Pi_k=c.Pi_k, k_codebook=c.k_codebook,
                Pi_v=c.Pi_v, v_codebook=c.v_codebook)
    for kw in (dict(k_plane=c.k_plane[..., :40].contiguous()), dict(k_norm=c.k_norm[:1]), dict(v_plane=c.v_plane[:1]),
               dict(k_codebook=c.k_codebook[:4]), dict(Pi_v=c.Pi_v[:1]), dict(k_norm=c.k_norm.float()), dict(Pi_k=c.Pi_k.transpose(1, 2))):
        with pytest.raises((TypeError, ValueError)):
            tq.PagedCache(**dict(good, **kw))
