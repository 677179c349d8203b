"""Host-only checks of the paged cache: the float64 definitions against brute force, and the
refusals of the C ABI and of the binding (nothing is launched)."""
import ctypes
import math

import numpy as np
import pytest

import oracle
from oracle import paged
from conftest import codebook
from compressed_kv_cache_gb300 import build as tqbuild
from compressed_kv_cache_gb300 import tq

D = 128


# ---- the definitions ----------------------------------------------------------

def test_append_rows_match_the_codec_and_zero_rows():
    rng = np.random.default_rng(1)
    cb = codebook(D, 3)[0].astype(np.float32)
    Pi = np.stack([oracle.haar_rotation(rng.standard_normal((D, D))) for _ in range(2)]).astype(np.float32)
    x = rng.standard_normal((5, 3, D))
    x[2, 1] = 0.0
    planes, norms = paged.append_rows(x, Pi, cb, 3)
    idx, norm = oracle.compress_mse(x[:, 2], Pi[0], cb)        # head 2 of 3 uses rotation 2 % 2
    assert np.array_equal(planes[:, 2], oracle.pack_indices(idx, 3)) and np.array_equal(norms[:, 2], norm)
    assert norms[2, 1] == 0.0
    zero = oracle.unpack_indices(planes[2, 1:2], 3, D)
    assert (zero == int(((cb[1:].astype(np.float64) + cb[:-1]) * 0.5 < 0).sum())).all()


def test_decode_paged_matches_the_dense_decode():
    rng = np.random.default_rng(2)
    cb = codebook(D, 2)[0].astype(np.float32)
    Pi = oracle.haar_rotation(rng.standard_normal((D, D))).astype(np.float32)[None]
    n, page, N = 41, 16, 6
    kp, vp = rng.integers(0, 256, (N, 1, page, 32), dtype=np.uint8), rng.integers(0, 256, (N, 1, page, 32), dtype=np.uint8)
    kn, vn = (rng.uniform(0.5, 2, (N, 1, page)).astype(np.float16) for _ in range(2))
    table = np.array([[4, 1, 5], [0, -1, -1]], dtype=np.int32)
    Q = rng.standard_normal((2, 2, D))
    out, w, bound, _ = paged.decode_paged(Q, kp, kn, vp, vn, table, np.array([n, 0]), Pi, cb, Pi, cb, 0.2, 2.0 ** -11)
    flat = lambda a: np.concatenate([a[4, 0], a[1, 0], a[5, 0]])[:n]
    want = oracle.decode_mse(Q[0] @ Pi[0].astype(np.float64).T, oracle.unpack_indices(flat(kp), 2, D), flat(kn), cb,
                             oracle.unpack_indices(flat(vp), 2, D), flat(vn), cb, Pi[0], 0.2)
    assert np.abs(out[0] - want).max() < 1e-12
    assert np.allclose(w[0, 0, :, :n].sum(-1), 1.0) and not w[0, 0, :, n:].any()
    assert not out[1].any() and not w[1].any()
    # the bound holds for operands that are rounded to fp16
    h = lambda a: np.asarray(a, np.float16).astype(np.float64)
    a = h(Q[0] @ Pi[0].astype(np.float64).T)
    s = 0.2 * (a @ h(cb)[oracle.unpack_indices(flat(kp), 2, D)].T) * flat(kn).astype(np.float64)
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    cv = cb.astype(np.float64)[oracle.unpack_indices(flat(vp), 2, D)]
    assert (np.abs(((p * flat(vn).astype(np.float64)) @ cv) @ Pi[0].astype(np.float64) - out[0]) <= bound[0] + 1e-12).all()


def test_evict_paged_by_hand():
    mass = np.array([[[5.0, 1.0, 5.0, np.nan, 9.0, 0.0]]])
    pos = np.array([[[0, 1, 2, 3, 4, 5]]])
    kept, to, fro = paged.evict_paged(mass, pos, [6], [6], 3, 1)[0, 0]
    assert kept.tolist() == [0, 4, 5] and to.tolist() == [1, 2] and fro.tolist() == [4, 5]
    kept, to, fro = paged.evict_paged(mass, pos, [4], [6], 3, 0)[0, 0]
    assert kept.tolist() == [0, 1, 2] and to.size == 0
    kept, to, fro = paged.evict_paged(mass, pos, [2], [6], 3, 0)[0, 0]
    assert kept.tolist() == [0, 1] and to.size == 0


# ---- refusals -----------------------------------------------------------------

FAKE = 0x100000       # 16-byte aligned, never dereferenced
FAR = 0x40000000
ODD = 0x100004


@pytest.fixture(scope="module")
def L():
    tqbuild.build()
    return tq.lib()


def struct(**kw):
    v = dict(k_plane=FAKE, k_norm=FAKE, v_plane=FAKE, v_norm=FAKE, Pi_k=FAKE, Pi_v=FAKE, k_codebook=FAKE,
             v_codebook=FAKE, n_pages=8, H=4, page_size=16, D=D, k_bits=3, v_bits=3, rot_heads=4)
    v.update(kw)
    return tq._PagedCacheStruct(*[v[n] for n, _ in tq._PagedCacheStruct._fields_])


BAD_CACHES = [(dict(k_plane=None), 1), (dict(v_norm=None), 1), (dict(Pi_v=ODD), 3), (dict(k_codebook=ODD), 3),
              (dict(n_pages=0), 1), (dict(H=0), 1), (dict(H=70000), 1), (dict(rot_heads=5), 1), (dict(rot_heads=0), 1),
              (dict(D=64), 2), (dict(D=0), 1), (dict(k_bits=1), 1), (dict(v_bits=5), 1), (dict(page_size=8), 2),
              (dict(page_size=48), 2), (dict(page_size=512), 2), (dict(page_size=0), 1)]


def calls(L, c):
    p = None if c is None else ctypes.byref(c)              # holds on to the struct

    def append(K=FAKE, type=0, rows=FAKE, n=4, table=FAKE, B=2, M=4, mass=None, pos=None, S=0):
        return L.tq_append_paged(p, K, FAKE, type, rows, n, table, B, M, mass, pos, S, None)

    def decode(Q=FAKE, type=0, table=FAKE, lengths=FAKE, B=2, G=2, M=4, scale=0.1, mass=None, S=0, out=FAKE, ws=FAKE,
               wsb=1 << 40):
        return L.tq_decode_paged(p, Q, type, table, lengths, B, G, M, scale, mass, S, out, ws, wsb, None)

    def evict(table=FAKE, lengths=FAKE, seen=FAKE, B=2, M=4, mass=FAKE, pos=FAKE + (1 << 20), S=64, budget=32, recent=0,
              mo=FAR, po=FAR + (1 << 20), ws=FAKE, wsb=1 << 40):
        return L.tq_evict_paged(p, table, lengths, seen, B, M, mass, pos, S, budget, recent, mo, po, ws, wsb, None)
    return append, decode, evict


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches(L, kw, status):
    for call in calls(L, struct(**kw)):
        assert call() == status


def test_shared_arguments(L):
    for call in calls(L, None):
        assert call() == 1
    for call in calls(L, struct()):
        assert call(table=None) == 1 and call(table=ODD) == 3
        assert call(B=0) == 1 and call(B=70000) == 1 and call(M=0) == 1 and call(M=1 << 28) == 1


def test_append_arguments(L):
    append, _, _ = calls(L, struct())
    assert append(n=-1) == 1 and append(type=2) == 1 and append(S=-1) == 1
    assert append(K=None) == 1 and append(K=ODD) == 3 and append(rows=None) == 1
    assert append(mass=FAKE, S=0) == 1 and append(mass=ODD, S=8) == 3 and append(pos=ODD, S=8) == 3
    assert append(n=1 << 30) == 1                             # n * H does not fit
    assert append(n=0, K=None) == 0                            # nothing to do


def test_decode_arguments(L):
    _, decode, _ = calls(L, struct())
    assert decode(Q=None) == 1 and decode(Q=ODD) == 3 and decode(lengths=None) == 1 and decode(out=ODD) == 3
    assert decode(G=0) == 1 and decode(type=7) == 1
    assert decode(scale=math.inf) == 1 and decode(scale=math.nan) == 1
    assert decode(mass=FAKE, S=0) == 1 and decode(mass=ODD, S=8) == 3 and decode(S=-1) == 1
    assert decode(G=1 << 24) == 1                              # too many queries
    assert decode(B=60000, M=100000) == 1                      # the key tiles do not fit 32 bits
    need = tq.decode_paged_workspace_bytes(2, 4, 2, 64, True)
    assert need > 0
    assert decode(ws=None) == 4 and decode(ws=ODD) == 3 and decode(mass=FAKE, S=64, wsb=need - 1) == 4


def test_evict_arguments(L):
    _, _, evict = calls(L, struct())
    for name in ("lengths", "seen", "mass", "pos", "mo", "po"):
        assert evict(**{name: None}) == 1 and evict(**{name: ODD}) == 3
    assert evict(budget=0) == 1 and evict(budget=-4) == 1 and evict(recent=-1) == 1 and evict(S=0) == 1
    assert evict(mo=FAKE) == 1 and evict(po=FAKE + (1 << 20) + 16) == 1 and evict(po=FAR) == 1     # overlaps
    need = tq.evict_paged_workspace_bytes(2, 4, 64, 32)
    assert need > 0
    assert evict(ws=None) == 4 and evict(ws=ODD) == 3 and evict(wsb=need - 1) == 4


def test_workspace_queries(L):
    assert tq.decode_paged_workspace_bytes(0, 1, 1, 1, False) == 0
    assert tq.decode_paged_workspace_bytes(1, 1, 1, 0, False) > 0
    small, large = (tq.decode_paged_workspace_bytes(4, 8, 4, S, True) for S in (1000, 100000))
    assert large - small >= 99000 * 4 * 8 * 4 * 4              # the logits
    assert tq.evict_paged_workspace_bytes(1, 1, 0, 1) == 0 and tq.evict_paged_workspace_bytes(1, 1, 8, 0) == 0
    assert tq.evict_paged_workspace_bytes(2, 3, 100, 1000) > 0


def test_binding_refuses_cpu_tensors(L):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="CUDA"):
        tq.PagedCache(torch.zeros(1, 1, 16, 48, dtype=torch.uint8), torch.zeros(1, 1, 16, dtype=torch.float16),
                      torch.zeros(1, 1, 16, 48, dtype=torch.uint8), torch.zeros(1, 1, 16, dtype=torch.float16),
                      torch.eye(D), torch.zeros(8), torch.eye(D), torch.zeros(8))
