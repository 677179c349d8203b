"""Host-only checks of the 8-bit paged cache and of norm_rope: the float64 definitions, the rotation's
table, and the refusals of the C ABI and of the binding (nothing is launched)."""
import ctypes
import math

import numpy as np
import pytest

from oracle import int8
from compressed_kv_cache_gb300 import build as tqbuild
from compressed_kv_cache_gb300 import tq


# ---- the definitions ----------------------------------------------------------

def empty(N, H, page, D, rng):
    """A cache as a server finds it: any bytes."""
    return (rng.integers(0, 256, (N, H, page, D), dtype=np.uint8), rng.integers(0, 256, (N, H, page, D), dtype=np.uint8),
            rng.integers(-128, 128, (N, H, page // 16, 2), dtype=np.int8))


@pytest.mark.parametrize("cuts", [(37,), (1,) * 37, (5, 11, 1, 20), (16, 16, 5), (15, 2, 20)])
def test_codes_do_not_depend_on_how_tokens_arrive(cuts):
    rng = np.random.default_rng(7)
    N, H, page, D, first = 4, 2, 16, 64, 3
    K = rng.standard_normal((first + 37, H, D)) * np.exp2(rng.integers(-40, 40, (first + 37, H, 1)).astype(np.float64))
    table = np.array([[2, 0, 3]])
    whole, parts = empty(N, H, page, D, rng), empty(N, H, page, D, rng)
    int8.append(*whole, K, -K, [0, first + 37], [0], table)
    at = 0
    for c in (first,) + cuts:
        int8.append(*parts, K[at:at + c], -K[at:at + c], [0, c], [at], table)
        at += c
    s = np.arange(at)
    for x, y in zip(whole[:2], parts[:2]):
        assert np.array_equal(x[table[0, s // page], :, s % page], y[table[0, s // page], :, s % page])
    assert np.array_equal(whole[2][table[0]], parts[2][table[0]])
    # half a step of the block at most, for values in the middle of a cell none
    v = int8.values(whole[0], whole[2], 0, table[0, s // page], s % page)
    step = np.exp2(whole[2][table[0, s // page], :, s % page // 16, 0].astype(np.float64))[..., None]
    assert (np.abs(v - K) <= step / 2).all()
    most = np.abs(K).max(-1)
    for blk in range(3):
        e = whole[2][table[0, blk], :, 0, 0].astype(np.float64)
        top = most[16 * blk:16 * blk + 16].max(0)
        assert (top < np.exp2(e + 7)).all() and (top >= np.exp2(e + 6)).all()


def test_exponents_at_the_ends():
    assert int8.exponent(0.0) == -120 and int8.exponent(1e-45) == -120
    assert int8.exponent(float(np.finfo(np.float32).max)) == 121 and int8.exponent(1.0) == -6
    assert int8.exponent(np.nextafter(np.float32(1), np.float32(0))) == -7
    x = np.array([np.inf, -np.inf, np.nan, 0.0, -1e-300, 127.9])
    assert int8.codes_of(x, 0).tolist() == [255, 0, 0, 128, 127, 255]


def test_attend_by_hand():
    rng = np.random.default_rng(2)
    N, H, page, D = 3, 1, 16, 64
    cache = empty(N, H, page, D, rng)
    K, V = rng.standard_normal((2, 20, H, D))
    table = np.array([[1, 2]])
    int8.append(*cache, K, V, [0, 20], [0], table)
    Q = rng.standard_normal((3, 2, D))
    out, _ = int8.attend(Q, *cache, [0, 3], [17], table, 0.125, window=4, sinks=2)
    s = np.arange(20)
    k, v = (int8.values(cache[i], cache[2], i, table[0, s // page], s % page)[:, 0] for i in range(2))
    for i, at in enumerate((17, 18, 19)):
        seen = [0, 1] + list(range(at - 3, at + 1))
        for g in range(2):
            z = 0.125 * k[seen] @ Q[i, g]
            w = np.exp(z) / np.exp(z).sum()
            assert np.abs(w @ v[seen] - out[i, g]).max() < 1e-12
    nothing, _ = int8.attend(Q, *cache, [0, 3], [17], np.array([[-1, 9]]), 0.125)
    assert not nothing.any()


def test_norm_rope_by_hand():
    rng = np.random.default_rng(3)
    x, w = rng.standard_normal((2, 3, 16)), rng.standard_normal(16)
    freq, axis = np.array([1.0, 0.1, 0.01, 0.5]), [0, 1, 1, 0]
    pos = np.array([[5, -7], [100000, 3]])
    for paired in (False, True):
        out, _ = int8.norm_rope(x, w, 1e-5, pos, freq, axis, paired)
        y = x[1, 2] / math.sqrt((x[1, 2] ** 2).mean() + 1e-5) * w
        for i in range(4):
            a, b = (2 * i, 2 * i + 1) if paired else (i, i + 4)
            t = pos[1, axis[i]] * freq[i]
            assert abs(out[1, 2, a] - (y[a] * math.cos(t) - y[b] * math.sin(t))) < 1e-12
            assert abs(out[1, 2, b] - (y[b] * math.cos(t) + y[a] * math.sin(t))) < 1e-12
        assert np.allclose(out[1, 2, 8:], y[8:])


def test_rotary_turns():
    torch = pytest.importorskip("torch")
    made = {}

    class Fake(tq.Rotary):      # the table without a device
        __slots__ = ()
    dev = tq._dev
    tq._dev = lambda t, name, dtypes: made.setdefault(name, t).data_ptr()
    try:
        freq = [1.0, 10000.0 ** -0.25, -0.5, 2 * math.pi * 3.25] + [0.0] * 4
        r = Fake(freq, torch.device("cpu"), axis=[0, 0, 1, 1, 2, 2, 0, 0])
    finally:
        tq._dev = dev
    assert r.axes == 3 and r.pairs == 8 and made["axis"].tolist() == [0, 0, 1, 1, 2, 2, 0, 0]
    for f, t in zip(freq, made["turns"].tolist()):
        # position * turn modulo 2^64 is the angle of a far position too: 64-bit floats have 2^-53 of 2^20 radians there
        for pos in (1, -3, 1 << 20):
            got = (t * pos % (1 << 64)) * 2.0 ** -64 * 2 * math.pi
            assert abs(math.remainder(got - f * pos, 2 * math.pi)) < 1e-8
    for bad in ([], [1.0] * 3, [math.inf] * 4, [1.0] * 132):
        with pytest.raises(ValueError):
            tq.Rotary(bad, torch.device("cpu"))
    with pytest.raises(ValueError):
        tq.Rotary([1.0] * 4, torch.device("cpu"), axis=[0, 0, 0, 8])
    with pytest.raises(ValueError, match="CUDA"):
        tq.Rotary([1.0] * 4, torch.device("cpu"))


# ---- refusals -----------------------------------------------------------------

FAKE = 0x100000       # 16-byte aligned, never dereferenced
FAR = 0x4000000000
ODD = 0x100004


@pytest.fixture(scope="module")
def L():
    tqbuild.build()
    return tq.lib()


def struct(**kw):
    v = dict(k_codes=FAKE, v_codes=FAKE, exponents=FAKE, n_pages=8, H=4, page_size=16, D=128)
    v.update(kw)
    return tq._Int8CacheStruct(*[v[n] for n, _ in tq._Int8CacheStruct._fields_])


BAD_CACHES = [(dict(k_codes=None), 1), (dict(v_codes=ODD), 3), (dict(exponents=None), 1), (dict(n_pages=0), 1), (dict(H=0), 1),
              (dict(H=70000), 1), (dict(D=96), 2), (dict(D=256), 2), (dict(D=0), 1), (dict(page_size=8), 2), (dict(page_size=48), 2),
              (dict(page_size=512), 2), (dict(page_size=0), 1), (dict(n_pages=1 << 30), 1)]


def calls(L, c):
    p = None if c is None else ctypes.byref(c)

    def append(K=FAKE, ks=512, V=FAKE, vs=512, type=0, starts=FAKE, lengths=FAKE, n=4, table=FAKE, B=2, M=4):
        return L.tq_append_int8(p, K, ks, V, vs, type, starts, lengths, n, table, B, M, None)

    def read(K=FAKE, V=FAKE, type=0, starts=FAKE, lengths=FAKE, n=4, table=FAKE, B=2, M=4):
        return L.tq_read_int8(p, K, V, type, starts, lengths, n, table, B, M, None)

    def attend(K=FAKE, type=0, starts=FAKE, lengths=FAKE, n=4, G=2, table=FAKE, B=2, M=4, window=0, sinks=0, scale=0.1, out=FAKE,
               ws=FAKE, wsb=1 << 40):
        return L.tq_attend_int8(p, K, type, starts, lengths, n, G, table, B, M, window, sinks, scale, out, ws, wsb, None)
    return append, read, attend


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches(L, kw, status):
    for call in calls(L, struct(**kw)):
        assert call() == status


def test_shared_arguments(L):
    for call in calls(L, None):
        assert call() == 1
    for call in calls(L, struct()):
        for name in ("starts", "lengths", "table", "K"):
            assert call(**{name: None}) == 1 and call(**{name: ODD}) == 3
        assert call(B=0) == 1 and call(B=70000) == 1 and call(M=0) == 1 and call(M=1 << 28) == 1
        assert call(n=-1) == 1 and call(n=1 << 30) == 1 and call(type=2) == 1
        assert call(n=0, K=None) == 0                            # nothing to do
    for call in calls(L, struct(H=60000)):
        assert call(B=60000) == 1                                # sequences times heads


def test_append_and_attend_arguments(L):
    append, _, attend = calls(L, struct())
    assert append(V=None) == 1 and append(V=ODD) == 3
    assert append(ks=-4) == 1 and append(ks=510) == 1 and append(vs=516, type=1) == 1
    assert attend(G=0) == 1 and attend(G=1 << 29) == 1 and attend(window=-1) == 1 and attend(sinks=-1) == 1
    assert attend(scale=math.inf) == 1 and attend(scale=math.nan) == 1 and attend(out=None) == 1 and attend(out=ODD) == 3
    need = tq.attend_int8_workspace_bytes(4, 2, 4, 2, 128)
    assert need > 0
    assert attend(ws=None) == 4 and attend(ws=ODD) == 3 and attend(wsb=need - 1) == 4
    for bad in ((0, 1, 1, 1, 128), (1, 0, 1, 1, 128), (1, 1, 0, 1, 128), (1, 1, 1, 0, 128), (1, 1, 1, 1, 96)):
        assert tq.attend_int8_workspace_bytes(*bad) == 0


def test_norm_rope_arguments(L):
    def call(q=FAKE, qt=1024, qh=128, k=FAKE + (1 << 24), kt=1024, kh=128, type=0, wq=None, wk=None, wt=0, eps=1e-6, pos=FAKE, axes=1,
             turns=FAKE, axis=FAKE, pairs=64, paired=0, qo=FAR, ko=FAR + (1 << 24), n=4, Hq=8, Hk=8, D=128):
        return L.tq_norm_rope(q, qt, qh, k, kt, kh, type, wq, wk, wt, eps, pos, axes, turns, axis, pairs, paired, qo, ko, n, Hq, Hk, D, None)
    assert call(n=0, q=None) == 0
    for name in ("q", "k", "pos", "turns", "axis", "qo", "ko"):
        assert call(**{name: None}) == 1 and call(**{name: ODD}) == 3
    assert call(wq=ODD) == 3 and call(wk=ODD) == 3
    assert call(n=-1) == 1 and call(Hq=0) == 1 and call(Hk=-1) == 1 and call(D=0) == 1 and call(D=264) == 1 and call(n=1 << 29) == 1
    assert call(type=2) == 1 and call(wt=3) == 1 and call(axes=0) == 1 and call(axes=9) == 1 and call(paired=2) == 1
    assert call(eps=-1.0) == 1 and call(eps=math.nan) == 1 and call(eps=math.inf) == 1
    assert call(pairs=0) == 1 and call(pairs=68) == 1 and call(pairs=6) == 2 and call(D=100, pairs=48) == 2
    assert call(qt=-1024) == 1 and call(qh=130) == 1 and call(kt=1026) == 1 and call(type=1, kh=132) == 1
    # outputs over inputs or each other
    assert call(qo=FAKE + 512) == 1 and call(ko=FAKE) == 1 and call(qo=FAKE + (1 << 24)) == 1 and call(ko=FAR) == 1
    assert call(qo=FAKE, qt=2048) == 1                            # in place only where q is dense


def test_binding_refuses_cpu_tensors(L):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="CUDA"):
        tq.Int8Cache(torch.zeros(1, 1, 16, 64, dtype=torch.uint8), torch.zeros(1, 1, 16, 64, dtype=torch.uint8),
                     torch.zeros(1, 1, 1, 2, dtype=torch.int8))
