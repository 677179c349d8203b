"""GPU parity of the 8-bit paged cache and of norm_rope against the float64 definitions in oracle/int8.py.

Codes, exponents and values read back are exact.  norm_rope: a coordinate is off by at most 26 * 2^-24 of
|y_a| + |y_b| (angle to fp32: pi * 2^-24, sine and cosine one step each, 2^-23; the norm 16 roundings of 2^-24, the
rotation's products and sum 4), and half a step of the result's type.  attend: logits to 2^-17 of
scale sum |q_d k_d| (queries as two fp16 parts, 2^-22; 16 additions of a product's parts, each to 2^-22 of what is
summed; exp2 and the scale's product 2^-22 more), weights rounded to fp16 (bf16 queries: one part, 2^-11; fp32: two, 2^-22), sums of values to 2^-14 (bf16) or
2^-17 (fp32), the output to half a step.  Weights are taken 2^7 above the largest's 1, so that the rounding of small ones,
2^-25 below fp16's normal numbers, is 2^-32 of the largest."""
import numpy as np
import pytest

from oracle import int8

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


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


def wide(t):
    return t.detach().cpu().double().numpy()


class Setup:
    """Sequences of `counts` new tokens behind `before` slots, on shuffled pages; the cache is filled by the
    definition (rows of live slots) over random bytes."""

    def __init__(self, counts, before, H=2, D=128, page=16, dtype=BF16, seed=0, spread=2, padding=0, spare=2):
        rng = self.rng = np.random.default_rng(seed)
        self.counts, self.before, self.H, self.D, self.page, self.dtype = counts, before, H, D, page, dtype
        B = len(counts)
        used = [-(-(c + n) // page) for c, n in zip(counts, before)]
        M, N = max(max(used), 1), sum(used) + spare
        self.table = np.full((B, M), -1, dtype=np.int32)
        ids, at = rng.permutation(N), 0
        for b in range(B):
            self.table[b, :used[b]] = ids[at:at + used[b]]
            at += used[b]
        self.starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.lengths = np.array(before, dtype=np.int32)
        self.n = int(self.starts[-1]) + padding
        self.cache = (rng.integers(0, 256, (N, H, page, D), dtype=np.uint8), rng.integers(0, 256, (N, H, page, D), dtype=np.uint8),
                      rng.integers(-128, 128, (N, H, page // 16, 2), dtype=np.int8))
        old = [self.rows(sum(before), spread) for _ in range(2)]
        int8.append(*self.cache, *(wide(x) for x in old), np.concatenate([[0], np.cumsum(before)]), np.zeros(B, int), self.table)
        self.K, self.V = self.rows(self.n, spread), self.rows(self.n, spread)

    def rows(self, n, spread):
        x = self.rng.standard_normal((n, self.H, self.D)) * np.exp2(self.rng.uniform(-spread, spread, (n, 1, 1)))
        x[:, :, 5] *= 8.0
        return torch.from_numpy(x).to(self.dtype)

    def append(self):
        int8.append(*self.cache, wide(self.K), wide(self.V), self.starts, self.lengths, self.table)

    def queries(self, G, size=1.0):
        return torch.from_numpy(self.rng.standard_normal((self.n, self.H * G, self.D)) * size).to(self.dtype)

    def device(self, tq):
        t = [dev(x) for x in self.cache]
        return tq.Int8Cache(*t), t, dev(self.table), dev(self.starts), dev(self.lengths)


def bounds(dtype):
    """logit, value, least of a definition's bound"""
    return (2.0 ** -17, 2.0 ** -11 + 2.0 ** -14, 2.0 ** -32) if dtype is BF16 else (2.0 ** -17, 2.0 ** -17, 2.0 ** -32)


def check_attend(tq, s, G=4, window=0, sinks=0, scale=None, size=1.0, Q=None, faults=0):
    Q = s.queries(G, size) if Q is None else Q
    cache, _, table, starts, lengths = s.device(tq)
    out = torch.full(Q.shape, 7.0, dtype=s.dtype, device="cuda")
    got = tq.attend_int8(Q.cuda(), starts, cache, table, lengths, window=window or None, sinks=sinks, scale=scale, out=out)
    torch.cuda.synchronize()
    assert tq.device_faults() == faults
    want, bound = int8.attend(wide(Q), *s.cache, s.starts, s.lengths, s.table, s.D ** -0.5 if scale is None else scale, window, sinks,
                              *bounds(s.dtype))
    got, rows = wide(got), slice(0, s.starts[-1])
    assert (got[s.starts[-1]:] == 7.0).all()
    err, allowed = np.abs(got[rows] - want[rows]), bound[rows] + HALF[s.dtype] * np.abs(want[rows]) + 1e-30
    assert np.isfinite(got).all()
    assert (err <= allowed).all(), ((err / allowed).max(), np.argwhere(err > allowed)[:4])
    return got


# ---- norm_rope ------------------------------------------------------------------

@pytest.mark.parametrize("n,Hq,Hk,D,pairs,axes,paired,weights,dtype", [
    (1, 32, 8, 128, 64, 1, False, BF16, BF16), (1, 1, 0, 128, 64, 1, False, None, F32), (37, 14, 2, 128, 32, 3, True, F32, F32),
    (300, 7, 7, 64, 32, 2, False, F32, BF16), (5, 3, 1, 256, 128, 1, True, BF16, BF16), (9, 5, 2, 96, 16, 4, False, F32, F32),
    (11, 2, 2, 8, 4, 1, False, F32, F32), (2000, 4, 1, 80, 40, 1, True, None, BF16), (3, 65, 9, 128, 60, 2, False, F32, F32),
    (700, 32, 8, 128, 64, 3, False, BF16, BF16), (4, 3, 2, 128, 4, 1, False, F32, F32)])
@pytest.mark.parametrize("joint", [False, True])
def test_norm_rope(tq, n, Hq, Hk, D, pairs, axes, paired, weights, dtype, joint):
    rng = np.random.default_rng(n + D)
    x = torch.from_numpy(rng.standard_normal((n, Hq + 2 * Hk, D)) * np.exp2(rng.uniform(-6, 6, (n, 1, 1)))).to(dtype).cuda()
    q, k = x[:, :Hq], x[:, Hq:Hq + Hk]
    if not joint:
        q, k = q.contiguous(), k.contiguous()
    k = k if Hk else None
    freq, axis = 10000.0 ** (-np.arange(pairs) / pairs), np.arange(pairs) * axes // pairs
    pos = rng.integers(-2 ** 31, 2 ** 31, (n, axes))
    pos[0], pos[n // 2:] = 0, rng.integers(0, 200000, (n - n // 2, axes))
    wq, wk = ((1 + 0.3 * torch.from_numpy(rng.standard_normal(D))).to(weights).cuda() if weights else None for _ in range(2))
    rotary = tq.Rotary(freq, "cuda", axis=axis, paired=paired)
    positions = dev(pos.astype(np.int32))
    got = tq.norm_rope(q, k, positions if axes > 1 else positions[:, 0].contiguous(), rotary, wq, wk, eps=1e-3)
    for y, g, w in ((q, got[0], wq), (k, got[1], wk)):
        if y is None:
            assert g is None
            continue
        want, of = int8.norm_rope(wide(y), None if w is None else wide(w), 1e-3, pos, freq, axis, paired)
        # the definition's own angle: 2^31 radians have a step of 2^-22 in 64 bits
        allowed = of * (26 * 2.0 ** -24 + 2.0 ** -53 * np.abs(pos).max(1).reshape(-1, 1, 1)) + HALF[dtype] * np.abs(want) + 1e-30
        err = np.abs(wide(g) - want)
        assert (err <= allowed).all(), (err / allowed).max()


def test_norm_rope_in_place_and_edges(tq):
    rotary = tq.Rotary(10000.0 ** (-np.arange(64) / 64), "cuda")
    q, k = torch.randn(50, 8, 128, device="cuda"), torch.randn(50, 2, 128, device="cuda")
    q[3], w = 0.0, torch.ones(128, device="cuda")
    q[4, 1, 7] = float("nan")
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    want = tq.norm_rope(q, k, pos, rotary, w, w)
    assert not want[0][3].any()
    assert want[0][4, 1].isnan().all() and want[0].isnan().sum() == 128      # a row's own NaN
    a, b = q.clone(), k.clone()
    got = tq.norm_rope(a, b, pos, rotary, w, w, out=(a, b))
    assert got[0] is a and torch.equal(a.nan_to_num(nan=9.0), want[0].nan_to_num(nan=9.0)) and torch.equal(b, want[1])
    none = tq.norm_rope(q[:0], k[:0], pos[:0], rotary, w, w)
    assert none[0].shape == (0, 8, 128) and none[1].shape == (0, 2, 128)
    # heads further apart than they are long, one row for all tokens
    far = torch.randn(50, 8, 192, device="cuda")[:, :, :128]
    same = torch.randn(1, 2, 128, device="cuda").expand(50, 2, 128)
    one, two = tq.norm_rope(far, same, pos, rotary, w, w), tq.norm_rope(far.contiguous(), same.contiguous(), pos, rotary, w, w)
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


# ---- append and read --------------------------------------------------------------

STEPS = [([1], [0]), ([1], [2048]), ([3, 0, 17, 1], [5, 9, 16, 31]), ([33] * 5, [0, 1, 15, 16, 200]), ([200], [7]), ([1] * 70, list(range(70))),
         ([0, 0, 5, 0], [3, 0, 40, 0])]


@pytest.mark.parametrize("counts,before", STEPS)
@pytest.mark.parametrize("H,D,page,dtype", [(2, 128, 16, BF16), (3, 64, 32, F32), (1, 128, 256, F32), (8, 64, 64, BF16)])
def test_append_and_read(tq, counts, before, H, D, page, dtype):
    s = Setup(counts, before, H, D, page, dtype, seed=len(counts) + D, spread=6, padding=3)
    cache, t, table, starts, lengths = s.device(tq)
    joint = torch.empty(s.n, 3 * H, D, dtype=dtype, device="cuda")
    joint[:, :H], joint[:, 2 * H:] = s.K.cuda(), s.V.cuda()
    for _ in range(2):                       # the second call finds its own rows: nothing changes
        tq.append_int8(joint[:, :H], joint[:, 2 * H:], starts, cache, table, lengths)
        s.append()
        for got, want, name in zip(t, s.cache, ("k", "v", "e")):
            assert np.array_equal(got.cpu().numpy(), want), name
    for kind in (F32, BF16):
        out = tuple(torch.full((s.n, H, D), 7.0, dtype=kind, device="cuda") for _ in range(2))
        tq.read_int8(cache, table, starts, lengths, s.n, kind, out=out)
        seq = np.repeat(np.arange(len(counts)), counts)
        slot = s.lengths[seq] + np.arange(len(seq)) - s.starts[seq]
        for of, x in enumerate(out):
            want = int8.values(s.cache[of], s.cache[2], of, s.table[seq, slot // page], slot % page)
            assert np.array_equal(wide(x)[:len(seq)], want) and (wide(x)[len(seq):] == 7.0).all()
    assert tq.device_faults() == 0


def test_codes_do_not_depend_on_the_steps(tq):
    """One prompt against token by token, with values that make the exponents grow all the time."""
    s = Setup([75], [0], H=2, D=128, page=32, dtype=F32, spread=0)
    s.K *= torch.exp2(torch.arange(75) * 0.7 - 20).view(-1, 1, 1).float()
    cache, t, table, starts, lengths = s.device(tq)
    tq.append_int8(s.K.cuda(), s.V.cuda(), starts, cache, table, lengths)
    s2 = Setup([75], [0], H=2, D=128, page=32, dtype=F32, spread=0)
    cache2, t2, table2, _, _ = s2.device(tq)
    for i in range(75):
        tq.append_int8(s.K[i:i + 1].cuda(), s.V[i:i + 1].cuda(), dev(np.array([0, 1], np.int32)), cache2, table2, dev(np.array([i], np.int32)))
    a = tq.read_int8(cache, table, starts, lengths, 75, F32)
    b = tq.read_int8(cache2, table2, starts, lengths, 75, F32)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_append_at_the_ends_of_the_range(tq, dtype):
    s = Setup([40, 20], [0, 8], H=2, D=64, page=16, dtype=dtype, spread=60)
    big, small = torch.finfo(dtype).max, torch.finfo(dtype).tiny
    s.K[3, 0, :4] = torch.tensor([big, -big, small, -small], dtype=dtype)
    s.K[17, 1, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), -small / 64], dtype=dtype)
    s.V[20:36] = 0.0
    s.V[37, 0] = float("nan")
    s.V[45, 1, 3] = small / 64
    cache, t, table, starts, lengths = s.device(tq)
    tq.append_int8(s.K.cuda(), s.V.cuda(), starts, cache, table, lengths)
    s.append()
    for got, want in zip(t, s.cache):
        assert np.array_equal(got.cpu().numpy(), want)
    got = tq.read_int8(cache, table, starts, lengths, s.n, dtype)
    assert all(x.isfinite().all() for x in got)


def test_append_and_read_out_of_range(tq):
    """Bad numbers write nothing and set the fault bit; the sequences beside them are served."""
    s = Setup([5, 6, 7, 8], [3, 10, 0, 20], H=2, D=128, page=16, dtype=BF16)
    before = [x.copy() for x in s.cache]
    for bad in ("page", "length", "beyond", "starts"):
        cache, t, table, starts, lengths = s.device(tq)
        table, lengths, starts = table.clone(), lengths.clone(), starts.clone()
        if bad == "page":
            table[1, 0] = s.cache[0].shape[0]
        elif bad == "length":
            lengths[1] = -1
        elif bad == "beyond":
            lengths[1] = s.table.shape[1] * 16 - 2 & -16
            lengths[1] += 16
        else:
            starts[4] = s.n + 1
        assert tq.device_faults() == 0
        tq.append_int8(s.K.cuda(), s.V.cuda(), starts, cache, table, lengths)
        assert tq.device_faults() == 32
        s.cache = tuple(x.copy() for x in before)
        lens, st = s.lengths.copy(), s.starts.copy()
        if bad == "starts":
            st[4] = st[3]
        tbl = s.table.copy()
        if bad != "starts":
            tbl[1] = -1                                 # absent for the definition
        if bad == "page":
            tbl[1, 1:] = s.table[1, 1:]
        int8.append(*s.cache, wide(s.K), wide(s.V), st, lens, tbl)
        for got, want in zip(t, s.cache):
            assert np.array_equal(got.cpu().numpy(), want), bad
        out = tuple(torch.full((s.n, 2, 128), 7.0, dtype=BF16, device="cuda") for _ in range(2))
        tq.read_int8(cache, table, starts, lengths, s.n, BF16, out=out)
        assert tq.device_faults() == 32
        if bad in ("page", "beyond"):
            first = 6 if bad == "page" else 0           # of sequence 1: slots 10 to 15 are on the absent page
            rows = slice(5, 5 + first) if bad == "page" else slice(5, 11)
            assert not out[0][rows].any() and out[0][11:].any()
        s.cache = before


# ---- attend -------------------------------------------------------------------------

@pytest.mark.parametrize("counts,before", [([1], [0]), ([1], [15]), ([1], [16]), ([1], [1020]), ([1] * 5, [0, 31, 32, 33, 400]),
                                           ([3, 0, 17, 1], [5, 9, 160, 31]), ([7], [300]), ([70], [65]), ([0, 2, 0], [4, 600, 0])])
@pytest.mark.parametrize("H,G,D,page,dtype", [(2, 4, 128, 16, BF16), (1, 1, 64, 64, F32), (2, 7, 64, 32, BF16), (1, 8, 128, 256, F32)])
def test_attend(tq, counts, before, H, G, D, page, dtype):
    s = Setup(counts, before, H, D, page, dtype, seed=len(counts) + D, padding=2)
    s.append()
    check_attend(tq, s, G)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 0), (100, 33), (5, 2 ** 31 - 1), (2 ** 31 - 1, 3), (511, 64)])
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_attend_window(tq, window, sinks, dtype, D):
    s = Setup([1, 6, 40, 2], [700, 90, 333, 0], 2, D, 16, dtype, seed=window % 97)
    s.append()
    check_attend(tq, s, 3, window=window, sinks=sinks)


def test_attend_reads_no_page_behind_the_window(tq):
    s = Setup([1, 4], [500, 300], 2, 128, 16, BF16)
    s.append()
    first = [500 - 63, 300 - 63]
    for b in range(2):
        s.table[b, 1:first[b] // 16] = -1 if b else 10 ** 6      # given back to the pool
    check_attend(tq, s, 4, window=64, sinks=5)


def test_attend_absent_pages(tq):
    """Slots on absent pages are not there; a token that sees none gives zeros."""
    s = Setup([1, 2, 3], [100, 20, 50], 2, 128, 16, BF16)
    s.append()
    s.table[0, 2], s.table[1, :], s.table[2, -1] = -5, s.cache[0].shape[0], -1
    got = check_attend(tq, s, 4, faults=32)
    assert not got[1:3].any() and got[0].any()


def test_attend_bad_numbers(tq):
    s = Setup([2, 3, 4], [30, 20, 50], 2, 128, 16, BF16)
    s.append()
    good = check_attend(tq, s, 4, Q=(Q := s.queries(4)))
    for bad in ("length", "beyond", "starts"):
        cache, _, table, starts, lengths = s.device(tq)
        if bad == "length":
            lengths[1] = -7
        elif bad == "beyond":
            lengths[1] = 2 ** 31 - 1
        else:
            starts[2] = 100
        out = torch.full(Q.shape, 7.0, dtype=BF16, device="cuda")
        tq.attend_int8(Q.cuda(), starts, cache, table, lengths, out=out)
        assert tq.device_faults() == 32
        out = wide(out)
        assert np.array_equal(out[:2], good[:2])
        if bad != "starts":
            assert np.array_equal(out[5:], good[5:]) and (out[2:5] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_large_and_small_values(tq, dtype):
    """Blocks of values 2^60 apart, where those with the weight are the small ones and the other way round; logits in the hundreds."""
    for flip in (False, True):
        s = Setup([2], [300], 2, 128, 16, dtype, spread=0)
        cache = s.cache
        up = np.arange(cache[2].shape[0]) % 3 == 0
        s.append()
        cache[2][up, :, :, 1] += 60 if flip else -50
        check_attend(tq, s, 4, size=20.0)


def test_attend_scale_and_nan_queries(tq):
    s = Setup([3, 2], [40, 70], 2, 128, 32, F32)
    s.append()
    for scale in (0.0, -0.3, 1.5):
        check_attend(tq, s, 2, scale=scale)
    Q = s.queries(2)
    good = check_attend(tq, s, 2, Q=Q)
    Q[1, 3, 5], Q[4, 0, 2], Q[2, 1] = float("nan"), float("inf"), 0.0
    cache, _, table, starts, lengths = s.device(tq)
    out = wide(tq.attend_int8(Q.cuda(), starts, cache, table, lengths))
    hit = np.zeros(out.shape[:2], bool)
    hit[1, 3] = hit[4, 0] = True
    assert np.isnan(out[hit]).all()
    hit[2, 1] = True
    assert np.array_equal(out[~hit], good[~hit])


# ---- together ---------------------------------------------------------------------------

def test_a_layer_step_by_step(tq):
    """Prompts of two sequences, then drafted tokens of which some are rejected, then single tokens: what a server runs."""
    H, G, D, page = 2, 4, 128, 16
    rng = np.random.default_rng(11)
    B, M = 3, 12
    table = rng.permutation(B * M + 1)[:B * M].reshape(B, M).astype(np.int32)
    host = (rng.integers(0, 256, (B * M + 1, H, page, D), dtype=np.uint8), rng.integers(0, 256, (B * M + 1, H, page, D), dtype=np.uint8),
            rng.integers(-128, 128, (B * M + 1, H, page // 16, 2), dtype=np.int8))
    cache = tq.Int8Cache(*(dev(x) for x in host))
    freq = 10000.0 ** (-np.arange(64) / 64)
    rotary, w = tq.Rotary(freq, "cuda"), torch.full((D,), 1.25, device="cuda", dtype=BF16)
    lengths = np.zeros(B, np.int32)
    for counts, accepted in (([70, 0, 33], None), ([4, 50, 4], [2, 50, 1]), ([1, 1, 1], None), ([5, 5, 5], [5, 1, 3]), ([1, 0, 1], None)):
        starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        n = int(starts[-1])
        x = torch.from_numpy(rng.standard_normal((n, H * G + 2 * H, D))).to(BF16).cuda()
        seq = np.repeat(np.arange(B), counts)
        pos = (lengths[seq] + np.arange(n) - starts[seq]).astype(np.int32)
        q, k = tq.norm_rope(x[:, :H * G], x[:, H * G:H * G + H], dev(pos), rotary, w, w)
        d = dev(starts), dev(lengths)
        tq.append_int8(k, x[:, H * G + H:], d[0], cache, dev(table), d[1])
        out = tq.attend_int8(q, d[0], cache, dev(table), d[1], window=64, sinks=2)
        int8.append(*host, wide(k), wide(x[:, H * G + H:]), starts, lengths, table)
        want, bound = int8.attend(wide(q), *host, starts, lengths, table, D ** -0.5, 64, 2, *bounds(BF16))
        assert (np.abs(wide(out) - want) <= bound + HALF[BF16] * np.abs(want)).all()
        roped, of = int8.norm_rope(wide(x[:, :H * G]), wide(w), 1e-6, pos[:, None], freq, np.zeros(64, int), False)
        assert (np.abs(wide(q) - roped) <= of * 26 * 2.0 ** -24 + HALF[BF16] * np.abs(roped)).all()
        lengths = (lengths + (counts if accepted is None else accepted)).astype(np.int32)
    for got, want in zip((cache.k_codes, cache.v_codes, cache.exponents), host):
        assert np.array_equal(got.cpu().numpy(), want)
    assert tq.device_faults() == 0
