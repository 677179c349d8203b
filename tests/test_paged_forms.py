"""The plain and the 64-bit forms of perf/operators.py against the float64 definitions of
oracle.paged, on the CPU at a few slots: the three say the same."""
import importlib.util
import os

import numpy as np
import pytest

import oracle
from oracle import paged
from conftest import ROOT, codebook

torch = pytest.importorskip("torch")

D = 128


@pytest.fixture(scope="module")
def forms():
    spec = importlib.util.spec_from_file_location("paged_forms", os.path.join(ROOT, "perf", "operators.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def state(op, B, H, S, page, kb, vb, seed, lengths=None):
    rng = np.random.default_rng(seed)
    M = -(-S // page)
    N = B * M + 2
    lengths = np.full(B, S) if lengths is None else np.asarray(lengths)
    s = dict(op=op, table=rng.permutation(N)[:B * M].reshape(B, M).astype(np.int32), lengths=lengths.astype(np.int32),
             kp=rng.integers(0, 256, (N, H, page, 16 * kb), dtype=np.uint8), vp=rng.integers(0, 256, (N, H, page, 16 * vb), dtype=np.uint8),
             kn=rng.uniform(0.5, 3, (N, H, page)).astype(np.float16), vn=rng.uniform(0.5, 3, (N, H, page)).astype(np.float16),
             kcb=codebook(D, kb)[0].astype(np.float32), vcb=codebook(D, vb)[0].astype(np.float32),
             Pk=np.stack([oracle.haar_rotation(rng.standard_normal((D, D))) for _ in range(H)]).astype(np.float32),
             Pv=np.stack([oracle.haar_rotation(rng.standard_normal((D, D))) for _ in range(H)]).astype(np.float32))
    for b, n in enumerate(lengths):
        s["table"][b, -(-int(n) // page):] = -1
    return s, rng


def tensors(s):
    return {k: torch.from_numpy(v.copy()) if isinstance(v, np.ndarray) else v for k, v in s.items()}


def exact(forms, monkeypatch, s, case):
    monkeypatch.setattr(forms, "prepare", lambda case, seed: tensors(s))
    return forms.exact(case, 0)


@pytest.mark.parametrize("S,budget,recent", [(32, 4, 8), (40, 13, 13), (40, 13, 40), (33, 33, 50), (50, 20, 7), (7, 3, 0), (24, 30, 2), (1, 1, 5)])
@pytest.mark.parametrize("ties", [False, True])
def test_evict(forms, monkeypatch, S, budget, recent, ties):
    """Windows of protected tokens shorter than the budget, as long and longer."""
    B, H, page = 2, 2, 16
    s, rng = state("evict", B, H, S, page, 2, 3, S + recent)
    mass = rng.integers(0, 4, (B, H, S)).astype(np.float32) if ties else np.exp(rng.standard_normal((B, H, S))).astype(np.float32)
    pos = np.stack([rng.permutation(S) for _ in range(B * H)]).reshape(B, H, S).astype(np.int32)
    s.update(mass=mass, positions=pos, seen=np.full(B, S, np.int32), budget=budget, recent=recent,
             mass_out=np.full((B, H, S), -3, np.float32), positions_out=np.full((B, H, S), -7, np.int32))
    plain = forms.run(tensors(s))
    want = {k: s[k].copy() for k in ("kp", "kn", "vp", "vn", "mass_out", "positions_out")}
    for (b, h), (kept, to, fro) in paged.evict_paged(mass, pos, s["lengths"], s["seen"], budget, recent).items():
        t = s["table"][b]
        for x in ("kp", "kn", "vp", "vn"):
            want[x][t[to // page], h, to % page] = want[x][t[fro // page], h, fro % page]
        for x, y in (("mass", "mass_out"), ("positions", "positions_out")):
            row = s[x][b, h].copy()
            row[to] = row[fro]
            want[y][b, h, :kept.size] = row[:kept.size]
    for k, v in want.items():
        assert np.array_equal(plain[k].numpy(), v), k
    got = exact(forms, monkeypatch, s, dict(op="evict", B=B, H=H, length=S, budget=budget, recent=recent, page=page))
    keep = min(S, budget)
    assert np.array_equal(got["mass_out"][..., :keep], want["mass_out"][..., :keep].astype(np.float64))
    assert np.array_equal(got["kn"], want["kn"].astype(np.float64)) and np.array_equal(got["vn"], want["vn"].astype(np.float64))


def test_evict_order_of_protected_slots():
    """32 tokens in order, the newest 8 protected, room for 4: the heaviest of the 8."""
    mass = np.zeros((1, 1, 32), np.float32)
    mass[0, 0, :24] = 9.0
    mass[0, 0, 24:] = [1, 2, 5, 6, 4, 2, 3, 0]
    pos = np.arange(32).reshape(1, 1, 32)
    kept, to, fro = paged.evict_paged(mass, pos, [32], [32], 4, 8)[0, 0]
    assert kept.tolist() == [26, 27, 28, 30] and to.tolist() == [0, 1, 2, 3] and fro.tolist() == kept.tolist()


@pytest.mark.parametrize("kb,vb,G", [(2, 4, 1), (3, 3, 4), (4, 2, 3)])
def test_decode(forms, monkeypatch, kb, vb, G):
    """fp32: 128 products and 45 slots, each sum off by less than 2^-17 of its terms."""
    B, H, S = 3, 2, 45
    s, rng = state("decode", B, H, S, 16, kb, vb, 10 * kb + G, [45, 17, 0])
    s.update(Q=rng.standard_normal((B, H * G, D)).astype(np.float32), mass=rng.random((B, H, S)).astype(np.float32))
    plain = forms.run(tensors(s))
    out, w, bound, wrel = paged.decode_paged(s["Q"], s["kp"], s["kn"], s["vp"], s["vn"], s["table"], s["lengths"], s["Pk"], s["kcb"],
                                             s["Pv"], s["vcb"], D ** -0.5, 2.0 ** -17, 2.0 ** -17)
    mass = s["mass"] + w.sum(2)[..., :S]
    assert (np.abs(plain["out"].numpy() - out) <= bound + 1e-5 * (1 + np.abs(out))).all()
    add = (w * (wrel[..., None] + 2.0 ** -17)).sum(2)[..., :S]
    assert (np.abs(plain["mass"].numpy() - mass) <= add + 2.0 ** -23 * mass).all()
    got = exact(forms, monkeypatch, s, dict(op="decode", B=B, H=H, G=G, length=S, page=16, kb=kb, vb=vb))
    assert np.abs(got["out"].numpy() - out).max() < 1e-12 and np.abs(got["mass"].numpy() - mass).max() < 1e-12


@pytest.mark.parametrize("kb,vb", [(2, 4), (3, 3), (4, 2)])
def test_append(forms, monkeypatch, kb, vb):
    B, H, n, page = 2, 2, 19, 16
    s, rng = state("append", B, H, n, page, kb, vb, kb)
    K, V = (rng.standard_normal((B * n, H, D)).astype(np.float32) for _ in range(2))
    rows = np.stack([np.repeat(np.arange(B), n), np.tile(np.arange(n), B), np.tile(np.arange(n), B) + 7], 1).astype(np.int32)
    s.update(K=K, V=V, rows=rows, mass=rng.random((B, H, n)).astype(np.float32), positions=np.full((B, H, n), -1, np.int32))
    plain = forms.run(tensors(s))
    got = exact(forms, monkeypatch, s, dict(op="append", B=B, H=H, tokens=n, page=page, kb=kb, vb=vb))
    assert not plain["mass"].any() and not got["mass"].any()
    for x, plane, norm, Pi, cb, bits in ((K, "kp", "kn", s["Pk"], s["kcb"], kb), (V, "vp", "vn", s["Pv"], s["vcb"], vb)):
        planes, norms = paged.append_rows(x, Pi, cb, bits)
        gap = paged.border_gap(x, Pi, cb)
        for i, (b, slot, at) in enumerate(rows):
            pg, r = s["table"][b, slot // page], slot % page
            differ = oracle.unpack_indices(plain[plane].numpy()[pg, :, r], bits, D) != oracle.unpack_indices(planes[i], bits, D)
            assert not (differ & (gap[i] > 1e-13)).any()
            step = np.spacing(norms[i]).astype(np.float64)     # fp32 on the way to fp16 may round a tie twice
            length = np.sqrt((x[i].astype(np.float64) ** 2).sum(-1))
            assert (np.abs(plain[norm].numpy()[pg, :, r] - norms[i].astype(np.float64)) <= step).all()
            assert np.abs(got[norm].numpy()[pg, :, r] - length).max() < 1e-12
            assert (plain["positions"].numpy()[b, :, slot] == at).all()
