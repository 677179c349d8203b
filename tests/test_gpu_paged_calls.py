"""Calls of the paged cache that a server makes and that sizes or order could break: the first
call of a process within a capture, two streams at once, batches and heads by the thousand.
Tolerances are those of test_gpu_paged.py."""
import os
import subprocess
import sys

import numpy as np
import pytest

from conftest import ROOT
from oracle import paged
from test_gpu_paged import D, Pages, check_append, check_mass, check_out, dev, tq  # noqa: F401  (tq: the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

FIRST = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
from compressed_kv_cache_gb300 import tq
from test_gpu_paged import Pages, dev
p = Pages(tq, 2, 2, 100, 16, seed=1, lengths=[100, 70])
q = torch.randn(2, 8, 128, device="cuda").to(torch.{dtype})
K = torch.randn(2, 2, 128, device="cuda").to(torch.{dtype})
rows = torch.tensor([[0, 3, 3], [1, 40, 40]], dtype=torch.int32, device="cuda")
mass, pos = torch.rand(2, 2, 112, device="cuda"), torch.zeros(2, 2, 112, dtype=torch.int32, device="cuda")
planes = (p.cache.k_plane, p.cache.k_norm, p.cache.v_plane, p.cache.v_norm)
save, m0 = [x.clone() for x in planes], mass.clone()
def step():
    tq.append_paged(K, K, rows, p.cache, p.t, mass=mass, positions=pos)
    out = tq.decode_paged(q, p.cache, p.t, p.n, mass=mass)
    return (out,) + tuple(tq.evict_paged(p.cache, p.t, p.n, p.n, mass, pos, 50, 0))
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    captured = step()
g.replay()
torch.cuda.synchronize()
got = [x.clone() for x in captured + planes]
for x, y in zip(planes, save):
    x.copy_(y)
mass.copy_(m0)
eager = step()
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(got, eager + planes))
print("same")
"""


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_first_calls_of_a_process_are_captured(tq, dtype):
    code = FIRST.format(root=ROOT, tests=os.path.join(ROOT, "tests"), dtype=dtype)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_two_streams_at_once(tq):
    """Two caches, each on a stream of its own with workspaces of its own, against the same calls
    one after another."""
    sides = []
    for seed in (1, 2):
        p = Pages(tq, 3, 4, 3000, 64, seed=seed, lengths=[3000, 1700, 20])
        q, K = torch.randn(3, 16, D, device="cuda"), torch.randn(600, 4, D, device="cuda").bfloat16()
        rows = np.stack([np.arange(600) % 2, 1000 + np.arange(600), np.arange(600)], 1).astype(np.int32)
        mass, pos = torch.rand(3, 4, 3008, device="cuda"), torch.zeros(3, 4, 3008, dtype=torch.int32, device="cuda")
        planes = (p.cache.k_plane, p.cache.k_norm, p.cache.v_plane, p.cache.v_norm)
        sides.append((p, q if seed == 1 else q.bfloat16(), K, dev(rows), mass, pos, mass.clone(), planes, [x.clone() for x in planes]))

    def step(side):
        p, q, K, rows, mass, pos, m0, planes, save = side
        for x, y in zip(planes, save):
            x.copy_(y)
        mass.copy_(m0)
        tq.append_paged(K, K, rows, p.cache, p.t, mass=mass, positions=pos)
        out = tq.decode_paged(q, p.cache, p.t, p.n, mass=mass)
        m, ps = tq.evict_paged(p.cache, p.t, p.n, p.n, mass, pos, 900, 100)
        return [out, m, ps] + [x.clone() for x in planes]

    want = [step(s) for s in sides]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sides]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(10):
        for s, side in zip(streams, sides):
            with torch.cuda.stream(s):
                got.append(step(side))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(g, want[i % 2]))
    assert tq.device_faults() == 0


@pytest.mark.parametrize("kind", ["f32", "bf16", "mass"])
def test_most_sequences(tq, kind):
    """65535 sequences of 0 to 20 slots on shared pages."""
    B, H, G, S = 65535, 2, 2, 32
    rng = np.random.default_rng(3)
    p = Pages(tq, 1, H, 16 * 200, 16, seed=4)
    pool = p.table[0]
    p.B, p.table, p.lengths = B, pool[rng.integers(0, pool.size, (B, 2))].astype(np.int32), rng.integers(0, 21, B).astype(np.int32)
    Q = rng.standard_normal((B, H * G, D)).astype(np.float32)
    q = dev(Q) if kind == "f32" else dev(Q).bfloat16()
    m = torch.zeros(B, H, S, device="cuda") if kind == "mass" else None
    out = tq.decode_paged(q, p.cache, dev(p.table), dev(p.lengths), mass=m)
    some = np.r_[0, B - 1, rng.integers(0, B, 300)]
    p.table, p.lengths = p.table[some], p.lengths[some]
    bf16 = kind != "f32"
    ke = 2.0 ** -11 + 2.0 ** -18 if kind == "bf16" else 2.0 ** -18
    want, w, bound, _ = p.want(q[some].float().cpu().numpy(), None, ke, 2.0 ** -11 if bf16 else 2.0 ** -18)
    check_out(out[some], want, bound, bf16)
    if m is not None:
        check_mass(m[some], np.zeros(1), w, p.want(q[some].float().cpu().numpy())[3])


def test_many_heads(tq):
    """5000 KV heads on three rotations: append, decode and evict of a few slots."""
    H, G, S = 5000, 1, 16
    p = Pages(tq, 1, H, S, 16, 2, 2, rot=3, seed=5, spare=0)
    rng = np.random.default_rng(6)
    K, V = (rng.standard_normal((3, H, D)).astype(np.float32) for _ in range(2))
    rows = np.array([[0, 2, 70], [0, 15, 71], [0, 4, 72]], np.int32)
    before = p.host()
    mass = torch.rand(1, H, S, device="cuda")
    pos = torch.zeros(1, H, S, dtype=torch.int32, device="cuda")
    tq.append_paged(dev(K), dev(V), dev(rows), p.cache, p.t, mass=mass, positions=pos)
    check_append(p, before, K.astype(np.float64), V.astype(np.float64), rows)
    p.kp, p.kn, p.vp, p.vn = p.host()
    q = torch.randn(1, H * G, D, device="cuda")
    want, _, bound, _ = p.want(q.cpu().numpy())
    check_out(tq.decode_paged(q, p.cache, p.t, p.n), want, bound, False)
    seen = torch.tensor([73], dtype=torch.int32, device="cuda")
    m0, p0 = mass.cpu().numpy(), pos.cpu().numpy()
    m, ps = tq.evict_paged(p.cache, p.t, p.n, seen, mass, pos, 5, 2)
    plan = paged.evict_paged(m0, p0, [S], [73], 5, 2)
    got, m = p.host(), m.cpu().numpy()
    for h in range(H):
        kept, to, fro = plan[0, h]
        row, x = m0[0, h].copy(), p.kp[0, h].copy()
        row[to], x[to] = row[fro], x[fro]
        assert np.array_equal(m[0, h, :5], row[:5]) and np.array_equal(got[0][0, h], x)
    assert tq.device_faults() == 0
