"""Calls of the 8-bit cache that a server makes and that sizes or order could break: the first call of a process within a capture,
two streams at once, sequences by the ten thousand, caches beyond 2^31 bytes, many heads on one, graphs that share a workspace."""
import os
import subprocess
import sys

import numpy as np
import pytest

from conftest import ROOT
from oracle import int8
from test_gpu_int8 import BF16, F32, HALF, Setup, bounds, check_attend, dev, tq, wide  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

FIRST = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import numpy as np
import torch
from compressed_kv_cache_gb300 import tq
from test_gpu_int8 import Setup
s = Setup([{count}, 1], [50, 20], 2, 128, 16, torch.{dtype}, seed=1)
cache, t, table, starts, lengths = s.device(tq)
rotary = tq.Rotary(10000.0 ** (-np.arange(64) / 64), "cuda")
x, K, V = s.queries(4).cuda(), s.K.cuda(), s.V.cuda()
pos = torch.arange(s.n, dtype=torch.int32, device="cuda")
w = torch.ones(128, device="cuda")
def step():
    q, k = tq.norm_rope(x, K, pos, rotary, w, w)
    tq.append_int8(k, V, starts, cache, table, lengths)
    return (tq.attend_int8(q, starts, cache, table, lengths),) + tuple(tq.read_int8(cache, table, starts, lengths, s.n, K.dtype))
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    captured = step()
g.replay()
torch.cuda.synchronize()
for a, b in zip(captured, step()):
    assert torch.equal(a, b)
assert captured[0].isfinite().all() and captured[0].abs().max() > 0 and tq.device_faults() == 0
"""


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("count", [1, 40])
def test_first_call_in_a_capture(tq, dtype, count):
    code = FIRST.format(root=ROOT, tests=os.path.join(ROOT, "tests"), dtype=dtype, count=count)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("counts", [[1, 1, 1], [60, 3, 40]])
def test_two_streams_at_once(tq, counts):
    """Calls on two streams with workspaces of their own, over and over, give what one alone gives."""
    sets = []
    for seed in (1, 2):
        s = Setup(counts, [3000, 500, 70], 2, 128, 64, BF16, seed=seed)
        s.append()
        cache, _, table, starts, lengths = s.device(tq)
        Q = s.queries(4).cuda()
        sets.append((Q, starts, cache, table, lengths, torch.empty(tq.attend_int8_workspace_bytes(s.n, 3, 2, 4, 128), dtype=torch.uint8, device="cuda")))
    alone = [tq.attend_int8(*a[:5], workspace=a[5]) for a in sets]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in sets], [[], []]
    for _ in range(10):
        for i, (st, a) in enumerate(zip(streams, sets)):
            with torch.cuda.stream(st):
                outs[i].append(tq.attend_int8(*a[:5], workspace=a[5]))
    torch.cuda.synchronize()
    for got, want in zip(outs, alone):
        assert all(torch.equal(g, want) for g in got)
    assert tq.device_faults() == 0


def test_graphs_that_share_a_workspace(tq):
    """Replayed one after the other, two graphs may have one workspace: nothing in it outlives a call."""
    made = []
    ws = torch.empty(max(tq.attend_int8_workspace_bytes(n, 2, 2, 4, 128) for n in (2, 80)), dtype=torch.uint8, device="cuda")
    for counts in ([1, 1], [40, 40]):
        s = Setup(counts, [2000, 100], 2, 128, 64, BF16, seed=counts[0])
        s.append()
        cache, _, table, starts, lengths = s.device(tq)
        Q = s.queries(4).cuda()
        want = tq.attend_int8(Q, starts, cache, table, lengths)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = tq.attend_int8(Q, starts, cache, table, lengths, workspace=ws)
        made.append((g, out, want, (Q, starts, cache, table, lengths)))
    for k in (0, 1, 1, 0, 1, 0):
        g, out, want, _ = made[k]
        out.zero_()
        ws.fill_(0x7f)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_65535_sequences(tq, dtype):
    """One token each on a page of its own: it attends to itself, so that the output is its value as stored."""
    B, D = 65535, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    cache = tq.Int8Cache(torch.zeros(B, 1, 16, D, dtype=torch.uint8, device="cuda"), torch.zeros(B, 1, 16, D, dtype=torch.uint8, device="cuda"),
                         torch.zeros(B, 1, 1, 2, dtype=torch.int8, device="cuda"))
    table = torch.randperm(B, generator=g, device="cuda").to(torch.int32).view(B, 1)
    starts, lengths = torch.arange(B + 1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    K, V = (torch.randn(B, 1, D, generator=g, device="cuda").to(dtype) for _ in range(2))
    tq.append_int8(K, V, starts, cache, table, lengths)
    k, v = tq.read_int8(cache, table, starts, lengths, B, dtype)
    step = torch.exp2(torch.floor(torch.log2(V.float().abs().amax(-1, keepdim=True))) - 6)
    assert ((v.float() - V.float()).abs() <= step / 2).all()
    out = tq.attend_int8(torch.randn(B, 3, D, generator=g, device="cuda").to(dtype), starts, cache, table, lengths)
    # weight 1 to 2^-11 or 2^-21, as the definitions' bounds have it
    slack = 2.0 ** -10 if dtype is BF16 else 2.0 ** -17
    assert ((out.float() - v.float()).abs() <= v.float().abs() * (slack + HALF[dtype])).all()
    assert tq.device_faults() == 0


def test_many_sequences_with_empty_ones(tq):
    counts = [0] * 700
    before = [0] * 700
    for i, (c, n) in {3: (1, 40), 127: (2, 0), 128: (1, 300), 400: (5, 17), 699: (1, 90)}.items():
        counts[i], before[i] = c, n
    s = Setup(counts, before, 2, 128, 16, BF16, seed=2)
    s.append()
    check_attend(tq, s, 4)


def test_cache_beyond_2_31_bytes(tq):
    """Rows on pages past the 2^31st byte of a plane, against the same rows at the front."""
    N, H, page, D = 9000, 8, 256, 128
    kc, vc = (torch.empty(N, H, page, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    assert kc.numel() > 2 ** 31
    cache = tq.Int8Cache(kc, vc, torch.empty(N, H, page // 16, 2, dtype=torch.int8, device="cuda"))
    g = torch.Generator(device="cuda").manual_seed(3)
    n = 600
    K, V = (torch.randn(n, H, D, generator=g, device="cuda").to(BF16) for _ in range(2))
    Q = torch.randn(n, H * 2, D, generator=g, device="cuda").to(BF16)
    starts, zero = torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    one, last = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    got = []
    for pages in ([0, 1, 2], [N - 1, N - 2, N - 3]):
        table = torch.tensor([pages], dtype=torch.int32, device="cuda")
        tq.append_int8(K, V, starts, cache, table, zero)
        got.append((*tq.read_int8(cache, table, starts, zero, n, BF16), tq.attend_int8(Q, starts, cache, table, zero),
                    tq.attend_int8(Q[:1], one, cache, table, last)))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert got[0][3].isfinite().all() and tq.device_faults() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_heads_on_one(tq, dtype):
    s = Setup([1, 2], [200, 33], 1, 64, 16, dtype, seed=6)
    s.append()
    check_attend(tq, s, 150)


def test_nothing_to_do(tq):
    s = Setup([0, 0], [5, 0], 2, 128, 16, BF16)
    cache, t, table, starts, lengths = s.device(tq)
    e = torch.empty(0, 2, 128, dtype=BF16, device="cuda")
    before = [x.clone() for x in t]
    tq.append_int8(e, e, starts, cache, table, lengths)
    assert tq.read_int8(cache, table, starts, lengths, 0)[0].shape == (0, 2, 128)
    assert tq.attend_int8(torch.empty(0, 8, 128, dtype=BF16, device="cuda"), starts, cache, table, lengths).shape == (0, 8, 128)
    # tokens there are, but of no sequence
    pad = torch.full((3, 2, 128), 7.0, dtype=BF16, device="cuda")
    tq.append_int8(pad, pad, starts, cache, table, lengths)
    out = tq.attend_int8(pad, starts, cache, table, lengths, out=pad.clone())
    assert (out == 7.0).all() and all(torch.equal(a, b) for a, b in zip(t, before)) and tq.device_faults() == 0


def test_binding_refusals(tq):
    s = Setup([2, 1], [5, 0], 2, 128, 16, BF16)
    cache, t, table, starts, lengths = s.device(tq)
    K, V, Q = s.K.cuda(), s.V.cuda(), s.queries(4).cuda()
    with pytest.raises(ValueError):
        tq.append_int8(K.transpose(0, 1), V, starts, cache, table, lengths)
    with pytest.raises(ValueError, match="heads"):
        tq.append_int8(torch.empty(3, 4, 128, dtype=BF16, device="cuda")[:, ::2], V, starts, cache, table, lengths)
    with pytest.raises(TypeError):
        tq.append_int8(K, V.float(), starts, cache, table, lengths)
    with pytest.raises(ValueError):
        tq.append_int8(K, V, starts[:2], cache, table, lengths)
    with pytest.raises(TypeError):
        tq.append_int8(K, V, starts.long(), cache, table, lengths)
    with pytest.raises(ValueError, match="heads"):
        tq.attend_int8(Q[:, :7], starts, cache, table, lengths)
    for kw in (dict(window=0), dict(window=-3), dict(sinks=-1), dict(window=2 ** 31)):
        with pytest.raises(ValueError):
            tq.attend_int8(Q, starts, cache, table, lengths, **kw)
    with pytest.raises(tq.TQError):
        tq.attend_int8(Q, starts, cache, table, lengths, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        tq.read_int8(cache, table, starts, lengths, 3, torch.float16)
    with pytest.raises(ValueError):
        tq.Int8Cache(t[0], t[1], t[2][:, :, :, :1])
    rotary = tq.Rotary([1.0] * 64, "cuda", axis=[0] * 32 + [1] * 32)
    pos = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="axes"):
        tq.norm_rope(Q, K, pos[:, 0].contiguous(), rotary)
    with pytest.raises(TypeError):
        tq.norm_rope(Q, K, pos, rotary, torch.ones(128, device="cuda"), torch.ones(128, device="cuda", dtype=BF16))
    with pytest.raises(ValueError):
        tq.norm_rope(Q, K, pos, rotary, out=(K, Q))
    joint = torch.zeros(3, 10, 128, dtype=BF16, device="cuda")
    with pytest.raises(tq.TQError):
        tq.norm_rope(joint[:, :8], joint[:, 8:], pos, rotary, out=(joint.view(-1)[:3 * 8 * 128].view(3, 8, 128), K))
    assert tq.device_faults() == 0
