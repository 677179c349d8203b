"""The scratch that the paged calls allocate where the caller gives none lives until the kernels are launched, so that nothing
else that the call allocates can lie in it.  Host only: the launch is a stand-in that looks at what is alive."""
import types
import weakref

import pytest

from compressed_kv_cache_gb300 import tq

torch = pytest.importorskip("torch")


@pytest.fixture
def call(monkeypatch):
    """Runs a call on CPU tensors; returns what it allocated as bytes, and the addresses alive at the launch."""
    made, seen = [], {}
    empty = torch.empty

    def allocate(*shape, device=None, **kw):
        t = empty(*shape, **kw)
        made.append((weakref.ref(t), t.data_ptr(), t.numel() * t.element_size(), kw.get("dtype")))
        return t

    def launch(name, index, *args):
        seen[name] = [(ref() is not None, at, size, dtype) for ref, at, size, dtype in made]
        seen["args"] = args

    monkeypatch.setattr(tq.torch, "empty", allocate)
    monkeypatch.setattr(tq, "_paged_call", launch)
    monkeypatch.setattr(tq, "_on", lambda index, t, name, dtype, shape: t.data_ptr())

    def run(name, f):
        f()
        scratch = [m for m in seen[name] if m[3] is torch.uint8]
        assert len(scratch) == 1
        return scratch[0], seen["args"]
    return run


def cache(H, D):
    return types.SimpleNamespace(_index=0, _ref=0, H=H, D=D, device="cpu")


def check(scratch, args):
    alive, at, size, _ = scratch
    assert size > 0 and args[-2:] == (at, size)
    assert alive, "the scratch has gone back to the allocator before the launch"


@pytest.mark.parametrize("n,B", [(1, 1), (300, 2)])
def test_attend_int8(call, n, B):
    table, ints = torch.zeros(B, 4, dtype=torch.int32), torch.zeros(B + 1, dtype=torch.int32)
    Q = torch.zeros(n, 8, 128, dtype=torch.bfloat16)
    check(*call("tq_attend_int8", lambda: tq.attend_int8(Q, ints, cache(2, 128), table, ints[:B])))


@pytest.mark.parametrize("mass", [False, True])
def test_decode_paged(call, mass):
    table, lengths = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    Q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    m = torch.zeros(2, 2, 64) if mass else None
    check(*call("tq_decode_paged", lambda: tq.decode_paged(Q, cache(2, 128), table, lengths, mass=m)))


def test_evict_paged(call):
    table, ints = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    mass, positions = torch.zeros(2, 2, 64), torch.zeros(2, 2, 64, dtype=torch.int32)
    check(*call("tq_evict_paged", lambda: tq.evict_paged(cache(2, 128), table, ints, ints, mass, positions, 32, 8)))
