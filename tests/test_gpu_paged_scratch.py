"""The paged calls without a workspace or an output of the caller's, where the outputs are large enough (above 1 MB) to come from the
allocator's pool of large blocks, as the scratch does: they lie apart, and results are those of a call that is given both."""
import numpy as np
import pytest

from test_gpu_int8 import BF16, F32, Setup, check_attend, tq  # noqa: F401
from test_gpu_paged import Pages, dev, run_decode

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture
def launches(tq, monkeypatch):
    """(pointer of the output, of the scratch, bytes of the scratch) of each call."""
    seen, call = [], tq._paged_call

    def spy(name, index, *args):
        seen.append(args[-3:])
        return call(name, index, *args)
    monkeypatch.setattr(tq, "_paged_call", spy)
    return seen


@pytest.mark.parametrize("counts,dtype", [([1] * 600, BF16), ([700], BF16), ([130, 170], F32)])
def test_attend_int8(tq, launches, counts, dtype):
    s = Setup(counts, [50 + (3 * i) % 40 for i in range(len(counts))], 4, 128, 16, dtype, seed=len(counts))
    s.append()
    Q = s.queries(8)
    given = check_attend(tq, s, 8, Q=Q)
    cache, _, table, starts, lengths = s.device(tq)
    Q = Q.cuda()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()              # no free blocks of other calls that an output would fit
    launches.clear()
    got = tq.attend_int8(Q, starts, cache, table, lengths)
    out, scratch, size = launches[-1]
    assert out == got.data_ptr() and got.numel() * got.element_size() > 1 << 20
    assert out + got.numel() * got.element_size() <= scratch or scratch + size <= out
    assert np.array_equal(got.double().cpu().numpy(), given) and tq.device_faults() == 0


def test_decode_paged(tq, launches):
    p = Pages(tq, 600, 4, 64, 32, lengths=[20 + i % 40 for i in range(600)], seed=1)
    given, _ = run_decode(tq, p, 8, bf16=True, seed=2)
    Q = dev((np.random.default_rng(2).standard_normal((600, 32, 128))).astype(np.float32)).bfloat16()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    launches.clear()
    got = tq.decode_paged(Q, p.cache, p.t, p.n)
    out, scratch, size = launches[-1]
    assert out == got.data_ptr() and got.numel() * got.element_size() > 1 << 20
    assert out + got.numel() * got.element_size() <= scratch or scratch + size <= out
    assert torch.equal(got, given) and tq.device_faults() == 0
