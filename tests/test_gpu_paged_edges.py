"""GPU parity of the paged cache's operators where their order or their arithmetic is decided by
little: windows of protected tokens longer than the budget."""
import numpy as np
import pytest

from test_gpu_paged import D, Pages, dev, run_evict, some_positions, tq  # noqa: F401  (tq: the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


# ---- evict: more protected slots than are kept --------------------------------

def test_evict_window_by_hand(tq):
    """32 tokens in order, the newest 8 protected, room for 4: the heaviest of the 8."""
    p = Pages(tq, 1, 1, 32, 16, seed=1)
    mass = np.full((1, 1, 32), 9.0, np.float32)
    mass[0, 0, 24:] = [1, 2, 5, 6, 4, 2, 3, 0]
    pos = np.arange(32, dtype=np.int32).reshape(1, 1, 32)
    _, got = tq.evict_paged(p.cache, p.t, p.n, p.n, dev(mass), dev(pos), 4, 8)
    assert got[0, 0, :4].tolist() == [26, 27, 28, 30]


@pytest.mark.parametrize("S,budget,recent", [(40, 1, 40), (600, 100, 101), (600, 100, 99), (600, 100, 100), (600, 599, 600), (5000, 700, 3000),
                                             (70001, 300, 5000), (393300, 1000, 200000)])
def test_evict_windows(tq, S, budget, recent):
    """Windows as long as the budget, shorter and longer by one, and much longer; one CTA,
    clusters, keys in device memory; weights all different and in ties."""
    rng = np.random.default_rng(S + recent)
    B, lengths = (3, [S, S - 7, S // 2]) if S < 10000 else (1, [S])
    p = Pages(tq, B, 2 if B > 1 else 1, S, 16 if S < 10000 else 256, 2, 2, rot=1, seed=3, lengths=lengths)
    pos = some_positions(rng, B, p.H, S, lengths)
    for mass in (np.exp(2 * rng.standard_normal(pos.shape)), rng.integers(0, 3, pos.shape), -rng.random(pos.shape)):
        run_evict(tq, p, mass.astype(np.float32), pos, np.asarray(lengths, np.int32) + 5, budget, recent)
