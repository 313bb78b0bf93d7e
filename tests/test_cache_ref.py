"""The references of the cache operators against hand-worked cases (CPU)."""
import math

import torch

import cache_ref as R


def test_quantise_by_hand():
    x = torch.zeros((3, 64), dtype=torch.float64)
    x[0, :4] = torch.tensor([7.0, -7.0, 2.5, -3.5])      # scale 1: ties go to the even code
    x[1, 0] = 1e-41                                       # a scale that rounds to zero
    c, s, _ = R.quantise(x)
    assert s[0] == 1 and c[0, :5].tolist() == [15, 1, 10, 4, 8]
    assert s[2] == 0 and set(c[2].tolist()) == {8} and set(c[1].tolist()) == {8}
    assert R.values(R.pack(c), s)[0, :4].tolist() == [7, -7, 2, -4]


def test_rotation_is_undone():
    g = torch.Generator().manual_seed(1)
    for d in (64, 128, 256):
        signs = (torch.randint(0, 2, (d,), generator=g) * 2 - 1).float()
        h = R.walsh(d)
        assert torch.equal(h @ h, d * torch.eye(d, dtype=torch.float64))
        x = torch.randn((5, d), generator=g, dtype=torch.float64)
        y = R.rotate(x, signs)
        assert torch.allclose((y @ h) * signs.double() / d, x, atol=1e-12)
        assert torch.allclose(y @ y.T / d, x @ x.T, atol=1e-10)


def test_eviction_by_hand():
    w = [5.0, 1.0, float("nan"), 1.0, 3.0, 1.0, 0.0]
    assert R.evict_keep(w, 4, 1, 1, 7) == [0, 2, 4, 6]     # row 0 and 6 protected, then NaN, then 3
    assert R.evict_keep(w, 5, 0, 0, 7) == [0, 1, 2, 3, 4]  # ties: the lowest row
    assert R.evict_keep(w, 9, 1, 1, 3) == [0, 1, 2]
    pos = [0, 1, 2, 3, 4, 5, 6]
    assert R.evict_slots(w, pos, 7, 7, 7, 2, 1, 1) == ([3, 5], 7)   # ties: the highest row
    assert R.evict_slots(w, pos, 5, 7, 7, 3, 0, 0) == ([5, 6, 3], 7)
    assert R.evict_slots(w, pos, 0, 0, 7, 3, 0, 0) == ([0, 1, 2], 3)


def test_weights_sum_to_the_number_of_queries():
    g = torch.Generator().manual_seed(2)
    q, k = (torch.randn((1, 4, 37, 64), generator=g, dtype=torch.float64) for _ in range(2))
    s = q @ k.transpose(-1, -2) / 8
    s = s.masked_fill(torch.ones(37, 37).triu(1).bool(), -math.inf)
    w = R.key_weights(q, k, torch.logsumexp(s, -1), True, 1 / 8, 37)
    assert abs(float(w.sum()) - 4 * 37) < 1e-9
