"""Workspaces of the beam and eviction calls: one that was made for the largest call serves every smaller one (CPU; without a
device the sizes are those of 148 SMs)."""

import random

import pytest

F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def st():
    import __graft_entry__
    return __graft_entry__.build()


def _log(r, lo, hi):
    return min(hi, int(round(lo * (hi / lo) ** r.random())))


def test_selections(st):
    size = st.beam_select_workspace_size
    assert size(18, 8, 32000, 8) <= size(24, 8, 32000, 8) and size(4, 8, 32000, 8) <= size(24, 8, 32000, 8)
    r = random.Random(1)
    for _ in range(20000):
        large = (_log(r, 1, 2000), r.randint(1, 64), _log(r, 2, 1 << 24), r.randint(1, 64))
        small = tuple(r.choice([n, _log(r, min(n, 2 if i == 2 else 1), n)]) for i, n in enumerate(large))
        assert size(*small) <= size(*large), (small, large)
    # all slices there can be for few rows, some more than one for each row of many
    assert size(1, 1, 1 << 24, 64) >= 256 + 32 * (64 * 8 + 8) and size(60000, 64, 32000, 8) <= 256 + 1.01 * 60000 * 64 * (8 * 8 + 8)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_weights(st, dtype):
    size = st.kv_weigh_workspace_size
    assert size(4, 8, 2, 100, 0, 517, 64, dtype) <= size(16, 8, 2, 100, 0, 517, 64, dtype) <= size(32, 8, 2, 100, 0, 517, 64, dtype)
    r = random.Random(2)
    for _ in range(20000):
        Hkv = r.choice([1, 2, 8, 32])
        heads = (Hkv * r.choice([1, 4, 8, 71 if Hkv == 1 else 2]), Hkv)
        B, T, P, L = _log(r, 1, 2000), _log(r, 1, 1 << 14), r.choice([0, 0, r.randint(1, 17)]), _log(r, 1, 1 << 20)
        b, t, p, n = (r.choice([x, _log(r, 1, x)]) if x else 0 for x in (B, T, P, L))
        assert size(b, *heads, t, p, n, 64, dtype) <= size(B, *heads, T, P, L, 64, dtype), (heads, (B, T, P, L), (b, t, p, n))


def test_evictions_of_one_budget(st):
    r = random.Random(3)
    for _ in range(20000):
        B, H, L, budget = _log(r, 1, 2000), r.randint(1, 32), _log(r, 1, 1 << 22), _log(r, 1, 1 << 22)
        b, n = (r.choice([x, _log(r, 1, x)]) for x in (B, L))
        assert st.kv_evict_workspace_size(b, H, n, budget) <= st.kv_evict_workspace_size(B, H, L, budget), ((B, L), (b, n), H, budget)
