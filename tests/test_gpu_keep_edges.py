"""Calls of the beam and eviction operators that lie between the others' cases (GPU)."""

import numpy as np
import pytest

from gpu_util import lib
from oracle import beam, evict

pytestmark = pytest.mark.gpu


def _i32(a):
    import torch
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def test_a_workspace_of_the_largest_batch_serves_every_smaller_one():
    """Of exactly the size that the largest call asks for, with what lies behind it left alone; results are those with a workspace of
    the call's own."""
    import torch
    st = lib()
    W, K, V, Hq, Hkv, D, L, T, most = 4, 4, 32000, 8, 2, 64, 517, 100, 40
    g = torch.Generator().manual_seed(21)
    sizes = (st.beam_select_workspace_size(most, W, V, K), st.kv_weigh_workspace_size(most, Hq, Hkv, T, 0, L, D, 0),
             st.kv_evict_workspace_size(most, Hkv, L, 200))
    room = [torch.full((n + 4096,), 171, dtype=torch.uint8, device="cuda") for n in sizes]
    for B in (most, 37, 24, 18, 16, 8, 4, 2, 1):
        ws = [r[:n] for r, n in zip(room, sizes)]
        x, scores = torch.randn(B, W, V, generator=g).cuda(), -torch.rand(B, W, generator=g).cuda()
        got, want = st.beam_select(x, scores, K, ws=ws[0]), st.beam_select(x, scores, K)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), B
        k, q = torch.randn(B, Hkv, L, D, generator=g).cuda(), torch.randn(B, Hq, T, D, generator=g).cuda()
        lse, n = torch.full((B, Hq, T), 4.0, device="cuda"), _i32(np.linspace(T, L, B).astype(int))
        acc = [torch.ones(B, Hkv, L, device="cuda") for _ in range(2)]
        pos = _i32(np.tile(np.arange(L), (B, Hkv, 1)))
        for a, w in zip(acc, (ws[1], None)):
            st.kv_weigh(q, lse, k, n, a, ws=w)
        assert torch.equal(*acc), B
        v = k.flip(2).contiguous()
        two = [(k, v, acc[0], pos), tuple(t.clone() for t in (k, v, acc[0], pos))]
        for c, w in zip(two, (ws[2], None)):
            st.kv_evict(c[0], c[1], n, c[2], c[3], 200, ws=w)
        assert all(torch.equal(a, b) for a, b in zip(*two)), B
        assert [st.spec_read_device_status(w) for w in ws] == [0, 0, 0]
    for r, n in zip(room, sizes):
        assert (r[n:] == 171).all()
