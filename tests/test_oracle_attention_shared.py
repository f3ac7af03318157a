"""Pins of the shared-prefix and scored attention oracle (CPU)."""

import numpy as np
import pytest
import torch

import oracle
from oracle import attention_shared as osh


def _case(seed=0, B=2, Hq=4, Hkv=2, D=8, Lmax=9, lens=(9, 4), Ls=6):
    rng = np.random.default_rng(seed)
    parent = [-1, 0, 0, 1, 1, 3]
    tree = oracle.tree_encode(parent, None)
    T = len(parent)
    n = rng.standard_normal
    return dict(q=n((B, Hq, T, D)), k_cache=n((B, Hkv, Lmax, D)), v_cache=n((B, Hkv, Lmax, D)), prefix_len=np.array(lens),
                k_tree=n((B, Hkv, T, D)), v_tree=n((B, Hkv, T, D)), tree=tree), n((Hkv, Ls, D)), n((Hkv, Ls, D))


def test_nothing_special_is_tree_attention():
    c, _, _ = _case()
    r = osh.attention(**c)
    f32 = {k: np.asarray(v, dtype=np.float32) if k[0] in "qkv" else v for k, v in c.items()}
    O, lse = oracle.tree_attention(f32["q"], f32["k_cache"], f32["v_cache"], c["prefix_len"], f32["k_tree"], f32["v_tree"],
                                   c["tree"], "f32")
    np.testing.assert_allclose(r["out"], O, atol=1e-5)
    np.testing.assert_allclose(r["lse"], lse, atol=1e-5)


@pytest.mark.parametrize("kw", [{}, {"softcap": 2.0}, {"window": 5}, {"window": 8, "slopes": np.array([1, .5, .1, -.2])}])
def test_a_shared_prefix_is_the_same_keys_in_every_cache(kw):
    c, ks, vs = _case()
    shared = osh.attention(**c, k_shared=ks, v_shared=vs, **kw)
    B = c["q"].shape[0]
    rep = lambda s, x: np.concatenate([np.broadcast_to(s, (B,) + s.shape), x], axis=2)  # noqa: E731
    plain = osh.attention(**{**c, "k_cache": rep(ks, c["k_cache"]), "v_cache": rep(vs, c["v_cache"]),
                             "prefix_len": c["prefix_len"] + ks.shape[1]}, **kw)
    for k in ("out", "lse"):
        np.testing.assert_allclose(shared[k], plain[k], atol=1e-12)


def test_capped_biased_windowed_scores_against_sdpa():
    """torch's attention given the whole additive mask; the cap through scores that are tanh by construction."""
    c, _, _ = _case(B=1, lens=(7,))
    slopes = np.array([0.5, 0.25, 0.1, 0.0])
    r = osh.attention(**c, window=6, slopes=slopes)
    n, depth = 7, np.asarray(c["tree"]["depth"])
    far = (n + depth)[:, None] - np.concatenate([np.arange(n), n + depth])[None]
    hidden = np.concatenate([np.zeros((6, n), dtype=bool), oracle.tree_mask(c["tree"]) != 0], 1) | (far >= 6)
    for h in range(4):
        K = np.concatenate([c["k_cache"][0, h // 2, :n], c["k_tree"][0, h // 2]])
        V = np.concatenate([c["v_cache"][0, h // 2, :n], c["v_tree"][0, h // 2]])
        mask = torch.tensor(np.where(hidden, -np.inf, -slopes[h] * far))
        o = torch.nn.functional.scaled_dot_product_attention(torch.tensor(c["q"][0, h]), torch.tensor(K), torch.tensor(V), mask)
        np.testing.assert_allclose(r["out"][0, h], o.numpy(), atol=1e-12)


def test_the_cap_binds_and_a_wide_cap_does_not():
    c, _, _ = _case()
    plain = osh.attention(**c)
    wide = osh.attention(**c, softcap=1e6)
    np.testing.assert_allclose(wide["out"], plain["out"], atol=1e-9)
    big = {**c, "q": c["q"] * 1e4}     # every score at +-cap: a softmax over signs
    r = osh.attention(**big, softcap=1.0)
    b, h, i = 0, 0, 0
    K = np.concatenate([c["k_cache"][b, 0, :9], c["k_tree"][b, 0, :1]])
    V = np.concatenate([c["v_cache"][b, 0, :9], c["v_tree"][b, 0, :1]])
    w = np.exp(np.sign(K @ c["q"][b, h, i]))
    np.testing.assert_allclose(r["out"][b, h, i], w @ V / w.sum(), atol=1e-9)


def test_a_window_of_one_sees_the_node_itself():
    c, ks, vs = _case()
    r = osh.attention(**c, k_shared=ks, v_shared=vs, window=1)
    np.testing.assert_allclose(r["out"], np.repeat(c["v_tree"], 2, axis=1), atol=1e-12)
