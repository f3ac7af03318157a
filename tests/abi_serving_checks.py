"""Host-side refusals of the serving calls (rotated appends, the tree's rotation, shared and scored tree attention):
each call below has one argument wrong and must fail its checks before anything is queued.  The device addresses
are invented and never dereferenced.  tests/test_abi_serving.py runs this file in a child process that sees no GPU."""

import ctypes
import os

import pytest

from conftest import ROOT  # noqa: F401  (puts the repository on sys.path)

EINVAL, EALIGN, EWORKSPACE, EUNSUPPORTED = 1, 3, 4, 5
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    assert os.environ.get("CUDA_VISIBLE_DEVICES") == "", "run through tests/test_abi_serving.py (no visible GPU)"
    import __graft_entry__
    __graft_entry__.build()
    from tree_speculative_decoding_spec_gb300 import _binding
    return _binding


def _tree(lib):
    """A root and two children: the host fields spec_tree_build would fill in, and invented addresses."""
    t = lib.spec_tree()
    t.T, t.words, t.max_depth, t.n_internal = 3, 1, 1, 1
    t.n_at_depth[0], t.n_at_depth[1], t.n_internal_at_depth[0] = 1, 2, 1
    for d in range(lib.SPEC_MAX_DEPTH + 1):
        t.max_rank_at_depth[d] = -1
    t.max_rank_at_depth[1] = 1
    for f in ["parent", "depth", "rank", "anc", "internal", "internal_off", "row_of", "child_off", "child_idx"]:
        setattr(t, f, 0x10000)
    return t


# Every buffer at an address of its own, 1 GB apart.
_GB = 1 << 30
_ATTN = {"q": 1 * _GB, "k_shared": 2 * _GB, "v_shared": 3 * _GB, "shared_len": 4 * _GB, "k_cache": 5 * _GB, "v_cache": 6 * _GB,
         "prefix_len": 7 * _GB, "k_tree": 8 * _GB, "v_tree": 9 * _GB, "out": 10 * _GB, "lse": 11 * _GB, "ws": 12 * _GB,
         "k_pool": 13 * _GB, "v_pool": 14 * _GB, "shared_table": 15 * _GB, "block_table": 16 * _GB, "slopes": 17 * _GB,
         "B": 2, "Hq": 4, "Hkv": 2, "D": 128, "Lshared": 64, "Lmax": 128, "num_blocks": 9, "shared_blocks": 4, "max_blocks": 8,
         "block_size": 16, "scale": 0.0, "dt": 1, "ws_bytes": 512 * MB, "softcap": 0.0, "window": 0, "tree": None}
_ORDER = {
    "tree_attention_shared": "q k_shared v_shared shared_len Lshared k_cache v_cache prefix_len k_tree v_tree tree B Hq Hkv Lmax D "
                             "scale score dt out lse ws ws_bytes",
    "tree_attention_shared_paged": "q k_pool v_pool num_blocks shared_table shared_blocks shared_len block_table max_blocks block_size "
                                   "prefix_len k_tree v_tree tree B Hq Hkv D scale score dt out lse ws ws_bytes",
    "tree_attention_scored": "q k_cache v_cache prefix_len k_tree v_tree tree B Hq Hkv Lmax D scale score dt out lse ws ws_bytes",
    "tree_attention_scored_paged": "q k_pool v_pool num_blocks block_table max_blocks block_size prefix_len k_tree v_tree tree B Hq "
                                   "Hkv D scale score dt out lse ws ws_bytes",
    "kv_append": "q k v q_stride k_stride v_stride N seq_start B Hq Hkv D prefix_len pos_base freq rot interleaved k_cache v_cache "
                 "Lmax dt q_out ws ws_bytes",
    "kv_append_paged": "q k v q_stride k_stride v_stride N seq_start B Hq Hkv D prefix_len pos_base freq rot interleaved k_pool v_pool "
                       "num_blocks block_table max_blocks block_size dt q_out ws ws_bytes",
    "tree_rope": "q k v q_stride k_stride v_stride tree B Hq Hkv D prefix_len pos_base freq rot interleaved dt q_out k_tree v_tree",
}


def _call(lib, name, base, **wrong):
    a = {**base, **wrong}
    tree = _tree(lib)
    if "tree" not in wrong:
        a["tree"] = ctypes.byref(tree)
    if "softcap" in a:
        a["score"] = ctypes.byref(lib.spec_score(a["softcap"], a["window"], wrong.get("slopes", 0)))
    return getattr(lib._lib, name)(*(a[n] for n in _ORDER[name].split()), None)


ATTENTION = [n for n in _ORDER if n.startswith("tree_attention")]


@pytest.mark.parametrize("name", ATTENTION)
def test_attention_refuses(lib, name):
    for wrong, code in [
        ({"tree": None}, EINVAL), ({"B": 0}, EINVAL), ({"B": 65536}, EINVAL), ({"Hkv": 0}, EINVAL), ({"Hq": 3}, EINVAL),
        ({"Hq": 1}, EINVAL), ({"Hq": 2048}, EINVAL), ({"D": 96}, EUNSUPPORTED), ({"D": 0}, EUNSUPPORTED), ({"dt": 2}, EINVAL),
        ({"q": 0}, EINVAL), ({"k_tree": 0}, EINVAL), ({"v_tree": 0}, EINVAL), ({"out": 0}, EINVAL), ({"prefix_len": 0}, EINVAL),
        ({"q": _GB + 8}, EALIGN), ({"k_tree": 8 * _GB + 4}, EALIGN), ({"out": 10 * _GB + 2}, EALIGN), ({"lse": 11 * _GB + 1}, EALIGN),
        ({"prefix_len": 7 * _GB + 2}, EALIGN), ({"slopes": 17 * _GB + 2}, EALIGN), ({"ws": 0}, EWORKSPACE),
        ({"ws_bytes": 512}, EWORKSPACE), ({"ws": 12 * _GB + 8}, EALIGN),
        ({"scale": -1.0}, EINVAL), ({"scale": float("nan")}, EINVAL), ({"scale": float("inf")}, EINVAL),
        ({"softcap": -1.0}, EINVAL), ({"softcap": float("nan")}, EINVAL), ({"softcap": 1e-7}, EINVAL), ({"softcap": 4097.0}, EINVAL), ({"softcap": float("inf")}, EINVAL),
        ({"window": -1}, EINVAL),
        ({"out": _GB}, EINVAL), ({"out": _GB + 16}, EINVAL), ({"out": 8 * _GB + 1024}, EINVAL), ({"out": 9 * _GB - 16}, EINVAL),
    ]:
        assert _call(lib, name, _ATTN, **wrong) == code, (wrong, lib.spec_last_error())
        assert lib.spec_last_error() != ""


def test_attention_refuses_its_own_arguments(lib):
    for name, wrong, code in [
        ("tree_attention_shared", {"k_shared": 0}, EINVAL), ("tree_attention_shared", {"shared_len": 0}, EINVAL),
        ("tree_attention_shared", {"Lshared": 0}, EINVAL), ("tree_attention_shared", {"Lshared": (1 << 22) + 1}, EINVAL),
        ("tree_attention_shared", {"v_shared": 3 * _GB + 8}, EALIGN), ("tree_attention_shared", {"shared_len": 4 * _GB + 2}, EALIGN),
        ("tree_attention_shared", {"k_cache": 0}, EINVAL), ("tree_attention_scored", {"Lmax": 0}, EINVAL),
        ("tree_attention_scored", {"Lmax": (1 << 22) + 1}, EINVAL), ("tree_attention_scored", {"v_cache": 6 * _GB + 4}, EALIGN),
        ("tree_attention_scored", {"B": 65535, "Lmax": 1 << 22}, EINVAL),
        ("tree_attention_shared_paged", {"shared_table": 0}, EINVAL), ("tree_attention_shared_paged", {"shared_blocks": 0}, EINVAL),
        ("tree_attention_shared_paged", {"shared_len": 0}, EINVAL), ("tree_attention_shared_paged", {"shared_table": 15 * _GB + 1}, EALIGN),
        ("tree_attention_shared_paged", {"shared_blocks": 1 << 20}, EINVAL),
    ] + [(n, w, c) for n in ATTENTION if n.endswith("paged") for w, c in [
        ({"block_size": 8}, EINVAL), ({"block_size": 24}, EINVAL), ({"block_size": 0}, EINVAL), ({"block_size": -16}, EINVAL),
        ({"num_blocks": 0}, EINVAL), ({"num_blocks": 1 << 30}, EINVAL), ({"max_blocks": 0}, EINVAL), ({"max_blocks": 1 << 20}, EINVAL),
        ({"block_table": 0}, EINVAL), ({"block_table": 16 * _GB + 2}, EALIGN), ({"k_pool": 0}, EINVAL), ({"v_pool": 14 * _GB + 8}, EALIGN)]]:
        assert _call(lib, name, _ATTN, **wrong) == code, (name, wrong, lib.spec_last_error())


def test_attention_workspaces(lib):
    t, L = _tree(lib), lib._lib
    shared = lambda *a: L.tree_attention_shared_workspace_size(ctypes.byref(t), *a)  # noqa: E731
    scored = lambda *a: L.tree_attention_scored_workspace_size(ctypes.byref(t), *a)  # noqa: E731
    assert shared(2, 4, 2, 64, 128, 128, 1) > scored(2, 4, 2, 128, 128, 1) > 0
    assert shared(2, 4, 2, 0, 128, 128, 1) == 0 and shared(2, 4, 2, 64, 0, 128, 1) == 0 and shared(2, 4, 3, 64, 128, 128, 1) == 0
    assert scored(0, 4, 2, 128, 128, 1) == 0 and scored(2, 4, 2, 128, 96, 1) == 0 and scored(2, 4, 2, 128, 128, 7) == 0


_ROPE = {"q": 1 * _GB, "k": 2 * _GB, "v": 3 * _GB, "q_stride": 512, "k_stride": 256, "v_stride": 256, "N": 6, "seq_start": 4 * _GB, "B": 2,
         "Hq": 4, "Hkv": 2, "D": 128, "prefix_len": 5 * _GB, "pos_base": 6 * _GB, "freq": 7 * _GB, "rot": 128, "interleaved": 0,
         "k_cache": 8 * _GB, "v_cache": 9 * _GB, "Lmax": 64, "dt": 1, "q_out": 10 * _GB, "ws": 11 * _GB, "ws_bytes": 256,
         "k_pool": 8 * _GB, "v_pool": 9 * _GB, "num_blocks": 9, "block_table": 12 * _GB, "max_blocks": 4, "block_size": 16,
         "k_tree": 13 * _GB, "v_tree": 14 * _GB, "tree": None}


@pytest.mark.parametrize("name", ["kv_append", "kv_append_paged", "tree_rope"])
def test_rotations_refuse(lib, name):
    for wrong, code in [
        ({"B": 0}, EINVAL), ({"B": 65536}, EINVAL), ({"Hkv": 0}, EINVAL), ({"Hq": 1025, "q_stride": 1 << 20}, EINVAL), ({"D": 0}, EINVAL),
        ({"D": 100}, EINVAL), ({"D": 1032, "q_stride": 1 << 20, "k_stride": 1 << 20, "v_stride": 1 << 20}, EINVAL), ({"dt": 3}, EINVAL),
        ({"k": 0}, EINVAL), ({"v": 0}, EINVAL), ({"prefix_len": 0}, EINVAL), ({"rot": 3}, EINVAL), ({"rot": -2}, EINVAL),
        ({"rot": 130}, EINVAL), ({"freq": 0}, EINVAL), ({"freq": 7 * _GB + 4}, EALIGN), ({"q_stride": 504}, EINVAL),
        ({"k_stride": 255}, EINVAL), ({"v_stride": 260}, EALIGN), ({"q": _GB + 8}, EALIGN), ({"v": 3 * _GB + 2}, EALIGN),
        ({"prefix_len": 5 * _GB + 2}, EALIGN), ({"pos_base": 6 * _GB + 1}, EALIGN), ({"q_out": 10 * _GB + 8}, EALIGN),
        ({"q_out": _GB}, EINVAL), ({"q_out": 2 * _GB + 512}, EINVAL), ({"q_out": 0}, EINVAL),
    ]:
        assert _call(lib, name, _ROPE, **wrong) == code, (wrong, lib.spec_last_error())
        assert lib.spec_last_error() != ""


def test_rotations_refuse_their_own_arguments(lib):
    both = [({"N": -1}, EINVAL), ({"N": (1 << 28) + 1}, EINVAL), ({"seq_start": 0}, EINVAL), ({"seq_start": 4 * _GB + 2}, EALIGN),
            ({"ws": 0}, EWORKSPACE), ({"ws_bytes": 16}, EWORKSPACE), ({"ws": 11 * _GB + 8}, EALIGN), ({"q": 0}, EINVAL)]
    for name, wrong, code in [(n, w, c) for n in ("kv_append", "kv_append_paged") for w, c in both] + [
        ("kv_append", {"Lmax": 0}, EINVAL), ("kv_append", {"Lmax": (1 << 22) + 1}, EINVAL), ("kv_append", {"k_cache": 0}, EINVAL),
        ("kv_append", {"v_cache": 9 * _GB + 8}, EALIGN),
        ("kv_append_paged", {"num_blocks": 0}, EINVAL), ("kv_append_paged", {"block_size": 0}, EINVAL),
        ("kv_append_paged", {"max_blocks": 1 << 20}, EINVAL), ("kv_append_paged", {"block_table": 0}, EINVAL),
        ("kv_append_paged", {"block_table": 12 * _GB + 1}, EALIGN), ("kv_append_paged", {"v_pool": 0}, EINVAL),
        ("tree_rope", {"tree": None}, EINVAL), ("tree_rope", {"q": 0}, EINVAL), ("tree_rope", {"k_tree": 0}, EINVAL),
        ("tree_rope", {"v_tree": 14 * _GB + 4}, EALIGN), ("tree_rope", {"v_tree": 3 * _GB + 64}, EINVAL),
    ]:
        assert _call(lib, name, _ROPE, **wrong) == code, (name, wrong, lib.spec_last_error())
