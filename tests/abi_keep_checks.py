"""Host-side refusals of the beam and eviction calls: each call below has one argument wrong and must fail its checks
before anything is queued.  The device addresses are invented and never dereferenced.  tests/test_abi_keep.py runs this
file in a child process that sees no GPU."""

import os

import pytest

from conftest import ROOT  # noqa: F401  (puts the repository on sys.path)

EINVAL, EALIGN, EWORKSPACE, EUNSUPPORTED = 1, 3, 4, 5
_GB = 1 << 30
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    assert os.environ.get("CUDA_VISIBLE_DEVICES") == "", "run through tests/test_abi_keep.py (no visible GPU)"
    import __graft_entry__
    __graft_entry__.build()
    from tree_speculative_decoding_spec_gb300 import _binding
    return _binding


_ORDER = {
    "beam_select": "logits row_stride scores ended length B W V K eos alpha dt token parent score ended_out length_out ws ws_bytes",
    "beam_reorder": "state row_bytes parent B W ws ws_bytes",
    "kv_reorder": "k_cache v_cache parent start end B W Hkv Lmax D dt ws ws_bytes",
    "kv_reorder_paged": "k_cache v_cache num_blocks block_table max_blocks block_size parent start end B W Hkv D dt ws ws_bytes",
    "kv_weigh": "q lse k_cache prefix_len seen n_rows accept_len accept_path path_len B Hq Hkv T Lmax D scale decay dt acc pos ws ws_bytes",
    "kv_weigh_paged": "q lse k_cache num_blocks block_table max_blocks block_size prefix_len seen n_rows accept_len accept_path path_len "
                      "B Hq Hkv T D scale decay dt acc pos ws ws_bytes",
    "kv_evict": "k_cache v_cache prefix_len seen acc pos B Hkv Lmax D budget sink recent k_out v_out acc_out pos_out Lout len_out dt ws "
                "ws_bytes",
    "kv_evict_paged": "k_cache v_cache num_blocks block_table max_blocks block_size prefix_len seen acc pos B Hkv D budget sink recent "
                      "out_table out_blocks acc_out pos_out len_out dt ws ws_bytes",
}
# Every buffer at an address of its own, 1 GB apart.
_NAMES = ["logits", "scores", "ended", "length", "token", "parent", "score", "ended_out", "length_out", "state", "k_cache", "v_cache",
          "start", "end", "block_table", "q", "lse", "prefix_len", "seen", "n_rows", "accept_len", "accept_path", "acc", "pos", "k_out",
          "v_out", "acc_out", "pos_out", "out_table", "len_out", "ws"]
_AT = {n: (i + 1) * _GB for i, n in enumerate(_NAMES)}
_BASE = {**_AT, "ws_bytes": 64 << 20, "B": 2, "W": 4, "V": 1000, "K": 4, "row_stride": 1024, "eos": 2, "alpha": 0.5, "dt": 1, "row_bytes": 64,
         "Hkv": 2, "Hq": 4, "T": 3, "Lmax": 64, "D": 128, "num_blocks": 9, "max_blocks": 4, "block_size": 16, "path_len": 0, "scale": 0.0,
         "decay": 1.0, "budget": 40, "sink": 4, "recent": 8, "Lout": 40, "out_blocks": 3}
_WEIGH = {**_BASE, "accept_len": 0, "accept_path": 0}
_PATH = {**_BASE, "n_rows": 0, "path_len": 5}


def _call(lib, name, base, **wrong):
    a = {**base, **wrong}
    return getattr(lib._lib, name)(*(a[n] for n in _ORDER[name].split()), None)


def _refuses(lib, name, base, cases):
    for wrong, code in cases:
        assert _call(lib, name, base, **wrong) == code, (name, wrong, lib.spec_last_error())
        assert lib.spec_last_error() != ""


WORKSPACE = [({"ws": 0}, EWORKSPACE), ({"ws_bytes": 128}, EWORKSPACE), ({"ws": _AT["ws"] + 8}, EALIGN)]


def test_selection_refuses(lib):
    _refuses(lib, "beam_select", _BASE, WORKSPACE + [
        ({"B": 0}, EINVAL), ({"B": 65536}, EINVAL), ({"W": 0}, EINVAL), ({"W": 65}, EINVAL), ({"K": 0}, EINVAL), ({"K": 65}, EINVAL),
        ({"V": 1}, EINVAL), ({"V": (1 << 24) + 1, "row_stride": 1 << 25}, EINVAL), ({"row_stride": 999}, EINVAL), ({"eos": -2}, EINVAL),
        ({"eos": 1000}, EINVAL), ({"eos": -1}, EINVAL), ({"alpha": -0.1}, EINVAL), ({"alpha": NAN}, EINVAL), ({"alpha": INF}, EINVAL),
        ({"alpha": 17.0}, EINVAL), ({"dt": 2}, EINVAL), ({"logits": 0}, EINVAL), ({"scores": 0}, EINVAL), ({"token": 0}, EINVAL),
        ({"parent": 0}, EINVAL), ({"score": 0}, EINVAL), ({"logits": _AT["logits"] + 8}, EALIGN), ({"scores": _AT["scores"] + 2}, EALIGN),
        ({"ended_out": _AT["ended_out"] + 1}, EALIGN), ({"token": _AT["logits"] + 64}, EINVAL), ({"token": _AT["scores"]}, EINVAL),
        ({"score": _AT["scores"] + 4}, EINVAL), ({"score": _AT["scores"], "K": 3}, EINVAL), ({"score": _AT["ended"]}, EINVAL),
        ({"ended_out": _AT["length"]}, EINVAL), ({"token": _AT["parent"] + 16}, EINVAL), ({"length_out": _AT["ended_out"]}, EINVAL)])


def test_reorders_refuse(lib):
    shared = WORKSPACE + [({"B": 0}, EINVAL), ({"B": 65536}, EINVAL), ({"W": 0}, EINVAL), ({"W": 65}, EINVAL), ({"parent": 0}, EINVAL),
                          ({"parent": _AT["parent"] + 2}, EALIGN)]
    _refuses(lib, "beam_reorder", _BASE, shared + [({"state": 0}, EINVAL), ({"state": _AT["state"] + 4}, EALIGN), ({"row_bytes": 0}, EINVAL),
                                                   ({"row_bytes": 6}, EINVAL), ({"row_bytes": -4}, EINVAL), ({"row_bytes": 1 << 33}, EINVAL)])
    caches = shared + [({"Hkv": 0}, EINVAL), ({"D": 0}, EINVAL), ({"D": 100}, EINVAL), ({"D": 1032}, EINVAL), ({"dt": 5}, EINVAL),
                       ({"k_cache": 0}, EINVAL), ({"v_cache": 0}, EINVAL), ({"v_cache": _AT["k_cache"]}, EINVAL), ({"v_cache": _AT["k_cache"] + 64}, EINVAL), ({"start": 0}, EINVAL),
                       ({"end": 0}, EINVAL), ({"start": _AT["start"] + 1}, EALIGN), ({"k_cache": _AT["k_cache"] + 8}, EALIGN)]
    _refuses(lib, "kv_reorder", _BASE, caches + [({"Lmax": 0}, EINVAL), ({"Lmax": (1 << 22) + 1}, EINVAL)])
    _refuses(lib, "kv_reorder_paged", _BASE, caches + PAGED)


PAGED = [({"num_blocks": 0}, EINVAL), ({"max_blocks": 0}, EINVAL), ({"block_size": 0}, EINVAL), ({"max_blocks": 1 << 20}, EINVAL),
         ({"block_table": 0}, EINVAL), ({"block_table": _AT["block_table"] + 2}, EALIGN)]


def test_weighing_refuses(lib):
    shared = WORKSPACE + [
        ({"B": 0}, EINVAL), ({"B": 65536}, EINVAL), ({"Hkv": 0}, EINVAL), ({"Hq": 3}, EINVAL), ({"Hq": 2048}, EINVAL), ({"T": 0}, EINVAL),
        ({"T": (1 << 22) + 1}, EINVAL), ({"D": 96}, EUNSUPPORTED), ({"dt": 2}, EINVAL), ({"scale": -1.0}, EINVAL), ({"scale": NAN}, EINVAL),
        ({"scale": INF}, EINVAL), ({"decay": -0.1}, EINVAL), ({"decay": 1.5}, EINVAL), ({"decay": NAN}, EINVAL), ({"q": 0}, EINVAL),
        ({"lse": 0}, EINVAL), ({"k_cache": 0}, EINVAL), ({"prefix_len": 0}, EINVAL), ({"acc": 0}, EINVAL), ({"q": _AT["q"] + 8}, EALIGN),
        ({"k_cache": _AT["k_cache"] + 4}, EALIGN), ({"lse": _AT["lse"] + 2}, EALIGN), ({"pos": _AT["pos"] + 1}, EALIGN),
        ({"acc": _AT["lse"]}, EINVAL), ({"acc": _AT["pos"] + 64}, EINVAL), ({"pos": _AT["k_cache"] + 64}, EINVAL),
        ({"acc": _AT["prefix_len"]}, EINVAL)]
    for name, more in (("kv_weigh", [({"Lmax": 0}, EINVAL), ({"Lmax": (1 << 22) + 1}, EINVAL)]),
                       ("kv_weigh_paged", PAGED + [({"block_size": 8}, EINVAL), ({"block_size": 24}, EINVAL)])):
        _refuses(lib, name, _WEIGH, shared + more + [({"accept_len": _AT["accept_len"]}, EINVAL), ({"accept_path": _AT["accept_path"]}, EINVAL)])
        _refuses(lib, name, _PATH, [({"path_len": 0}, EINVAL), ({"path_len": 18}, EINVAL), ({"path_len": -1}, EINVAL),
                                    ({"n_rows": _AT["n_rows"]}, EINVAL), ({"accept_len": 0}, EINVAL), ({"accept_path": 0}, EINVAL),
                                    ({"accept_path": _AT["accept_path"] + 2}, EALIGN)])


def test_eviction_refuses(lib):
    shared = WORKSPACE + [
        ({"B": 0}, EINVAL), ({"B": 65536}, EINVAL), ({"Hkv": 0}, EINVAL), ({"B": 60000}, EINVAL), ({"D": 0}, EINVAL), ({"D": 100}, EINVAL),
        ({"dt": 2}, EINVAL), ({"budget": 0}, EINVAL), ({"budget": -5}, EINVAL), ({"sink": -1}, EINVAL), ({"recent": -1}, EINVAL),
        ({"sink": 33}, EINVAL), ({"recent": 2147483647}, EINVAL), ({"k_cache": 0}, EINVAL), ({"v_cache": 0}, EINVAL), ({"acc": 0}, EINVAL),
        ({"pos": 0}, EINVAL), ({"prefix_len": 0}, EINVAL), ({"len_out": 0}, EINVAL), ({"len_out": _AT["prefix_len"]}, EINVAL),
        ({"len_out": _AT["seen"] + 4}, EINVAL), ({"k_cache": _AT["k_cache"] + 8}, EALIGN), ({"pos": _AT["pos"] + 2}, EALIGN)]
    into = shared + [({"acc_out": 0}, EINVAL), ({"pos_out": 0}, EINVAL), ({"acc_out": _AT["acc"]}, EINVAL), ({"pos_out": _AT["acc_out"] + 64}, EINVAL),
                     ({"acc_out": _AT["acc_out"] + 2}, EALIGN)]
    here = {"k_out": 0, "v_out": 0, "acc_out": 0, "pos_out": 0, "out_table": 0}
    sizes = [({"Lmax": 0}, EINVAL), ({"Lmax": (1 << 22) + 1}, EINVAL)]
    _refuses(lib, "kv_evict", {**_BASE, **here}, shared + sizes + [({"k_out": _AT["k_out"]}, EINVAL)])
    _refuses(lib, "kv_evict", _BASE, into + sizes + [
        ({"k_out": 0}, EINVAL), ({"v_out": 0}, EINVAL), ({"Lout": 39}, EINVAL), ({"Lout": 0}, EINVAL), ({"Lout": (1 << 22) + 1}, EINVAL),
        ({"k_out": _AT["k_cache"]}, EINVAL), ({"v_out": _AT["k_out"] + 1024}, EINVAL), ({"v_out": _AT["v_out"] + 4}, EALIGN)])
    _refuses(lib, "kv_evict_paged", {**_BASE, **here}, shared + PAGED + [({"out_table": _AT["out_table"]}, EINVAL)])
    _refuses(lib, "kv_evict_paged", _BASE, into + PAGED + [({"out_table": 0}, EINVAL), ({"out_blocks": 2}, EINVAL), ({"out_blocks": 0}, EINVAL),
                                                           ({"out_blocks": 1 << 20}, EINVAL), ({"out_table": _AT["out_table"] + 2}, EALIGN)])


def test_workspaces(lib):
    L = lib._lib
    assert L.beam_select_workspace_size(2, 4, 1000, 4) >= 256 + 8 * 8 * 4 and L.beam_reorder_workspace_size() == 256
    assert L.beam_select_workspace_size(1, 65, 1000, 4) == L.beam_select_workspace_size(0, 4, 1000, 4) == L.beam_select_workspace_size(1, 4, 1, 4) == 0
    assert L.kv_weigh_workspace_size(2, 4, 2, 3, 0, 64, 128, 1) >= 256
    assert L.kv_weigh_workspace_size(2, 4, 3, 3, 0, 64, 128, 1) == L.kv_weigh_workspace_size(2, 4, 2, 3, 18, 64, 128, 1) == 0
    assert L.kv_evict_workspace_size(2, 2, 64, 40) >= 256 + 4 * 24 * 8 and L.kv_evict_workspace_size(2, 2, 64, 64) > 0
    assert L.kv_evict_workspace_size(2, 2, 0, 40) == L.kv_evict_workspace_size(2, 2, 64, 0) == L.kv_evict_workspace_size(65535, 2, 64, 4) == 0
