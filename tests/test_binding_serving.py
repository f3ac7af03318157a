"""What the binding of the serving calls checks before the library sees it (no GPU needed)."""

import pytest


@pytest.fixture(scope="module")
def binding():
    import __graft_entry__
    __graft_entry__.build()
    from tree_speculative_decoding_spec_gb300 import _binding
    return _binding


@pytest.mark.parametrize("window", [0, 1, 4096, 4096.0, (1 << 31) - 1, -1])
def test_whole_windows_reach_the_library_as_they_are(binding, window):
    score = binding._score(0.0, window, None)
    assert (score.window if score else 0) == window       # (what is negative is the library's to refuse)


@pytest.mark.parametrize("window", [1 << 31, 1 << 32, (1 << 32) + 5, -(1 << 32) + 5, 0.5, 2.5, float("inf"), float("nan")])
def test_windows_that_would_change_on_the_way_are_refused(binding, window):
    with pytest.raises(ValueError, match="window"):
        binding._score(0.0, window, None)
