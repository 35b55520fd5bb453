"""Edges of the language-model operators' C entries that need no GPU."""
import pytest

import sampling_threshold_filtering_amd as stf


@pytest.mark.parametrize("B", [0, 1, 61, 1 << 22, (1 << 31) - 1])
@pytest.mark.parametrize("V", [1, 50257, 1 << 17, 1 << 24])
def test_sampling_uses_no_scratch(B, V):
    assert stf.load_library().profk_sample_tokens_scratch(B, V) == 0
