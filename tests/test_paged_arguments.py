"""Numbers that the binding hands to the paged calls as C integers."""
import pytest
import torch

import gated_delta_rule_45_amd as kda


@pytest.mark.parametrize("window", [-1, 2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1, -(2 ** 32) + 7])
def test_windows_that_are_no_c_integer(window):
    """2^32 + 5 would arrive as 5."""
    q, pages = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16), torch.zeros(9, 2, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 5, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="window"):
        kda.paged_attention(q, pages, pages, table, lens, window=window)


def test_frequencies_under_another_default_device():
    """They are written by host code: in host memory, whatever torch.empty would take."""
    want, _ = kda.rope_frequencies(48)
    with torch.device("meta"):
        freq, amplitude = kda.rope_frequencies(48)
    assert freq.device.type == "cpu" and torch.equal(freq, want) and amplitude == 1.0
