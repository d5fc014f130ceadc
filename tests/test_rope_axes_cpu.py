"""CPU: the axes of the pairs, in the forms in which a program may have them."""
import numpy as np
import pytest
import torch

from paged_kv_cache_312_gb300 import _binding

AXES = [0, 2, 1, 1, 0, 2, 2, 0] * 2
WANT = bytes(AXES)


@pytest.mark.parametrize("form", [
    list, tuple, bytes, bytearray, iter, np.array, torch.tensor,
    lambda a: np.array(a, dtype=np.int32), lambda a: np.array(a, dtype=np.uint8),
    lambda a: torch.tensor(a, dtype=torch.uint8)])
def test_any_sequence_of_whole_numbers(form):
    assert _binding._axis_bytes("pkv_rope", form(AXES), len(AXES)) == WANT


@pytest.mark.parametrize("bad", [
    AXES[:-1], AXES + [0], [], len(AXES), 0, np.array(AXES[:2]), np.array(AXES[:4], dtype=np.int32),
    np.array(AXES, dtype=np.float32), [0.0] * 16, [0, -1] * 8, [0, 256] * 8, ["0"] * 16, "0" * 16,
    [[0, 1]] * 16, torch.zeros(8, 2, dtype=torch.int64), torch.zeros(16, 2, dtype=torch.int64)])
def test_what_names_no_axis_for_each_pair_is_refused(bad):
    """Among them arrays whose memory, and numbers, that as bytes have the right length."""
    with pytest.raises(ValueError, match="pair_axis must name an axis for each of 16 pairs"):
        _binding._axis_bytes("pkv_rope", bad, 16)
