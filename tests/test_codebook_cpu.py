"""The levels that a QuantizedNF4 hands to the library are its own, bit for
bit (no GPU: the structure is filled, nothing is launched)."""
import numpy as np
import pytest
import torch


def weight(levels):
    import bit_nf4_quantized_20_b200 as q
    z = torch.zeros(4, dtype=torch.uint8)
    return q.QuantizedNF4(z, z, torch.zeros(1), 64, 64, levels)


def handed_over(levels):
    return bytes(weight(levels).struct().codebook)


@pytest.mark.parametrize("order", [(0.0, -0.0), (-0.0, 0.0)])
def test_the_sign_of_a_zero_level_is_its_own(order):
    """0.0 == -0.0: two weights whose levels differ in that alone, in either order."""
    for zero in order:
        levels = [-1.0 + i / 8 for i in range(16)]
        levels[8] = zero
        assert handed_over(levels) == np.array(levels, np.float32).tobytes()


@pytest.mark.parametrize("kind", [list, tuple, np.array, torch.tensor, lambda v: np.array(v, np.float32)])
def test_any_sequence_of_levels(kind):
    rng = np.random.default_rng(3)
    levels = np.sort(rng.uniform(-1, 1, 16)).tolist()
    assert handed_over(kind(levels)) == np.array(levels, np.float32).tobytes()


def test_a_changed_level_is_seen_by_the_next_call():
    levels = [i / 16 for i in range(16)]
    w = weight(levels)
    a = bytes(w.struct().codebook)
    w.codebook[3] = 0.5
    b = bytes(w.struct().codebook)
    levels[3] = 0.5
    assert a != b and b == np.array(levels, np.float32).tobytes()


def test_number_of_levels():
    """Fewer levels leave the rest zero, as they always have; more are refused."""
    assert handed_over([1.0, 2.0]) == np.array([1, 2] + [0] * 14, np.float32).tobytes()
    with pytest.raises((ValueError, IndexError)):
        weight([0.0] * 17).struct()
