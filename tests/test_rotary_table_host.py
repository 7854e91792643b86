"""The rotary table on the CPU: its values and what it refuses."""
import pytest
import torch


@pytest.fixture(scope="module")
def ta():
    import tree_masked_speculative_gb300 as m
    return m


@pytest.mark.parametrize("positions,dim,base", [(1, 16, 10000.0), (40, 64, 500.0), (7, 2, 10000.0), (0, 32, 10.0)])
def test_values(ta, positions, dim, base):
    got = ta.rotary_table(positions, dim, base=base, device="cpu")
    assert got.shape == (positions, dim) and got.dtype == torch.float32
    for p in range(positions):
        for i in range(dim // 2):
            angle = torch.tensor(p * base ** (-2.0 * i / dim), dtype=torch.float64)
            # the nearest f32 of values that two ways of computing in 64 bits give: half a step, and their difference
            assert abs(got[p, i].double() - angle.cos()) <= 2.0 ** -24 + 1e-12
            assert abs(got[p, dim // 2 + i].double() - angle.sin()) <= 2.0 ** -24 + 1e-12


@pytest.mark.parametrize("dim", [15, 1, 129, 0, -2])
def test_odd_or_empty_dimensions_are_refused(ta, dim):
    """An odd count would give a wider table of other angles, which a call that turns 16 elements takes for its own."""
    with pytest.raises(ValueError, match="rotary_dim"):
        ta.rotary_table(10, dim, device="cpu")


@pytest.mark.parametrize("positions", [-1])
def test_negative_counts_are_refused(ta, positions):
    with pytest.raises(ValueError, match="positions"):
        ta.rotary_table(positions, 16, device="cpu")


@pytest.mark.parametrize("base", [0.0, -1.0, float("nan"), float("inf")])
def test_bases_that_give_no_angles_are_refused(ta, base):
    with pytest.raises(ValueError, match="base"):
        ta.rotary_table(10, 16, base=base, device="cpu")
