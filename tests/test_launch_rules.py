"""The host's choice between a product's forms (no GPU needed)."""
import pytest

from tests import launch_rules

SMS = 152


def share(m, n, k, e, swiglu=False):
    return launch_rules.gemv_share(swiglu, m, n, k, e, SMS)


@pytest.mark.parametrize("chunks", range(1, 29))
@pytest.mark.parametrize("swiglu", [False, True])
def test_warps_of_a_unit_fall_as_the_units_grow(chunks, swiglu):
    """Eight warps to a unit are for few units: no length of k has a range of its own in which they come back."""
    taken = [share(e, 1024, 256 * chunks, e, swiglu) for e in range(1, 129)]  # 32 units an expert
    assert taken == sorted(taken, reverse=True) and taken[0] == 8
    assert all(s == 8 for s in taken[:9]) and all(s in (2, 4) for s in taken[9:])  # from two units an SM on


def test_the_products_bits_are_compared_between_all_forms():
    from tests.test_gpu_gemv_forms import EXPERTS, N, shares

    for swiglu in (False, True):
        assert shares(1856, swiglu, SMS) == {8, 4}
        assert shares(512, swiglu, SMS) == {8, 2}
        assert shares(1536, swiglu, SMS) == shares(2368, swiglu, SMS) == {8, 4, 2}
        assert share(2 * EXPERTS, N, 7168, EXPERTS, swiglu) == 4
