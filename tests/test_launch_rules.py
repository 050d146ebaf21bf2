"""The host's choice between a product's forms (no GPU needed)."""
import pytest

from tests import launch_rules

SMS = 152


def few(m, n, k, e):
    return launch_rules.few_halves(m, n, k, e, SMS)


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


@pytest.mark.parametrize("m,n,e", [(1, 4864, 1), (16, 4864, 1), (4, 1024, 4)])
def test_items_of_64_rows_whatever_the_k(m, n, e):
    """Items of 32 rows of W on more than half of the SMs pay from a k of 2560 on, items of 64 for every k."""
    for k in (64, 512, 1024, 2048, 2552):
        assert few(m, n, k, e) == 4
    for k in (2560, 4096, 7168):
        assert few(m, n, k, e) == 8
    for k in (64, 512, 1024, 2048, 2552, 2560, 4096, 7168):
        assert few(m, 2 * n, k, e) == 4  # each of 64 has an SM to itself, of 32 not


def test_the_forwards_few_rows_are_tested_in_all_forms():
    """The sizes of test_forward_of_few_rows_in_items_of_any_height."""
    taken = {few(m, n, k, e) for n in (40, 1000, 4096, 9000) for k in (64, 200, 520, 1400)
             for m, e in ((1, 1), (16, 1), (3, 5), (17, 1), (32, 2), (33, 1))}
    assert taken == {2, 4, 8}
