"""Host-side checks of numbers that the descriptors of the calls around the paged cache cannot hold."""
import math

import pytest
import torch


@pytest.fixture(scope="module")
def ha():
    from long_context_sparse_score_gb300 import hashattn
    return hashattn


@pytest.mark.parametrize("window", [1 << 31, (1 << 32) + 5, 1 << 63, -(1 << 31) - 1])
def test_windows_past_32_bits(ha, window):
    with pytest.raises(ValueError, match="window"):
        ha.score_opts(window=window)


def test_windows_of_32_bits(ha):
    assert ha.score_opts(window=(1 << 31) - 1).window == (1 << 31) - 1


@pytest.mark.parametrize("name", ["scale", "softcap"])
@pytest.mark.parametrize("x", [1e-50, -1e-50, 5e-324])
def test_numbers_that_float32_makes_a_default(ha, name, x):
    with pytest.raises(ValueError, match="scale and softcap"):
        ha.score_opts(**{name: x})


def test_numbers_of_float32(ha):
    o = ha.score_opts(scale=2.0 ** -60, softcap=2.0 ** 60)
    assert (o.scale, o.softcap) == (2.0 ** -60, 2.0 ** 60)
    assert math.isinf(ha.score_opts(softcap=1e300).softcap)  # which the calls refuse
    assert (ha.score_opts().scale, ha.score_opts().softcap) == (0.0, 0.0)


@pytest.mark.parametrize("name", ["n_pages", "page_size", "total"])
def test_paging_past_32_bits(ha, name):
    table = torch.zeros(2, 3, dtype=torch.int32)
    good = dict(n_pages=5, page_size=16, total=7)
    assert ha.make_paging(table, **good).page_size == 16
    with pytest.raises(ValueError, match=name):
        ha.make_paging(table, **{**good, name: (1 << 32) + 16})
