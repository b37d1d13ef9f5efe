"""More refusals of the paged 8-bit cache, without a GPU (no call here launches)."""
import pytest

from test_cache_host import FAKE, INV, MIS, L, _attend  # noqa: F401 (L: the fixture)


@pytest.mark.parametrize("c,status", [(2.0 ** 127, INV), (2.5e38, INV), (3.4e38, INV), (1.7e38, MIS), (1e-45, MIS)])
def test_softmax_scales_whose_product_with_log2_e_is_no_float(L, c, status):  # noqa: F811
    # a workspace that the next check refuses
    assert _attend(L, c=c, work=FAKE + 128) == status
