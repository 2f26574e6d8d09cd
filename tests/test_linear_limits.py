"""Limits of the combine, refused before anything is enqueued."""
import pytest

from tests.test_linear import P, m, refused  # noqa: F401


@pytest.mark.parametrize("k", [(1 << 30) + 1, 2 ** 31 - 8, 2 ** 31 - 1])
@pytest.mark.parametrize("hidden", [1, 64])
def test_combine_of_more_routes_than_it_counts(m, k, hidden):  # noqa: F811
    """The route loop's next step would pass 2^31 and never reach k."""
    refused(m, m.MOE_ERR_UNSUPPORTED, lambda: m.moe_combine(P, 8, P * 2, P * 3, None, P * 5, 2, k, hidden, stream=0))
