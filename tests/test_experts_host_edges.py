"""The expert layer's host side at its edges, without a GPU."""
import pytest

from test_block_host import refused, z  # noqa: F401
from test_block_host_edges import accepted

F = 1 << 32


@pytest.mark.parametrize("block,limit,ends", [(-1, 100, F), (2, 100, F), (0, 0, F), (1, (1 << 22) + 1, F), (0, 100, 0),
                                              (1, 100, F + 2)])
def test_pair_timeout_arguments(z, block, limit, ends):  # noqa: F811
    refused(z, z.zero_selftest_pair_timeout, block, limit, ends, 0)


def test_pair_timeout_passes_the_checks(z):  # noqa: F811
    accepted(z, z.zero_selftest_pair_timeout, 0, 100, F, 0)
