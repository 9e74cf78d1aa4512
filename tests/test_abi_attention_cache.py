"""Host-checkable errors of the paged cache's entry points for pools and tables without
entries: what a kernel would read must be there (these calls touch no GPU)."""
import pytest

from gated_deltanet_linear_recurrence_gb300 import _lib
from gated_deltanet_linear_recurrence_gb300.build import build
from tests.test_abi_attention import NULL, paged, rows


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def test_a_table_with_entries_is_needed_for_an_empty_pool(lib):
    """The kernels look a position's page up before they compare it with the pool's size."""
    for name in ("gdn_kv_append", "gdn_kv_gather"):
        assert rows(lib, name, pages=0, kp=None, vp=None, ke=None, ve=None, table=None) == NULL, name
    assert paged(lib, pages=0, kp=None, vp=None, ke=None, ve=None, table=None) == NULL
