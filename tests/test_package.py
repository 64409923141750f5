"""What the package re-exports of its binding (no GPU needed)."""
import pytest

import mla_paged_kv_03_b200 as package
from mla_paged_kv_03_b200 import binding as B


@pytest.mark.parametrize("name", [
    "mla_cache_append", "mla_shared_prefix_get_metadata", "mla_shared_prefix_decode_fwd",
    "mla_shared_prefix_workspace_size", "mla_page_keys_update", "mla_page_sparse_decode",
    "mla_page_sparse_workspace_size"])
def test_the_calls_around_the_cache_and_their_sizes(name):
    assert getattr(package, name) is getattr(B, name)


def test_other_names_are_not_there():
    with pytest.raises(AttributeError):
        package.mla_cache_prepend
