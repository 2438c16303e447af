"""What include/rg.h says of the paged cache's calls, without a GPU."""
import pytest

from quantized_weight_out_gb300 import binding as rg
from quantized_weight_out_gb300 import inputs
from test_kv_host import _attend, _batch, _cache, _store, lib  # noqa: F401  (lib: the fixture)


def test_the_range_message_is_for_every_call(lib):  # noqa: F811
    """RG_ERR_RANGE comes from the products and from the cache's calls."""
    text = rg.strerror(rg.RG_ERR_RANGE)
    for word in ("dY", "key", "value", "query"):
        assert word in text, text


def test_reserved_is_zero(lib):  # noqa: F811
    b = _batch()
    b.reserved = 1
    for call in (rg.rg_kv_write, rg.rg_kv_read):
        assert _store(call, _cache(), b) == rg.RG_ERR_ARG
    assert _attend(_cache(), b) == rg.RG_ERR_ARG
    assert rg.rg_kv_attend_workspace_bytes(_cache(), b, 32) == 0
    b.seqs = 0
    assert _attend(_cache(), b) == rg.RG_ERR_ARG  # an empty batch's description too
