"""What a refused call says fits every entry point."""

import os

import pytest

from ternary_weights_hadamard_amd import tb


@pytest.mark.skipif(not os.path.exists(tb.LIB_PATH), reason="libtb.so not built")
def test_refusals_name_what_all_calls_have():
    assert "stride" in tb.status_string(2) and "size" in tb.status_string(2)   # not of products alone
    assert "elements" in tb.status_string(3)                                  # not 16 bytes everywhere
    assert "VALUE" in tb.status_string(10) and "unknown" in tb.status_string(11)
