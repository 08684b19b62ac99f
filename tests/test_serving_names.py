"""Names that are arguments of the serving operators (no GPU)."""
import pytest

from compressed_linear_amd import serving


def test_unknown_layout_is_a_value_error():
    assert serving.ROPE_LAYOUT["half"] == 0 and serving.ROPE_LAYOUT["interleaved"] == 1
    with pytest.raises(ValueError, match="'other' is none of .*half.*interleaved"):
        serving.ROPE_LAYOUT["other"]
    with pytest.raises(KeyError):  # as before
        serving.ROPE_LAYOUT["other"]
