"""A stream of another device than the logits' is refused, not passed over for the logits' device's own."""
import types

import pytest

from deterministic_token_logprob_gb300 import logits


def test_a_stream_of_another_device_is_refused():
    stream = types.SimpleNamespace(device_index=1, device="cuda:1")
    with pytest.raises(ValueError, match="stream"):
        with logits._elsewhere(stream, 0, ()):
            raise AssertionError("entered")
