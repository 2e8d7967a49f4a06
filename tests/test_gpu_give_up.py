"""Waits that are given up: what is still in flight is waited for."""
import pytest

import gqa_attention_cu_gb300 as pva

pytestmark = pytest.mark.gpu


def test_what_is_in_flight_is_waited_for_after_a_given_up_wait():
    """The call fails where the second wait (for an arrival 0.2 ms later) returns early."""
    assert pva.pva_selftest_wait(1000) == pva.DEV_FLAGS["wait_timeout"]
