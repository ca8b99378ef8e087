"""The temperature limits that the header states for the log-probability and
policy calls, checked on the host: inside them a call goes on to the checks
behind (a missing workspace), outside it is refused for its temperature."""
import math

import pytest

import draft_block_causal_amd as D

E_ARG, E_WS = -5, -6


@pytest.fixture(scope="module")
def lib():
    return D.load_library()


@pytest.mark.parametrize("T,good", [
    (math.nextafter(2e-38, 1), True), (3e-38, True), (1.0, True), (9.9e19, True), (math.nextafter(1e20, 0), True),
    (2e-38, False), (1.9e-38, False), (1e-38, False), (5e-39, False), (1e20, False), (1.2e20, False), (1.4e20, False),
    (float("inf"), False), (float("nan"), False), (0.0, False), (-1.0, False),
])
def test_temperature_limits(lib, T, good):
    want = E_WS if good else E_ARG
    assert lib.domino_token_logprobs(2, 3, 50, 0x100000, 0x20000, None, T, 0x30000, None, None, 0, None) == want
    assert lib.domino_policy_loss(2, 3, 50, 0x100000, 0x20000, 0x21000, None, 0x23000, None, T, 0.2, 0.2, 0.0, 0x30000,
                                  None, None, None, None, 0, None) == want
