"""The temperature's range on the CPU: what lies outside is refused, its ends are taken as far as the next check."""
import math

import pytest

from test_distillation_abi import _backward, _forward


@pytest.mark.parametrize("call", [_forward, _backward], ids=["forward", "backward"])
def test_temperatures(call):
    for T in (2.0 ** -60, 2.0 ** 60, 1.0):
        assert call(T=T, k=257) == 2          # (the temperature is right, the number of entries is not served)
    for T in (2.0 ** -61, math.nextafter(2.0 ** -60, 0) * (1 - 2.0 ** -23), 2.0 ** 60 * (1 + 2.0 ** -23), 2.0 ** 61, 3e38, -math.inf):
        assert call(T=T, k=257) == 1
