"""Numbers of a dropout's configuration that do not fit its fields are refused, not cut."""
import pytest


@pytest.fixture(scope="module")
def S():
    from mixed_precision_adam_grad_gb300 import build
    build.build()
    import mixed_precision_adam_grad_gb300 as S
    return S


@pytest.mark.parametrize("first", [1 << 63, 1 << 64, (1 << 64) + 5, -(1 << 63) - 1, -(1 << 64)])
def test_first_beyond_64_bits(S, first):
    with pytest.raises(ValueError, match="first"):
        S.dropout_config(0.1, 1, first=first)


def test_first_as_it_is(S):
    for first in (0, 5, 1 << 62):
        assert S.dropout_config(0.1, 1, first=first).first == first
