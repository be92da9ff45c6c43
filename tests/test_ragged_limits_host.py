"""Limits of a ragged step's calls that the library keeps without a GPU (fake addresses are never touched)."""
import pytest

FAKE = 0x100000


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import build
    build.build()
    from persistent_kv_cache_gb300 import kvc
    return kvc


def test_last_position_of_a_table(K):
    """Positions are 32-bit everywhere else: none past 2^31 - 1."""
    def f(first, positions, cos=FAKE):
        return K.library().kvc_rope_tables(cos, FAKE << 20, first, positions, 64, 1e4, 0, 0.0, 0, 0.0, 0.0, 1.0, None)
    assert f(2 ** 31 - 7, 8) == 2 and f(2 ** 31, 1) == 2 and f(2 ** 40, 8) == 2 and f(2, 2 ** 31 - 1) == 2
    # (as far as the addresses: the sizes are fine)
    assert f(2 ** 31 - 8, 8, None) == 1 and f(1, 2 ** 31 - 1, None) == 1 and f(2 ** 31, 0, None) == 0
