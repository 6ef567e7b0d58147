"""kvq_attend_wait_limit without a GPU: it returns the limit before and keeps to its range."""
import pytest


@pytest.fixture(scope="module")
def kvq():
    from compress_kv_write_gb300 import build
    build.build()
    from compress_kv_write_gb300 import kvq
    kvq.lib()
    return kvq


def test_limit_is_set_and_returned(kvq):
    before = kvq.attend_wait_limit(7)
    try:
        assert before == 1 << 20
        assert kvq.attend_wait_limit(0) == 7
        assert kvq.attend_wait_limit((1 << 32) - 1) == 0
        assert kvq.attend_wait_limit(5) == 1 << 24          # bounded, so that a wait always ends
        for bad in (-1, 1 << 32):
            with pytest.raises(ValueError):
                kvq.attend_wait_limit(bad)
    finally:
        kvq.attend_wait_limit(before)
    assert kvq.attend_wait_limit(before) == before
