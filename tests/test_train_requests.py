"""Which adapter each request of ``train_linear`` has (no GPU)."""
import pytest

from shared_memory_tiled_gb300.train_linear import adapter_of


@pytest.mark.parametrize("requests", [1, 8, 9, 20, 500])
def test_every_adapter_is_used(requests):
    index = adapter_of(requests, 8).tolist()
    assert len(index) == requests
    assert set(index) - {-1} == set(range(min(requests, 8)))
    assert index.count(-1) == requests // 9


def test_no_adapter_is_left_to_the_bare_requests():
    """Over many requests each adapter loses as many to the bare ones as another."""
    index = adapter_of(72 * 5, 8).tolist()
    assert {index.count(g) for g in range(8)} == {40}
