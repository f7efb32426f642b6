"""What the status that kernels record is called (CPU)."""
from dynamic_block_sparse_fractal_b200 import api


def test_the_device_status_names_both_of_its_causes():
    words = api.status_string(api.SA_ERR_DEVICE_TIMEOUT)
    assert "wait ran out" in words and "index out of range" in words
