"""mi_kv_copy_planes with a list as long as 32 bits allow."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_row_to_all_others(cuda_device):
    """The last rows of the list are in an item that ends where an int does."""
    import paged_kv_decode_25_gb300 as mi
    rows = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("no room for the lists")
    x = torch.zeros(rows, 1, dtype=torch.int32, device=cuda_device)
    x[0] = 0x12345678
    src = torch.zeros(rows - 1, dtype=torch.int32, device=cuda_device)
    dst = torch.arange(1, rows, dtype=torch.int32, device=cuda_device)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    mi.check(mi.mi_kv_copy_planes(mi.kv_planes([x]), src, dst, rows - 1, err))
    assert err.item() == 0
    for part in x.split(1 << 28):
        assert bool((part == 0x12345678).all())
    del x, src, dst
    torch.cuda.empty_cache()
