"""csa_page_plan at the batch sizes whose sums just fit the shared memory that a kernel has without asking for more."""
import pytest
import torch

from compressed_sparse_attention_hca_b200 import csa

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("n_maps,batch", [(0, 4095), (0, 4090), (0, 3500), (1, 2456), (1, 2440), (2, 1754), (2, 1740),
                                          (2, 1600)])
def test_sums_near_48_kb(n_maps, batch):
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need a CUDA device")
    i32, i64 = dict(dtype=torch.int32, device=DEV), dict(dtype=torch.int64, device=DEV)
    after = torch.arange(batch, **i64) % 5 * 100
    table = torch.full((batch, 4), -1, **i32)
    free = torch.arange(4 * batch, **i32)
    count = torch.tensor([4 * batch], **i32)
    maps = [csa.slot_map(m, batch, 16) for m in (4, 128)[:n_maps]]
    info = csa.page_plan(torch.zeros_like(after), after, 128, table, free, count, maps=maps)
    torch.cuda.synchronize()
    held = (after + 127) // 128
    n = int(held.sum())
    assert info.tolist() == [n, 0, 0, 0] and int(count) == 4 * batch - n
    first = held.cumsum(0) - held
    j = torch.arange(4, device=DEV)
    want = torch.where(j < held[:, None], 4 * batch - 1 - first[:, None] - j, -1)
    assert torch.equal(table.long(), want)
    csa.check_device_status()
