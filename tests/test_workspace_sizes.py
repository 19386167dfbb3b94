"""Workspace sizes of absurd shapes: 256 bytes, as for every shape that the call refuses (CPU only)."""
from compressed_sparse_attention_hca_b200 import csa


def test_sizes_whose_product_overflows():
    n = 1 << 30
    assert csa.tree_mqa_workspace_size(n, n, 128, 64, 100, csa.F32, csa.F32) == 256
    assert csa.mqa_workspace_size(n, n, 128, 64, 100, csa.F32, csa.F32) == 256
    assert csa.mqa_workspace_size(n, n, 128, 512, 100, csa.BF16, csa.BF16) == 256
