"""The attention calls' compression option where there is no query (a tree whose tokens were all rejected): the entry is
compressed all the same."""
import pytest
import torch

from compressed_sparse_attention_hca_b200 import csa
from compressed_sparse_attention_hca_b200 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call", ["tree", "dense"])
def test_compression_happens(call):
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need a CUDA device")
    B, E, m, dim, H = 2, 30, 128, 512, 64
    tok = W.compress_inputs(W.generator(3), B, m, dim, m, False, torch.bfloat16, c_std=1.0)
    t = {k: (v.to("cuda") if isinstance(v, torch.Tensor) else v) for k, v in tok.items()}
    out = [torch.zeros(B, E, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    jobs = [csa.compress_job(t["Ca"], t["Za"], t["Ba"], m, tok0=m * (E - 1), e0=E - 1, n_out=1, out=o, out_dt=csa.BF16)
            for o in out]
    csa.compress_ex(jobs[0], B)
    Q = torch.empty(B, 0, H, dim, dtype=torch.bfloat16, device="cuda")
    win = torch.zeros(B, 1, dim, dtype=torch.bfloat16, device="cuda")
    zero = torch.zeros(B, dtype=torch.int64, device="cuda")
    pos = torch.empty(B, 0, dtype=torch.int64, device="cuda")
    args = (128, m, torch.zeros(H, device="cuda"), 0.04)
    opt = csa.mqa_options(compress=jobs[1])
    O = (csa.tree_mqa(Q, out[1], win, zero, None, None, zero + m * E, pos, *args, options=opt) if call == "tree" else
         csa.hca_dense_mqa(Q, out[1], win, zero, pos, *args, options=opt))
    torch.cuda.synchronize()
    assert O.shape == Q.shape and bool(out[0][:, E - 1].any()) and torch.equal(out[0], out[1])
