"""Tree attention before anything is committed: a window that holds no rows."""
import ctypes
import math

import pytest
import torch

from compressed_sparse_attention_hca_b200 import csa

P = ctypes.c_void_p
A = P(4096)  # aligned and non-null; never dereferenced by this call


def test_no_rows_need_no_address():
    """The call gets as far as its workspace; window rows that are there need an address."""
    def call(win, win_len):
        st = csa.load().csa_tree_mqa(A, csa.BF16, A, 100000, None, 0, win, win_len, A, A, 4, A, A, A, None, 16, 4, A, 1.0,
                                     1, 2, 64, 512, csa.BF16, A, A, 0, None, None)
        assert st == 1
        return csa.load().csa_last_error().decode()
    assert "workspace" in call(None, 0)
    assert "win" in call(None, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("H,dim,dt", [(64, 512, torch.bfloat16), (4, 64, torch.float32)])
def test_first_tokens_of_a_request(H, dim, dt):
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need a CUDA device")
    g = torch.Generator(device="cuda").manual_seed(1)
    B, T = 2, 3
    Q = torch.randn(B, T, H, dim, generator=g, device="cuda").to(dt)
    draft = torch.randn(B, T, dim, generator=g, device="cuda").to(dt)
    sink = torch.randn(H, generator=g, device="cuda")
    zero = torch.zeros(B, dtype=torch.int64, device="cuda")
    mask = torch.tensor([1, 3, 7], dtype=torch.int32, device="cuda").expand(B, T)[..., None].contiguous()
    pos = torch.arange(T, device="cuda").expand(B, T).contiguous()
    empty = torch.empty(B, 0, dim, dtype=dt, device="cuda")
    out = csa.tree_mqa(Q, empty, empty, zero, draft, mask, zero, pos, 128, 4, sink, 1 / math.sqrt(dim))
    torch.cuda.synchronize()
    csa.check_device_status()
    z = torch.einsum("bthd,bjd->bthj", Q.double(), draft.double()) / math.sqrt(dim)
    z = z.masked_fill(~torch.tril(torch.ones(T, T, dtype=torch.bool, device="cuda"))[:, None], -math.inf)
    p = torch.softmax(torch.cat([z, sink.double()[:, None].expand(B, T, H, 1)], -1), -1)[..., :-1]
    want, A_ = torch.einsum("bthj,bjd->bthd", p, draft.double()), torch.einsum("bthj,bjd->bthd", p, draft.double().abs())
    # bf16: weights and output rounded once each; fp32: sums over dim and logits of up to ~40
    eps = 2 * 2.0 ** -8 + 2.0 ** -12 if dt == torch.bfloat16 else 2.0 ** -16
    assert bool(((out.double() - want).abs() <= eps * A_ + 1e-30).all())
