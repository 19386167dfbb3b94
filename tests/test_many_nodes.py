"""Attention calls of more than 65,535 query positions, which a grid's second and third extents do not hold."""
import ctypes
import math

import pytest
import torch

from compressed_sparse_attention_hca_b200 import csa

INVALID = 1
P = ctypes.c_void_p
A = P(4096)  # aligned and non-null; never dereferenced by these calls


def _tree(B, T, H, dim, q_dt, kv_dt, ws_bytes, opt=None, E=4000):
    return csa.load().csa_tree_mqa(A, q_dt, A, E, None, 0, A, 16, A, None, 0, None, A, A, None, 16, 4, A, 1.0, B, T, H,
                                   dim, kv_dt, A, A, ws_bytes, ctypes.byref(opt) if opt else None, None)


def test_query_options_are_supported_for_many_nodes():
    """The tensor-core kernel has no such limit, so neither have its options: the call gets as far as its workspace."""
    norm = csa.MqaOptions(splits=2, q_rope_dims=64, rope_base=1e4)
    assert _tree(70000, 2, 64, 512, csa.BF16, csa.BF16, 0, norm) == INVALID
    assert "workspace" in csa.load().csa_last_error().decode()


@pytest.mark.parametrize("B,T,H", [(1 << 20, 1 << 11, 1), (1 << 27, 1, 128)])
def test_more_than_a_grid_holds_is_refused(B, T, H):
    assert _tree(B, T, H, 64, csa.F32, csa.F32, 1 << 62, E=8) == INVALID
    assert "query positions" in csa.load().csa_last_error().decode()
    st = csa.load().hca_dense_mqa(A, csa.F32, A, 8, A, 16, A, A, 16, 4, A, 1.0, B, T, H, 64, csa.F32, A, A, 1 << 62,
                                  None)
    assert st == INVALID and "query positions" in csa.load().csa_last_error().decode()


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need a CUDA device")


@pytest.mark.gpu
@pytest.mark.parametrize("splits", [0, 2])
@pytest.mark.parametrize("B,T", [(1, 65537), (32770, 2)])
def test_f32_nodes(B, T, splits):
    """Every node against the definition, tree call and dense call."""
    _need_gpu()
    g = torch.Generator(device="cuda").manual_seed(1)
    H, dim, E, Wn = 2, 64, 9, 40
    Q = torch.randn(B, T, H, dim, generator=g, device="cuda")
    ent = torch.randn(B, E, dim, generator=g, device="cuda")
    win = torch.randn(B, Wn, dim, generator=g, device="cuda")
    sink = torch.randn(H, generator=g, device="cuda")
    start = torch.zeros(B, dtype=torch.int64, device="cuda")
    pos = torch.randint(0, Wn, (B, T), generator=g, device="cuda")
    scale = 1 / math.sqrt(dim)
    opt = csa.mqa_options(splits=splits) if splits else None
    ctx = start + Wn
    out = csa.tree_mqa(Q, ent, win, start, None, None, ctx, pos, Wn, 4, sink, scale, options=opt)
    dense = csa.hca_dense_mqa(Q, ent, win, start, pos, Wn, 4, sink, scale, options=opt)
    torch.cuda.synchronize()
    tok = torch.arange(Wn, device="cuda")

    def want(vis):
        rows = torch.cat([ent, win], 1).double()
        z = torch.einsum("bthd,brd->bthr", Q.double(), rows) * scale
        keep = torch.cat([torch.arange(E, device="cuda") < vis[..., None], tok <= pos[..., None]], -1)
        z = torch.cat([z.masked_fill(~keep[:, :, None], -math.inf), sink.double()[:, None].expand(B, T, H, 1)], -1)
        return torch.einsum("bthr,brd->bthd", torch.softmax(z, -1)[..., :-1], rows)
    for got, w in ((out, want((ctx // 4).clamp(max=E)[:, None].expand(B, T))), (dense, want(((pos + 1) // 4).clamp(max=E)))):
        # fp32: sums over 64 dims (logits of up to ~40) and 49 rows
        assert float((got.double() - w).abs().max()) <= 2e-5


@pytest.mark.gpu
def test_tensor_core_nodes_with_a_turned_query():
    """65,600 nodes with the query's rotation: those of request 0's bytes, over and over."""
    _need_gpu()
    g = torch.Generator(device="cuda").manual_seed(2)
    B, T, H = 16400, 4, 64
    q = torch.randn(1, T, H, 512, generator=g, device="cuda").bfloat16()
    ent = torch.randn(1, 20, 512, generator=g, device="cuda").bfloat16()
    sink = torch.zeros(H, device="cuda")

    def run(n):
        zero = torch.zeros(n, dtype=torch.int64, device="cuda")
        pos = (80 + torch.arange(T, device="cuda")).expand(n, T).contiguous()
        return csa.tree_mqa(q.expand(n, T, H, 512).contiguous(), ent.expand(n, 20, 512).contiguous(),
                            ent[:, :1].expand(n, 1, 512).contiguous(), zero, None, None, zero + 80, pos, 0, 4, sink,
                            0.04, options=csa.mqa_options(splits=1, q_rope_dims=64))
    one, many = run(1), run(B)
    torch.cuda.synchronize()
    csa.check_device_status()
    assert bool((many == one).all())
