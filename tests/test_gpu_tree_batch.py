"""csa_tree_mqa: the bytes of a request do not depend on the batch when the number of splits is fixed, and a call
repeated gives the same bytes."""
import math

import pytest
import torch

from compressed_sparse_attention_hca_b200 import csa
from compressed_sparse_attention_hca_b200 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need a CUDA device")
    csa.load()


def _batch(B, T, H, dim, kv, E, k, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rand(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device=DEV)
    x = dict(kv=kv, scale=1 / math.sqrt(dim), sink=torch.randn(H, generator=g, device=DEV))
    x["Q"] = torch.randn(B, T, H, dim, generator=g, device=DEV).to(torch.float32 if kv == csa.F32 else torch.bfloat16)
    x["entries"] = W.rows(g, kv, (B, E), dim, device=DEV)
    x["win"] = W.rows(g, kv, (B, 128), dim, device=DEV)
    x["draft"] = W.rows(g, kv, (B, T), dim, device=DEV)
    x["ctx"] = 4 * rand(E // 2, E, B) + rand(0, 4, B)
    x["win_start"] = x["ctx"] - 128
    x["q_pos"] = x["ctx"][:, None] + torch.arange(T, device=DEV)
    x["mask"] = ((2 << torch.arange(T, device=DEV)) - 1).to(torch.int32).expand(B, T)[..., None].contiguous()
    x["idx"] = rand(0, E // 2, B, T, k).to(torch.int32) if k else None
    return x


def _run(x, splits, rows=slice(None)):
    c = {n: v[rows].clone() if isinstance(v, torch.Tensor) and n != "sink" else v for n, v in x.items()}
    return csa.tree_mqa(c["Q"], c["entries"], c["win"], c["win_start"], c["draft"], c["mask"], c["ctx"], c["q_pos"], 128,
                        4, c["sink"], c["scale"], idx=c["idx"], kv_dt=c["kv"],
                        options=csa.mqa_options(splits=splits) if splits else None)


@pytest.mark.parametrize("splits", [1, 2, 5, 16, 17, 40])
@pytest.mark.parametrize("kv,H,dim,E,k,T", [
    (csa.BF16, 64, 512, 5200, 0, 3),
    (csa.KV_FP8MIX, 64, 512, 5200, 0, 3),
    (csa.BF16, 128, 512, 5200, 1900, 1),
    (csa.KV_FP8MIX, 128, 512, 5200, 1900, 2),
    (csa.F32, 8, 64, 900, 0, 3),
])
def test_fixed_splits_are_batch_invariant(kv, H, dim, E, k, T, splits):
    x = _batch(40, T, H, dim, kv, E, k, seed=splits)
    o40, o8 = _run(x, splits), _run(x, splits, slice(0, 8))
    assert torch.equal(o40[:8], o8)
    for b in (0, 3, 7):
        assert torch.equal(_run(x, splits, slice(b, b + 1))[0], o8[b]), f"request {b}"
    torch.cuda.synchronize()
    csa.check_device_status()


@pytest.mark.parametrize("splits", [0, 7])
@pytest.mark.parametrize("kv,H,dim,E,k,B", [(csa.BF16, 64, 512, 3000, 0, 5), (csa.KV_FP8MIX, 128, 512, 3000, 600, 5),
                                           (csa.BF16, 64, 512, 600, 0, 400), (csa.F32, 4, 64, 300, 16, 3)])
def test_repeated_calls_give_the_same_bytes(kv, H, dim, E, k, B, splits):
    x = _batch(B, 3, H, dim, kv, E, k, seed=1)
    first = _run(x, splits)
    for _ in range(20):
        assert torch.equal(_run(x, splits), first)
