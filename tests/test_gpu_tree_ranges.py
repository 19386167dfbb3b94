"""csa_tree_mqa over rows of very different magnitudes, zeros among them.

Tolerance.  With A = sum_j p_j |v_j|: the weights and an FP8MIX row's scales, values and partials are rounded to 11 bits
(2^-11 each, four times), BF16 weights to 8 (2^-8), the output to 8 (2^-8); logits of FP8MIX rows take the row's two
roundings (d = scale sum |q k| 2^-10, and dim 2^-24 for the sums), and a logit off by d moves a weight by e^d, in
numerator and sum: 2 d.  FP8MIX weights are 2^(s + e - M) in fp16, e the row's exponent and M the largest s + e: a
weight below fp16's normal range is off by 2^-25 2^M, on a value below 2^16 2^e', so a row by 2^-24 of the largest
contribution there is, as that one has a value of at least 2^14.  BF16 rows have no such term.
"""
import math

import pytest
import torch

from compressed_sparse_attention_hca_b200 import csa
from compressed_sparse_attention_hca_b200 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"
DIM, H = 512, 64
N8 = DIM - 64


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need a CUDA device")
    csa.load()


def _f64(rows, kv):
    if kv != csa.KV_FP8MIX:
        return rows.double()
    codes = rows[..., :N8].contiguous().view(torch.float8_e4m3fn).double()
    tail = rows[..., N8:N8 + 128].contiguous().view(torch.bfloat16).double()
    sc = rows[..., N8 + 128:N8 + 156].contiguous().view(torch.float32).double()
    return torch.cat([codes * sc.repeat_interleave(64, -1), tail], -1)


def _rows(kv, groups, seed):
    """Rows in order: n of about N(0, size^2) for each (n, size)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = W.rows(g, kv, (sum(n for n, _ in groups),), DIM, device=DEV)
    size = torch.cat([torch.full((n,), float(s), dtype=torch.float64) for n, s in groups]).to(DEV)[:, None]
    if kv == csa.KV_FP8MIX:
        for lo, hi, t in ((N8, N8 + 128, torch.bfloat16), (N8 + 128, N8 + 156, torch.float32)):
            part = x[:, lo:hi].contiguous().view(t)
            x[:, lo:hi] = (part.double() * size).to(t).contiguous().view(torch.uint8)
        return x
    return (x.double() * size).bfloat16()


def _check(kv, groups, logit=0.0, favoured=None, sink=-math.inf, splits=0, seed=0):
    """All rows are entries of one node.  Its query is zero (all logits 0), or points along row `favoured` so that this
    row's logit is `logit` times 0 .. 1, head by head."""
    rows = _rows(kv, groups, seed)
    n = len(rows)
    v = _f64(rows, kv)
    Q = torch.zeros(H, DIM, dtype=torch.float64, device=DEV)
    if logit:
        r = v[favoured]
        Q = torch.linspace(0, 1, H, dtype=torch.float64, device=DEV)[:, None] * logit * (r / r.abs().max()) / (
            (r / r.abs().max()) @ r)
    Q = Q.bfloat16()
    sinks = torch.full((H,), sink, device=DEV)
    none = torch.zeros(1, dtype=torch.int64, device=DEV)
    out = csa.tree_mqa(Q[None, None], rows[None], rows[None, :1].contiguous(), none, None, None, none + n,
                       none[None] + n, 0, 1, sinks, 1.0, kv_dt=kv, options=csa.mqa_options(splits=splits))[0, 0]
    torch.cuda.synchronize()
    csa.check_device_status()
    z = Q.double() @ v.T
    p = torch.softmax(torch.cat([z, sinks.double()[:, None]], 1), 1)[:, :-1]
    want, A = p @ v, p @ v.abs()
    d = (Q.double().abs() @ v.abs().T).amax(1, keepdim=True) * ((2.0 ** -10 if kv == csa.KV_FP8MIX else 0) + DIM * 2.0 ** -24)
    d = d + 2.0 ** -20
    if kv == csa.KV_FP8MIX:
        tol = A * (2.0 ** -8 + 4 * 2.0 ** -11 + 2 * d)
        tol = tol + n * 2.0 ** -24 * (p * v.abs().amax(1)).amax(1, keepdim=True)
    else:
        tol = A * (2 * 2.0 ** -8 + 2.0 ** -11 + 2 * d)
    err = (out.double() - want).abs()
    assert bool((err <= tol + 1e-30).all()), f"{float((err / (tol + 1e-30)).max()):.3g} times the bound"


SPLITS = [0, 1, 3, 16]
GROUPS = [
    [(1, 2.0 ** 31), (1, 0)],
    [(1, 0), (1, 2.0 ** 31)],
    [(150, 0), (150, 1), (150, 0)],
    [(300, 2.0 ** -60), (300, 2.0 ** 70)],
    [(300, 2.0 ** 70), (300, 2.0 ** -60)],
    [(400, 2.0 ** 75), (400, 2.0 ** -75), (400, 1)],
    [(20000, 0), (300, 1)],                       # zeros ahead of ordinary rows
    [(20000, 0), (1, 2.0 ** 76)],
    [(17000, 2.0 ** -76), (130, 1)],
    [(600, 0)],                                   # nothing but zeros
    [(600, 2.0 ** -76)],
]


@pytest.mark.parametrize("splits", SPLITS)
@pytest.mark.parametrize("groups", GROUPS, ids=str)
@pytest.mark.parametrize("kv", [csa.BF16, csa.KV_FP8MIX])
def test_equal_logits(kv, groups, splits):
    """Every row weighs the same, whatever its size."""
    _check(kv, groups, splits=splits, seed=1)


@pytest.mark.parametrize("splits", SPLITS)
@pytest.mark.parametrize("groups,favoured,logit", [
    ([(20000, 0), (1, 2.0 ** 76)], 20000, 9.0),       # 20,000 zeros outweigh e^9
    ([(1, 2.0 ** 76), (20000, 0)], 0, 9.0),
    ([(8000, 0), (200, 1)], 8100, 8.0),
    ([(500, 2.0 ** -70), (2, 2.0 ** 60)], 501, 7.0),
], ids=str)
@pytest.mark.parametrize("kv", [csa.BF16, csa.KV_FP8MIX])
def test_small_rows_against_a_favoured_one(kv, groups, favoured, logit, splits):
    _check(kv, groups, logit=logit, favoured=favoured, splits=splits, seed=2)


@pytest.mark.parametrize("splits", SPLITS)
@pytest.mark.parametrize("sink", [0.0, 12.0])
@pytest.mark.parametrize("kv", [csa.BF16, csa.KV_FP8MIX])
def test_sinks_beside_zeros(kv, sink, splits):
    _check(kv, [(3000, 0), (200, 1)], sink=sink, splits=splits, seed=3)
    _check(kv, [(130, 2.0 ** 40), (3000, 2.0 ** -70)], sink=sink, splits=splits, seed=4)
