"""Shapes that the binding of the drafted-step calls must refuse, as the C ABI gets addresses and sizes only: a library
that just records the calls stands in for the real one, and tensors on the CPU for those of the current device."""
import pytest
import torch

from compressed_sparse_attention_hca_b200 import csa

B, T, H, C, E, K, D = 2, 4, 64, 512, 40, 6, 3


class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if not name.startswith(("csa_", "hca_")):
            raise AttributeError(name)

        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    r = _Recorder()
    monkeypatch.setattr(csa, "_lib", r)
    monkeypatch.setattr(csa, "_device_of", lambda t: -1)  # where a CPU tensor says it is
    monkeypatch.setattr(csa, "_current_stream", lambda dev: 0)
    monkeypatch.setattr(csa, "_need_cuda", lambda *ts: None)
    return r


def _tree(**kw):
    a = dict(Q=torch.zeros(B, T, H, C, dtype=torch.bfloat16), entries=torch.zeros(B, E, C, dtype=torch.bfloat16),
             win=torch.zeros(B, 128, C, dtype=torch.bfloat16), win_start=torch.zeros(B, dtype=torch.int64),
             draft=torch.zeros(B, D, C, dtype=torch.bfloat16), mask=torch.zeros(B, T, 1, dtype=torch.int32),
             ctx=torch.zeros(B, dtype=torch.int64), q_pos=torch.zeros(B, T, dtype=torch.int64), sink=torch.zeros(H),
             idx=torch.zeros(B, T, K, dtype=torch.int32), n_nodes=None, options=None, n_entries=None)
    a.update(kw)
    return csa.tree_mqa(a["Q"], a["entries"], a["win"], a["win_start"], a["draft"], a["mask"], a["ctx"], a["q_pos"], 128,
                        4, a["sink"], 1.0, idx=a["idx"], n_nodes=a["n_nodes"], options=a["options"],
                        n_entries=a["n_entries"])


def test_tree_takes_the_documented_shapes(lib):
    _tree()
    _tree(idx=None)
    assert lib.calls.count("csa_tree_mqa") == 2


@pytest.mark.parametrize("kw", [
    dict(idx=torch.zeros(B, T, dtype=torch.int32)),                       # k would be read as T
    dict(idx=torch.zeros(B, T, K, 2, dtype=torch.int32)),
    dict(entries=torch.zeros(B, C, dtype=torch.bfloat16)),                # [B, E] with E as long as a row
    dict(entries=torch.zeros(B, C, 2, C, dtype=torch.bfloat16)),
    dict(win=torch.zeros(B, 128, C, 2, dtype=torch.bfloat16)),
    dict(draft=torch.zeros(B, D, C, 2, dtype=torch.bfloat16)),
    dict(draft=torch.zeros(B, D, dtype=torch.bfloat16)),
    dict(Q=torch.zeros(B, T, C, dtype=torch.bfloat16)),
    dict(n_entries=E + 1),
], ids=lambda kw: f"{next(iter(kw))}-{getattr(next(iter(kw.values())), 'ndim', '')}")
def test_tree_refuses_other_shapes(lib, kw):
    with pytest.raises((ValueError, IndexError)):
        _tree(**kw)
    assert "csa_tree_mqa" not in lib.calls


@pytest.mark.parametrize("rows,batch,n_pages,fits", [(3 * 8, B, 3, True), (3 * 8 - 1, B, 3, False), (3 * 8, B - 1, 3, False),
                                                     (3 * 8, B, 4, False)])
def test_tree_refuses_pools_and_tables_that_are_too_small(lib, rows, batch, n_pages, fits):
    """A page of the table stands for page_entries rows of the pool, and every request has a row of the table."""
    opt = csa.mqa_options(entry_pages=csa.pages(torch.zeros(batch, 5, dtype=torch.int32), 8, n_pages))
    kw = dict(entries=torch.zeros(rows, C, dtype=torch.bfloat16), options=opt, n_entries=E)
    if fits:
        _tree(**kw)
        assert "csa_tree_mqa" in lib.calls
    else:
        with pytest.raises(ValueError):
            _tree(**kw)
        assert "csa_tree_mqa" not in lib.calls


@pytest.mark.parametrize("g,fits", [(torch.ones(C), True), (torch.ones(C - 4), False),
                                    (torch.ones(C, dtype=torch.bfloat16), False)])
def test_tree_refuses_query_norm_weights_of_other_sizes(lib, g, fits):
    opt = csa.mqa_options(q_norm_g=g)
    if fits:
        _tree(options=opt)
        assert "csa_tree_mqa" in lib.calls
    else:
        with pytest.raises(ValueError):
            _tree(options=opt)
        assert "csa_tree_mqa" not in lib.calls


def _linear(x, w, out=None):
    u8 = dict(dtype=torch.uint8)
    return csa.nvfp4_linear(torch.zeros(*x, **u8), torch.zeros(1 << 16, **u8), torch.zeros(*w, **u8),
                            torch.zeros(1 << 16, **u8), out=out, ws=torch.zeros(256, **u8))


def test_product_takes_matrices_only(lib):
    """Codes of three dimensions, as quant_nvfp4 gives them for such rows, are not multiplied by their first ones."""
    _linear((6, 64), (8, 64))
    assert lib.calls.count("csa_nvfp4_linear") == 1
    for x, w in (((6, 64, 64), (8, 64)), ((6, 64), (8, 64, 2)), ((64,), (8, 64)), ((6, 64), (64,)), ((6, 64), (8, 32))):
        with pytest.raises(ValueError):
            _linear(x, w)
    with pytest.raises(ValueError):
        _linear((6, 64), (8, 64), out=torch.zeros(8, 6))
    assert lib.calls.count("csa_nvfp4_linear") == 1
