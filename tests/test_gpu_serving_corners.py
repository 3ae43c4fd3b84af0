"""Corners of the serving operators on the GPU against 64-bit references: sequences
shorter than the query tokens."""
import pytest
import torch

from sparse_kv_cache_kmax_b200 import binding as B

from serving_helpers import Paged, check_decode
from test_gpu_serving import _decode

pytestmark = pytest.mark.gpu
BOTH = pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])


# ------------------------------------------------------------------ fewer tokens than queries
SHORT = {
    # lens, G, d, S, T, options: rows at positions below 0 see nothing, whatever the prefix
    "t32": ([20, 100, 16, 31, 32], 2, 64, 16, 32, {"prefix": [20, 40, 16, 31, 32]}),
    "t32_window": ([20, 100, 16, 31, 32], 2, 128, 16, 32, {"prefix": [20, 40, 16, 17, 5], "window": 9}),
    "t17_page32": ([16, 17, 40], 1, 64, 32, 17, {"prefix": [16, 16, 33], "slopes": "alibi"}),
    "t64": ([20, 40, 63, 64, 90], 1, 64, 16, 64, {"prefix": [20, 33, 48, 64, 80], "cap": 20.0}),
    "t16_g4": ([15, 16, 48], 4, 128, 16, 16, {"prefix": [15, 16, 16]}),
    "t40_start": ([39, 24], 1, 128, 16, 40, {"prefix": [32, 24], "start": [16, 3], "slopes": "rising"}),
}


@BOTH
@pytest.mark.parametrize("name", list(SHORT))
def test_rows_before_a_sequences_first_token_see_no_prefix(name, q4):
    lens, G, d, S, T, opts = SHORT[name]
    pg = Paged(lens, 2, d, S, seed=700 + list(SHORT).index(name))
    q = pg.randn(len(lens), T, 2 * G, d)
    out, lse, want = _decode(pg, q, opts, q4=q4)
    assert B.ekv_get_error() == 0
    check_decode(out, lse, want)
    for b, L in enumerate(lens):
        assert (out[b, : max(0, T - L)] == 0).all() and torch.isneginf(lse[b, : max(0, T - L)]).all()


@BOTH
def test_rows_before_a_sequences_first_token_see_no_picked_page(q4):
    lens, T = [20, 60], 32
    pg = Paged(lens, 2, 64, 16, seed=710)
    sel = torch.tensor([[[0, 1, 0], [1, 0, 0]], [[0, 2, 3], [0, 1, 2]]], dtype=torch.int32, device="cuda")
    n = torch.tensor([[2, 2], [3, 3]], dtype=torch.int32, device="cuda")
    out, lse, want = _decode(pg, pg.randn(2, T, 4, 64), {"prefix": [20, 40]}, q4=q4, sel=sel, n_sel=n)
    assert B.ekv_get_error() == 0
    check_decode(out, lse, want)
