"""Corners of the serving operators on the GPU against 64-bit references: sequences
shorter than the query tokens, and many short sequences in one run of a CTA."""
import numpy as np
import pytest
import torch

from sparse_kv_cache_kmax_b200 import binding as B

from serving_helpers import Paged, check_decode, decode64, np64, q4_values
from test_gpu_serving import _decode

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
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


# ------------------------------------------------------------------ units one after another
@BOTH
@pytest.mark.parametrize("G,T", [(4, 1), (8, 3), (16, 4)])
def test_runs_over_many_units_with_masked_tails(G, T, q4):
    """More units than CTAs, so that a CTA's ring goes from one unit to the next right
    after steps that zeroed masked rows of V in it: junk behind every length, the
    reference's values, and the same bits every time."""
    hkv, d, S = 4, 64, 16
    lens = [17 + 37 * i % 211 for i in range(90)]
    pg = Paged(lens, hkv, d, S, seed=770)
    pools = pg.pool_q4() if q4 else pg.pools()
    q = pg.randn(len(lens), T, hkv * G, d)
    scale, some = float(np.float32(1 / np.sqrt(d))), [0, 1, 2, 30, 61, 87, 88, 89]
    K, V = q4_values(pools, d) if q4 else (np64(pools[0]), np64(pools[1]))
    few = Paged.__new__(Paged)
    few.__dict__.update(pg.__dict__)
    few.lens, few.pages, few.table_h = [lens[b] for b in some], [pg.pages[b] for b in some], pg.table_h[some]
    want = decode64(few, K, V, q[some], scale, window=50)
    for b, L in enumerate(lens):
        if L % S:
            at = (int(pg.table_h[b, L // S]), slice(None))
            if q4:
                pools[at][..., 0, 16 * d:].view(BF).view(hkv, 2, 16, 2)[:, :, L % S:] = float("nan")
            else:
                for x in pools:
                    x[at][:, L % S:] = float("nan")
    cache = B.make_cache_q4(pools, d) if q4 else B.make_cache(*pools)
    seqs, mod = B.make_seqs(pg.table, pg.seq_lens), B.make_score_mod(window=50)
    ws = B.workspace(B.ekv_softmax_mod_workspace_bytes(d, hkv, hkv * G, T), "cuda")
    call = B.ekv_softmax_decode_q4 if q4 else B.ekv_softmax_decode_mod
    got = []
    for _ in range(20):
        out, lse = torch.full(q.shape, 7.0, device="cuda"), torch.full(q.shape[:3], 7.0, device="cuda")
        call(cache, seqs, q, scale, mod, None, None, pg.max_pages, out, ws, lse=lse)
        got.append((out, lse))
    assert B.ekv_get_error() == 0
    check_decode(got[0][0][some], got[0][1][some], want)
    assert all(torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1]) for out, lse in got[1:])
