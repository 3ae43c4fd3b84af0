"""Corners of the serving operators on the GPU against 64-bit references: sequences
shorter than the query tokens, many short sequences in one run of a CTA, numbers that are
not finite, and sizes near the ends of fp32."""
import numpy as np
import pytest
import torch

from sparse_kv_cache_kmax_b200 import binding as B

from serving_helpers import (Paged, check_decode, decode64, np64, q4_values, quantise64, rope_table, rotate64,
                             unpack)
from test_gpu_serving import _decode

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
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


# ------------------------------------------------------------------ numbers that are not finite
@pytest.mark.parametrize("rotate", [None, False, True], ids=["plain", "halves", "neighbours"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_4_bit_rows_with_a_number_that_is_not_finite_are_nan(d, dtype, rotate):
    """One NaN or infinity in a row of K or V, at every lane's place: that row reads back
    as NaN, step and metadata show it, and the rows beside it are what they would be."""
    rows, hkv, S, rot = 70, 2, 16, d // 2
    pg = Paged([rows], hkv, d, S, seed=720 + d)
    k, v = pg.randn(rows, hkv, d, dtype=dtype), pg.randn(rows, hkv, d, dtype=dtype)
    table = rope_table(rows, rot)
    junk = [float("nan"), float("inf"), -float("inf")]
    hit = np.zeros((2, rows, hkv), bool)
    for n in range(0, rows, 3):                      # with untouched rows between: two share a warp's step
        part, h, at = n % 2, (n // 3) % hkv, (n * 13) % d
        (k, v)[part][n, h, at] = junk[n % 7 % 3]
        hit[part, n, h] = True
    pool = torch.zeros_like(pg.pool_q4())
    box = torch.zeros(hkv, pg.n_phys, 2, d, dtype=BF, device="cuda")
    mom = torch.zeros_like(box)
    cache, seqs = B.make_cache_q4(pool, d, box, mom), B.make_seqs(pg.table, pg.seq_lens)
    indptr = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    B.ekv_rope_append_q4(cache, seqs, None if rotate is None else B.make_rope(table, rotate),
                         B.make_new_tokens(k, v, indptr=indptr))
    got = [torch.zeros(rows, hkv, d, device="cuda") for _ in range(2)]
    B.ekv_q4_read(cache, seqs, indptr, *got)
    assert B.ekv_get_error() == 0
    codes, step, zero = unpack(pool, d)
    x = [np64(k), np64(v)]
    if rotate is not None:
        with np.errstate(invalid="ignore"):
            x[0] = rotate64(x[0], np64(table), np.arange(rows), rotate)
    for n in range(rows):
        ph, s = int(pg.table_h[0, n // S]), n % S
        for h in range(hkv):
            for part in (0, 1):
                at = (ph, h, 0, part, s)
                if hit[part, n, h]:
                    assert torch.isnan(got[part][n, h]).all(), (part, n, h)
                    assert not np.isfinite(step[at])
                else:
                    c, st, ze = quantise64(x[part][n, h])
                    assert np.array_equal(codes[at], c) and step[at] == st and zero[at] == ze, (part, n, h)
    for p in range(pg.pages[0]):                     # the moments of a page that holds such a key are NaN
        ph = int(pg.table_h[0, p])
        for h in range(hkv):
            bad = hit[0, p * S: (p + 1) * S, h].any()
            assert bool(torch.isnan(mom[h, ph]).all()) == bad and bool(torch.isnan(mom[h, ph]).any()) == bad


@pytest.mark.parametrize("part", [0, 1], ids=["key", "value"])
def test_an_appended_nan_reaches_the_rows_that_see_it(part):
    """Append, then decode: of two query tokens only the one that sees the NaN token is NaN."""
    pg = Paged([41], 1, 64, 16, seed=730)
    k, v = pg.randn(41, 1, 64), pg.randn(41, 1, 64)
    (k, v)[part][40, 0, 17] = float("nan")
    pool = torch.zeros_like(pg.pool_q4())
    indptr = torch.tensor([0, 41], dtype=torch.int32, device="cuda")
    B.ekv_rope_append_q4(B.make_cache_q4(pool, 64), B.make_seqs(pg.table, pg.seq_lens), None,
                         B.make_new_tokens(k, v, indptr=indptr))
    out, _, _ = _decode(pg, pg.randn(1, 2, 4, 64), {}, q4=True, pools=pool)
    assert torch.isfinite(out[:, 0]).all() and torch.isnan(out[:, 1]).all()
    assert B.ekv_get_error() == 0


# ------------------------------------------------------------------ sizes near the ends of fp32
def _pairs(pool, d, part, step, zero):
    """Sets the (step, zero) of K (part 0) or V (part 1) of every token."""
    sz = torch.stack([torch.as_tensor(step, device="cuda").expand(16), torch.as_tensor(zero, device="cuda").expand(16)], -1)
    at = 16 * d + 64 * part
    pool[..., at: at + 64] = sz.to(BF).contiguous().view(torch.uint8).reshape(64)


@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("step,zero", [
    (0.0, 2.0 ** 126), (0.0, -2.0 ** 97), (2.0 ** -20, 2.0 ** 110), (2.0 ** 60, -2.0 ** 63), (2.0 ** 62, 2.0 ** 120),
    (0.0, 2.0 ** -100), (2.0 ** -60, 2.0 ** 40)])
def test_4_bit_values_of_every_size(step, zero, T):
    """Rows of V far larger than their steps: the weighted mean of finite values is finite."""
    d = 64
    pg = Paged([700, 3], 2, d, 16, seed=740)
    pool = pg.pool_q4()
    lens = torch.arange(16, device="cuda") % 3 / 8.0 + 0.75  # tokens of a tile differ
    _pairs(pool, d, 1, step * lens, zero * lens)
    out, lse, want = _decode(pg, pg.randn(2, T, 8, d), {}, q4=True, pools=pool)
    assert B.ekv_get_error() == 0
    check_decode(out, lse, want)


@pytest.mark.parametrize("T", [1, 4])
def test_4_bit_values_of_mixed_sizes(T):
    """Small and large rows of V side by side, the large ones at the far end."""
    d = 128
    pg = Paged([900], 1, d, 16, seed=741)
    pool = pg.pool_q4()
    big = torch.tensor(pg.table_h[0, :9].astype(np.int64), device="cuda")
    part = pool[big].clone()
    _pairs(part, d, 1, 0.0, 2.0 ** 115)
    pool[big] = part
    out, lse, want = _decode(pg, pg.randn(1, T, 4, d), {}, q4=True, pools=pool)
    assert B.ekv_get_error() == 0
    check_decode(out, lse, want)


@BOTH
@pytest.mark.parametrize("cap,scale", [(1e-37, None), (1e-25, None), (1e-20, 1.0), (3.0, 1e30), (1e-30, 1e10), (0.0, 1e38)])
def test_small_caps_and_large_scales_with_scores_of_zero(cap, scale, q4):
    """A query of zeros and keys of zeros score 0 exactly, however large the factor."""
    d = 64
    pg = Paged([200, 40], 1, d, 16, seed=750)
    pools = pg.pool_q4() if q4 else pg.pools()
    q = pg.randn(2, 1, 4, d)
    q[:, :, 1] = 0
    q[:, :, 3, ::2] = 0
    if scale is not None and scale > 1e9:            # larger scores would be decided by the signs of sums near 0
        q.zero_()
    ph = torch.tensor(pg.table_h[0, 2:5].astype(np.int64), device="cuda")
    if q4:
        part = pools[ph].clone()
        part[..., : 8 * d] = 0
        _pairs(part, d, 0, 0.0, 0.0)
        pools[ph] = part
    else:
        pools[0][ph] = 0
    out, lse, want = _decode(pg, q, {"cap": cap}, q4=q4, pools=pools, scale=scale)
    assert B.ekv_get_error() == 0
    assert torch.isfinite(out).all()
    check_decode(out, lse, want)


@pytest.mark.parametrize("G", [4, 16])
def test_large_queries_against_small_4_bit_keys(G):
    d = 128
    pg = Paged([300, 5], 1, d, 16, seed=751)
    pool = pg.pool_q4()
    by = 0.75 + torch.arange(16, device="cuda") % 3 / 8.0
    _pairs(pool, d, 0, 2.0 ** -98 * by, -2.0 ** -95 * by)
    out, lse, want = _decode(pg, (pg.randn(2, 1, G, d).float() * 2.0 ** 97).to(BF), {}, q4=True, pools=pool)
    assert B.ekv_get_error() == 0
    check_decode(out, lse, want)


@BOTH
def test_scores_near_the_lowest_of_fp32_still_count(q4):
    """Tokens alike at a score below -3e38 in base 2: their softmax is their mean all the same."""
    d, lens = 64, [1, 40]
    pg = Paged(lens, 1, d, 16, seed=760)
    pools = pg.pool_q4() if q4 else pg.pools()
    q = torch.zeros(2, 1, 4, d, device="cuda", dtype=BF)
    q[..., 0] = 2.0 ** 64
    low = -1.296875 * 2.0 ** 63                      # the score: -2.2e38, times log2(e) -3.18e38
    if q4:
        _pairs(pools, d, 0, 0.0, low)
    else:
        pools[0][:] = 0
        pools[0][..., 0] = low
    out, lse = torch.empty(2, 1, 4, d, device="cuda"), torch.empty(2, 1, 4, device="cuda")
    ws = B.workspace(B.ekv_softmax_mod_workspace_bytes(d, 1, 4, 1), "cuda")
    call = B.ekv_softmax_decode_q4 if q4 else B.ekv_softmax_decode_mod
    call(B.make_cache_q4(pools, d) if q4 else B.make_cache(*pools), B.make_seqs(pg.table, pg.seq_lens), q, 1.0, None,
         None, None, pg.max_pages, out, ws, lse=lse)
    assert B.ekv_get_error() == 0
    V = q4_values(pools, d)[1] if q4 else np64(pools[1])
    for b, L in enumerate(lens):
        rows = V[pg.table_h[b, : pg.pages[b]], 0].reshape(-1, d)[:L]
        # equal weights: sums of L and of L products round by 2**-24 each, and so does the quotient
        assert (np.abs(np64(out[b, 0]) - rows.mean(0)) <= (L + 2) * 2.0 ** -23 * np.abs(rows).max()).all()
        assert (np.abs(np64(lse[b]) / (2.0 ** 64 * low) - 1) <= 4 * 2.0 ** -24).all()


def test_4_bit_steps_and_zeros_are_rounded_by_way_of_fp32():
    """2^-26 beyond the middle of two bf16 numbers: on it in fp32, so to the even one."""
    d = 64
    pg = Paged([1], 1, d, 16, seed=780)
    v = torch.linspace(0, 15, d, dtype=F32, device="cuda")[None, None].clone()
    v[0, 0, 0], v[0, 0, 1] = -15 * 2.0 ** -26, 15 + 15 / 256           # (max - min)/15 = 1 + 2^-8 + 2^-26
    k = torch.zeros_like(v)
    k[0, 0, 0], k[0, 0, d // 2] = -(1 + 2.0 ** -8), 1                  # turned: min = -(1 + 2^-8 + 2^-26)
    table = torch.zeros(1, d, device="cuda")
    table[:, : d // 2] = 1
    table[0, d // 2] = 2.0 ** -26
    pool = torch.zeros_like(pg.pool_q4())
    B.ekv_rope_append_q4(B.make_cache_q4(pool, d), B.make_seqs(pg.table, pg.seq_lens), B.make_rope(table),
                         B.make_new_tokens(k, v))
    codes, step, zero = unpack(pool, d)
    ph = int(pg.table_h[0, 0])
    assert step[ph, 0, 0, 1, 0] == 1.0 and zero[ph, 0, 0, 0, 0] == -1.0
    for part, row in ((0, rotate64(np64(k), np64(table), np.array([0]), False)[0, 0]), (1, np64(v)[0, 0])):
        c, st, ze = quantise64(row)
        assert np.array_equal(codes[ph, 0, 0, part, 0], c) and step[ph, 0, 0, part, 0] == st and zero[ph, 0, 0, part, 0] == ze
    assert B.ekv_get_error() == 0
