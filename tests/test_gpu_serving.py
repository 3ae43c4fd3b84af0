"""The serving operators on the GPU against 64-bit references: the rotated append
into bf16, fp32 and 4-bit caches, the 4-bit read-back, and the softmax decode
with capped, biased and masked scores over bf16 and 4-bit caches."""
import numpy as np
import pytest
import torch

from sparse_kv_cache_kmax_b200 import binding as B

from serving_helpers import (HALF, Paged, check_decode, decode64, np64, q4_values, quantise64, rope_table, rotate64,
                             rotation_slack, unpack)

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------ append
def _tokens(pg, new, hq, dtype, strided, pad):
    rows = sum(new) + pad
    if strided:
        x = pg.randn(rows, hq + 2 * pg.hkv, pg.d, dtype=dtype)
        q, k, v = x[:, :hq], x[:, hq:hq + pg.hkv], x[:, hq + pg.hkv:]
    else:
        q, k, v = (pg.randn(rows, n, pg.d, dtype=dtype) for n in (hq, pg.hkv, pg.hkv))
    q_out = torch.full((rows, hq, pg.d), 7.0, dtype=dtype, device="cuda")
    indptr = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    return q, k, v, q_out, indptr


def _places(pg, new):
    """(row, sequence, position, physical page, slot) of every new token."""
    row = 0
    for b, (L, n) in enumerate(zip(pg.lens, new)):
        for p in range(L - n, L):
            yield row, b, p, int(pg.table_h[b, p // pg.S]), p % pg.S
            row += 1


APPENDS = {
    # name: dtype, d, S, Hkv, G, rot, interleaved, strided rows, lengths after, new tokens, padding rows
    "one_each": (BF, 128, 16, 2, 4, 128, False, True, [1, 17, 16, 33, 700], [1, 1, 1, 1, 1], 3),
    "one_each_f32": (F32, 64, 32, 3, 1, 64, False, False, [1, 32, 33], [1, 1, 1], 0),
    "prompts": (BF, 128, 16, 2, 2, 128, False, True, [100, 16, 1, 257], [100, 16, 1, 257], 0),
    "chunks_interleaved": (BF, 128, 32, 2, 1, 64, True, True, [90, 64, 65, 12], [41, 2, 33, 12], 5),
    "chunks_f32_partial": (F32, 64, 16, 1, 8, 32, True, False, [75, 40], [50, 7], 1),
    "partial_half": (BF, 64, 16, 4, 16, 16, False, False, [31, 48, 5], [16, 18, 2], 0),
    "idle_and_none": (BF, 128, 16, 2, 4, 128, False, True, [0, 40, 0, 33, 20], [0, 0, 0, 18, 1], 2),
    "many_short": (BF, 64, 16, 1, 2, 64, False, True, [3 + i % 40 for i in range(77)], [1 + i % 3 for i in range(77)], 0),
}


def _case(name):
    dtype, d, S, hkv, G, rot, inter, strided, lens, new, pad = APPENDS[name]
    pg = Paged(lens, hkv, d, S, seed=list(APPENDS).index(name))
    return pg, new, hkv * G, dtype, rot, inter, strided, pad


@pytest.mark.parametrize("name", list(APPENDS))
def test_rope_append(name):
    pg, new, hq, dtype, rot, inter, strided, pad = _case(name)
    q, k, v, q_out, indptr = _tokens(pg, new, hq, dtype, strided, pad)
    kp, vp = pg.pools(dtype)
    k0, v0 = kp.clone(), vp.clone()
    cache = B.make_cache(kp, vp)
    cache.box_t.fill_(3.0)
    cache.mom_t.fill_(4.0)
    seqs = B.make_seqs(pg.table, pg.seq_lens)
    table = rope_table(max(pg.lens), rot)
    once = all(n == 1 for n in new)
    B.ekv_rope_append(cache, seqs, B.make_rope(table, inter),
                      B.make_new_tokens(k, v, q, q_out, None if once else indptr))
    assert B.ekv_get_error() == 0
    places = list(_places(pg, new))
    rows, pos = [p[0] for p in places], np.array([p[2] for p in places])
    tab = np64(table)
    for got, x in ((q_out[rows], q[rows]), (torch.stack([kp[p[3], :, p[4]] for p in places]), k[rows])):
        x = np64(x)
        want, slack = rotate64(x, tab, pos, inter), rotation_slack(x, tab, inter)
        assert (np.abs(np64(got) - want) <= HALF[dtype] * np.abs(want) + (1 + HALF[dtype]) * slack).all()
    touched = torch.zeros(pg.n_phys, pg.S, dtype=torch.bool)
    for r, _, _, ph, s in places:
        touched[ph, s] = True
        assert torch.equal(vp[ph, :, s], v[r])
    rest = ~touched.cuda()
    assert torch.equal(kp.transpose(1, 2)[rest], k0.transpose(1, 2)[rest])
    assert torch.equal(vp.transpose(1, 2)[rest], v0.transpose(1, 2)[rest])
    assert (q_out[sum(new):] == 7).all()
    # metadata: what a fresh build over the same keys gives, of touched pages alone
    fresh = B.make_cache(kp, vp, torch.zeros_like(cache.box_t), torch.zeros_like(cache.mom_t))
    idle = [b for b, L in enumerate(pg.lens) if L == 0]
    lens = pg.seq_lens.clone()
    lens[idle] = 1
    B.ekv_build_page_meta(fresh, B.make_seqs(pg.table, lens))
    hit = touched.any(1).cuda()
    assert torch.equal(cache.box_t[:, hit], fresh.box_t[:, hit]) and torch.equal(cache.mom_t[:, hit], fresh.mom_t[:, hit])
    assert (cache.box_t[:, ~hit] == 3).all() and (cache.mom_t[:, ~hit] == 4).all()


def test_rope_append_without_rotation_matches_append_and_rotates_in_place():
    pg = Paged([50, 16, 129], 2, 128, 16, seed=5)
    k, v = pg.randn(3, 2, 128), pg.randn(3, 2, 128)
    kp, vp = pg.pools()
    meta = lambda: torch.zeros(2, pg.n_phys, 2, 128, dtype=BF, device="cuda")  # noqa: E731
    a, b = (B.make_cache(kp.clone(), vp.clone(), meta(), meta()) for _ in range(2))
    seqs = B.make_seqs(pg.table, pg.seq_lens)
    for c in (a, b):
        B.ekv_build_page_meta(c, seqs)
    B.ekv_append(a, seqs, k, v)
    B.ekv_rope_append(b, seqs, None, B.make_new_tokens(k, v))
    for x, y in zip(a._keep, b._keep):
        assert torch.equal(x, y)
    q = pg.randn(3, 8, 128)
    q1, q2 = torch.empty_like(q), q.clone()
    rope = B.make_rope(rope_table(129, 128))
    B.ekv_rope_append(b, seqs, rope, B.make_new_tokens(k, v, q, q1))
    B.ekv_rope_append(b, seqs, rope, B.make_new_tokens(k, v, q2, q2))
    assert torch.equal(q1, q2) and not torch.equal(q1, q)
    assert B.ekv_get_error() == 0


def test_appends_without_metadata():
    """box and mom left out: the same K, V and q, and nothing else is touched."""
    pg = Paged([50, 16, 129], 2, 64, 32, seed=7)
    new = [50, 3, 129]
    q, k, v, q_out, indptr = _tokens(pg, new, 4, BF, True, 0)
    seqs, rope = B.make_seqs(pg.table, pg.seq_lens), B.make_rope(rope_table(129, 64))
    got = []
    for meta in (True, False):
        kp, vp = pg.pools()[0].fill_(1), pg.pools()[0].fill_(2)
        c = B.make_cache(kp, vp)
        if not meta:
            c.box = c.mom = None
        B.ekv_rope_append(c, seqs, rope, B.make_new_tokens(k, v, q, q_out, indptr))
        pool = torch.zeros_like(pg.pool_q4())
        box = torch.zeros(2, pg.n_phys, 2, 64, dtype=BF, device="cuda")
        B.ekv_rope_append_q4(B.make_cache_q4(pool, 64, *((box, box.clone()) if meta else ())), seqs, rope,
                             B.make_new_tokens(k, v, q, q_out, indptr))
        got.append((kp, vp, pool, q_out.clone()))
    assert all(torch.equal(a, b) for a, b in zip(*got)) and B.ekv_get_error() == 0


def test_append_faults_are_flagged_and_skipped():
    pg = Paged([40, 33, 20], 2, 64, 16, seed=6)
    rope = B.make_rope(rope_table(35, 64))

    def run(indptr, lens=None, table=None, rows=40):
        kp, vp = pg.pools()
        c = B.make_cache(kp, vp, *(torch.zeros(2, pg.n_phys, 2, 64, dtype=BF, device="cuda") for _ in range(2)))
        before = [t.clone() for t in c._keep]
        k, v = pg.randn(rows, 2, 64), pg.randn(rows, 2, 64)
        seqs = B.make_seqs(pg.table if table is None else table,
                           pg.seq_lens if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda"))
        B.ekv_rope_append(c, seqs, rope, B.make_new_tokens(
            k, v, indptr=None if indptr is None else torch.tensor(indptr, dtype=torch.int32, device="cuda")))
        same = all(torch.equal(x, y) for x, y in zip(before, c._keep))
        return B.ekv_get_error(), same

    assert run([0, 0, 0, 0]) == (0, True)
    assert run([0, 0, 0, 21]) == (B.EKV_EFLAG_BAD_LEN, True)         # more new tokens than the sequence has
    assert run([0, 0, 0, 41], rows=40)[0] == B.EKV_EFLAG_BAD_LEN      # rows past num_tokens
    assert run([0, 3, 1, 1])[0] & B.EKV_EFLAG_BAD_LEN                 # decreasing
    assert run([-7, -7, -7, -7])[0] in (0, B.EKV_EFLAG_BAD_LEN)
    assert run([0, 0, 0, 2], lens=[40, 33, 20 + 16 * pg.max_pages])[0] == B.EKV_EFLAG_BAD_LEN
    assert run([0, 0, 0, 2], lens=[40, 33, -5]) == (B.EKV_EFLAG_BAD_LEN, True)
    bad = pg.table.clone()
    bad[2, 1] = pg.n_phys
    assert run([0, 0, 0, 2], table=bad) == (B.EKV_EFLAG_BAD_PAGE, True)
    bad[2, 1] = -1
    assert run([0, 0, 0, 2], table=bad) == (B.EKV_EFLAG_BAD_PAGE, True)
    assert run([0, 1, 1, 1])[0] == B.EKV_EFLAG_BAD_POS               # position 39, table of 35
    assert run(None, lens=[0, 33, 0])[0] == 0                         # idle slots of a step


# ------------------------------------------------------------------ 4 bits
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("name", [n for n in APPENDS if "f32" not in n])
def test_rope_append_q4(name, dtype):
    pg, new, hq, _, rot, inter, strided, pad = _case(name)
    q, k, v, q_out, indptr = _tokens(pg, new, hq, dtype, strided, pad)
    pool = pg.pool_q4()
    before = pool.clone()
    box = torch.full((pg.hkv, pg.n_phys, 2, pg.d), 3.0, dtype=BF, device="cuda")
    mom = torch.full_like(box, 4.0)
    cache = B.make_cache_q4(pool, pg.d, box, mom)
    seqs = B.make_seqs(pg.table, pg.seq_lens)
    table = rope_table(max(pg.lens), rot)
    once = all(n == 1 for n in new)
    B.ekv_rope_append_q4(cache, seqs, B.make_rope(table, inter),
                         B.make_new_tokens(k, v, q, q_out, None if once else indptr))
    assert B.ekv_get_error() == 0
    places = list(_places(pg, new))
    rows, pos = [p[0] for p in places], np.array([p[2] for p in places])
    tab = np64(table)
    x = np64(q[rows])
    want, slack = rotate64(x, tab, pos, inter), rotation_slack(x, tab, inter)
    assert (np.abs(np64(q_out[rows]) - want) <= HALF[dtype] * np.abs(want) + (1 + HALF[dtype]) * slack).all()
    assert (q_out[sum(new):] == 7).all()
    kr, vr = rotate64(np64(k[rows]), tab, pos, inter), np64(v[rows])
    codes, step, zero = unpack(pool, pg.d)
    touched = np.zeros((pg.n_phys, pg.S // 16, 16), bool)
    for n, (_, _, _, ph, s) in enumerate(places):
        touched[ph, s // 16, s % 16] = True
        for h in range(pg.hkv):
            for part, row in ((0, kr[n, h]), (1, vr[n, h])):
                c, st, ze = quantise64(row)
                at = (ph, h, s // 16, part, s % 16)
                assert np.array_equal(codes[at], c) and step[at] == st and zero[at] == ze
    old = unpack(before, pg.d)
    for a, b in zip((codes, step, zero), old):
        keep = np.broadcast_to(~touched[:, None, :, None, :], step.shape)
        assert np.array_equal(a[keep], b[keep])
    # metadata of touched pages: bounds of, and moments over, the values the codes stand for
    kv, _ = q4_values(pool, pg.d)
    pages = {}
    for _, b, p, ph, s in places:
        pages[ph] = min(pg.S, pg.lens[b] - p // pg.S * pg.S)
    bx, mo = np64(box), np64(mom)
    for ph in range(pg.n_phys):
        if ph not in pages:
            assert (bx[:, ph] == 3).all() and (mo[:, ph] == 4).all()
            continue
        vals = kv[ph][:, : pages[ph]]
        hi, lo = vals.max(1), vals.min(1)
        vals32 = vals.astype(np.float32).astype(np.float64)  # as the cache's values are read
        assert (bx[:, ph, 0] >= vals32.max(1)).all() and (bx[:, ph, 1] <= vals32.min(1)).all()
        assert (bx[:, ph, 0] - hi <= 2.0 ** -7 * np.abs(hi) + 1e-30).all()
        assert (lo - bx[:, ph, 1] <= 2.0 ** -7 * np.abs(lo) + 1e-30).all()
        mean, var = vals32.mean(1), vals32.var(1)
        near = 2.0 ** -50 * np.abs(vals32).max() ** 2
        assert (np.abs(mo[:, ph, 0] - mean) <= 2.0 ** -8 * np.abs(mean) + near).all()
        assert (np.abs(mo[:, ph, 1] - var) <= 2.0 ** -8 * np.abs(var) + near).all()
    # the read-back: zero + step·n, rounded once to fp32, and from there to bf16
    for out in (F32, BF):
        total = max(sum(new), 1) + 2
        ko, vo = (torch.full((total, pg.hkv, pg.d), 9.0, dtype=out, device="cuda") for _ in range(2))
        B.ekv_q4_read(cache, seqs, indptr, ko, vo)
        k64, v64 = q4_values(pool, pg.d)
        for got, src in ((ko, k64), (vo, v64)):
            for r, _, _, ph, s in places:
                want = torch.tensor(src[ph, :, s].astype(np.float32))
                assert torch.equal(got[r].cpu(), want.to(out))
            assert (got[sum(new):] == 9).all()
    assert B.ekv_get_error() == 0


def test_q4_rows_of_one_value_borders_and_one_output():
    """Constant rows, rows whose quotients fall on borders between codes, tiny and large scales."""
    d = 64
    pg = Paged([12], 1, d, 16, seed=9)
    x = np.zeros((12, d), np.float64)
    x[0] = 1.5                                        # one value: step 0
    x[1] = np.arange(d) % 31 / 2.0                    # step 1, halves everywhere
    x[2] = -x[1] * 2.0 ** 60
    x[3] = x[1] * 2.0 ** -90
    x[4] = 2.0 ** -110 * (np.arange(d) % 3)           # below the smallest step
    x[5, 0] = 300.0                                   # one outlier
    x[6] = 1000 + np.arange(d) % 8
    x[7] = (np.arange(d) - 31) / 4.0
    x[8] = 2.0 ** 20 + np.arange(d) % 13 / 8.0        # a step far below zero's own spacing
    x[9] = -(2.0 ** 23) + np.arange(d) % 2
    x[10] = np.arange(d) % 16 + (np.arange(d) % 3 - 1) * 2.0 ** -20   # next to the codes
    x[11] = np.arange(d) % 15 + 0.5 + (np.arange(d) % 3 - 1) * 2.0 ** -19   # next to the borders
    x[11, :2] = 0, 15
    v = torch.tensor(x, dtype=F32, device="cuda")[:, None]
    assert np.array_equal(np64(v)[:, 0], x)
    pool = pg.pool_q4()
    cache = B.make_cache_q4(pool, d)
    seqs = B.make_seqs(pg.table, pg.seq_lens)
    indptr = torch.tensor([0, 12], dtype=torch.int32, device="cuda")
    B.ekv_rope_append_q4(cache, seqs, None, B.make_new_tokens(v, v, indptr=indptr))
    codes, step, zero = unpack(pool, d)
    ph = int(pg.table_h[0, 0])
    for r in range(12):
        c, st, ze = quantise64(x[r])
        for part in (0, 1):
            assert np.array_equal(codes[ph, 0, 0, part, r], c), r
            assert step[ph, 0, 0, part, r] == st and zero[ph, 0, 0, part, r] == ze
    only = torch.zeros(12, 1, d, device="cuda")
    B.ekv_q4_read(cache, seqs, indptr, None, only)
    assert torch.equal(only.cpu()[:, 0].double(), torch.tensor(q4_values(pool, d)[1][ph, 0, :12].astype(np.float32)).double())
    assert B.ekv_get_error() == 0


def test_page_scores_of_a_4_bit_cache_bound_its_token_scores():
    lens = [75, 40]
    pg = Paged(lens, 2, 128, 16, seed=11)
    k, v = pg.randn(sum(lens), 2, 128), pg.randn(sum(lens), 2, 128)
    pool = pg.pool_q4()
    box = torch.zeros(2, pg.n_phys, 2, 128, dtype=BF, device="cuda")
    cache = B.make_cache_q4(pool, 128, box, torch.zeros_like(box))
    seqs = B.make_seqs(pg.table, pg.seq_lens)
    indptr = torch.tensor([0, 75, 115], dtype=torch.int32, device="cuda")
    B.ekv_rope_append_q4(cache, seqs, B.make_rope(rope_table(75, 128)), B.make_new_tokens(k, v, indptr=indptr))
    q = pg.randn(2, 8, 128)
    ub = torch.zeros(2, 2, pg.max_pages, device="cuda")
    B.ekv_score_pages(cache.meta, seqs, q, 0.1, ub)
    kv, _ = q4_values(pool, 128)
    for b, L in enumerate(lens):
        for p in range(pg.pages[b]):
            for h in range(2):
                keys = kv[pg.table_h[b, p], h, : min(16, L - 16 * p)]
                z = keys @ np64(q[b, 4 * h: 4 * h + 4]).T * 0.1
                room = 1e-5 * 0.1 * (np.abs(np64(q[b, 4 * h: 4 * h + 4])) @ np.abs(keys).max(0)).max()
                assert z.max() <= float(ub[b, h, p]) + room


# ------------------------------------------------------------------ decode
DECODES = {
    # lens, Hkv, G, d, S, T, options
    "one_token": ([1], 1, 1, 64, 16, 1, {}),
    "lengths": ([1, 2, 15, 16, 17, 31, 32, 33, 255, 700], 2, 4, 128, 16, 1, {}),
    "page32": ([1, 31, 32, 33, 511], 2, 4, 128, 32, 1, {"cap": 50.0}),
    "long": ([20011, 3], 2, 4, 128, 16, 1, {"cap": 20.0}),
    "long_d64": ([9001], 3, 8, 64, 32, 1, {"slopes": "alibi"}),
    "cap": ([300, 77], 2, 8, 128, 16, 1, {"cap": 5.0}),
    "tiny_cap": ([300, 77], 1, 2, 64, 16, 1, {"cap": 0.01}),
    "g16": ([513, 20], 2, 16, 128, 16, 1, {"cap": 30.0, "slopes": "alibi"}),
    "bias": ([1000, 40, 1], 2, 4, 128, 16, 1, {"slopes": "alibi"}),
    "bias_rising": ([1000, 40, 1], 2, 4, 64, 16, 1, {"slopes": "rising"}),
    "bias_steep": ([5000], 1, 4, 128, 16, 1, {"slopes": "steep"}),
    "window": ([600, 40, 100, 5], 2, 4, 128, 16, 1, {"window": 37}),
    "window_one": ([600, 1], 2, 2, 128, 16, 1, {"window": 1}),
    "window_wide": ([600, 40], 2, 2, 64, 32, 1, {"window": 10 ** 9}),
    "window_widest": ([600, 40, 1], 2, 2, 64, 16, 5, {"window": 2 ** 31 - 1, "prefix": [2 ** 31 - 1, 3, -2 ** 31],
                                                      "start": [-2 ** 31, 2, 0]}),
    "cap_widest": ([200], 1, 2, 64, 16, 1, {"cap": 3e38}),
    "cap_smallest": ([200], 1, 2, 64, 16, 1, {"cap": 1e-37}),
    "prefix": ([600, 40, 100, 5], 2, 4, 128, 16, 1, {"window": 20, "prefix": [33, 39, 100, 7]}),
    "prefix_near": ([600, 40], 1, 4, 128, 16, 1, {"window": 32, "prefix": [566, 5]}),
    "start": ([600, 40, 100, 5], 2, 4, 128, 16, 1, {"start": [599, 16, 0, 2]}),
    "start_empty": ([600, 40, 100, 5], 2, 4, 128, 16, 1, {"start": [600, 1000, -3, 2]}),
    "all_masks": ([600, 40, 100, 0], 2, 4, 128, 16, 1,
                  {"window": 20, "prefix": [64, 0, -5, 3], "start": [10, 30, 99, 0], "cap": 9.0, "slopes": "alibi"}),
    "t2": ([300, 1, 17, 2], 2, 4, 128, 16, 2, {}),
    "t4": ([300, 3, 16, 0, 33], 2, 4, 128, 16, 4, {"cap": 30.0, "slopes": "alibi"}),
    "t4_masks": ([300, 3, 16, 40], 2, 2, 64, 16, 4, {"window": 5, "prefix": [9, 3, 15, 40], "start": [2, 0, 14, 38]}),
    "t7_rows28": ([200, 9], 2, 4, 128, 16, 7, {"window": 3}),
    "t16_rows64": ([200, 30], 2, 4, 128, 32, 16, {"slopes": "rising"}),
    "t4_g16": ([400, 90], 1, 16, 128, 16, 4, {"cap": 15.0}),
    "t64_g1": ([100, 70], 2, 1, 64, 16, 64, {"window": 11}),
    "many_units": ([5 + 7 * i % 90 for i in range(150)], 4, 2, 64, 16, 1, {}),
    "batch_over_128": ([1 + i % 3 for i in range(300)], 1, 1, 64, 16, 1, {"cap": 4.0}),
}


def _slopes(kind, hq):
    if kind is None:
        return None
    s = 0.5 ** (8.0 * np.arange(1, hq + 1) / hq)
    return {"alibi": s, "rising": -s / 8, "steep": 40.0 * s}[kind].astype(np.float32)


def _decode(pg, q, opts, *, q4, sel=None, n_sel=None, pools=None, scale=None, ws=None, stream=None):
    """(out, lse, reference) of one decode."""
    d, hq, T = pg.d, q.shape[2], q.shape[1]
    scale = float(np.float32(scale or 1.0 / np.sqrt(d)))
    dev = lambda x, dt: None if x is None else torch.tensor(x, dtype=dt, device="cuda")  # noqa: E731
    slopes = _slopes(opts.get("slopes"), hq)
    mod = B.make_score_mod(opts.get("cap", 0.0), dev(slopes, F32), opts.get("window", 0),
                           dev(opts.get("prefix"), torch.int32), dev(opts.get("start"), torch.int32))
    if pools is None:
        pools = pg.pool_q4() if q4 else pg.pools()
    cache = B.make_cache_q4(pools, d) if q4 else B.make_cache(*pools)
    seqs = B.make_seqs(pg.table, pg.seq_lens)
    out = torch.full(q.shape, float("nan"), device="cuda")
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    if ws is None:
        ws = B.workspace(B.ekv_softmax_mod_workspace_bytes(d, pg.hkv, hq, T), "cuda")
        ws.fill_(0xff)
    cap = pg.max_pages if sel is None else sel.shape[-1]
    call = B.ekv_softmax_decode_q4 if q4 else B.ekv_softmax_decode_mod
    call(cache, seqs, q, scale, mod, sel, n_sel, cap, out, ws, lse=lse)
    K, V = q4_values(pools, d) if q4 else (np64(pools[0]), np64(pools[1]))
    want = decode64(pg, K, V, q, scale, cap=opts.get("cap", 0.0), slopes=slopes, window=opts.get("window", 0),
                    prefix=opts.get("prefix"), start=opts.get("start"), sel=None if sel is None else sel.cpu().numpy(),
                    n_sel=None if sel is None else n_sel.cpu().numpy())
    return out, lse, want


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
@pytest.mark.parametrize("name", list(DECODES))
def test_decode(name, q4):
    lens, hkv, G, d, S, T, opts = DECODES[name]
    pg = Paged(lens, hkv, d, S, seed=100 + list(DECODES).index(name))
    q = pg.randn(len(lens), T, hkv * G, d)
    out, lse, want = _decode(pg, q, opts, q4=q4)
    assert B.ekv_get_error() == 0
    check_decode(out, lse, want)


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
@pytest.mark.parametrize("opts", [{}, {"window": 70, "prefix": [20, 0, 300], "start": [3, 0, 40], "slopes": "alibi"}],
                         ids=["plain", "masks"])
@pytest.mark.parametrize("S,T", [(16, 1), (32, 3)])
def test_decode_of_selected_pages(q4, opts, S, T):
    pg = Paged([500, 20, 333], 2, 128, S, seed=300)
    rng = np.random.default_rng(1)
    cap = 9
    sel, n = np.zeros((3, 2, cap), np.int32), np.zeros((3, 2), np.int32)
    for b in range(3):
        for h in range(2):
            n[b, h] = min(cap, pg.pages[b]) if (b, h) != (2, 1) else 0      # one unit selects nothing
            sel[b, h, : n[b, h]] = np.sort(rng.permutation(pg.pages[b])[: n[b, h]])
    sel[0, 0, 1] = sel[0, 0, 0]                                             # the same page twice counts twice
    q = pg.randn(3, T, 8, 128)
    out, lse, want = _decode(pg, q, opts, q4=q4, sel=torch.tensor(sel, device="cuda"), n_sel=torch.tensor(n, device="cuda"))
    assert B.ekv_get_error() == 0
    check_decode(out, lse, want)


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
def test_masked_places_may_hold_anything(q4):
    """NaN and infinities behind the last token, before the document, outside the window and in unused pages."""
    lens, S, d = [70, 33, 161], 16, 128
    opts = {"window": 25, "start": [40, 9, 0], "prefix": [0, 0, 19]}
    for T in (1, 3):
        pg = Paged(lens, 2, d, S, seed=400 + T)
        pools = pg.pool_q4() if q4 else pg.pools()
        dirty = pools.clone() if q4 else [x.clone() for x in pools]
        bad = torch.ones(pg.n_phys, S, dtype=torch.bool)
        for b, L in enumerate(lens):
            for j in range(L):
                i = L - T
                near = j > i - opts["window"] or j < opts["prefix"][b]
                if near and j >= opts["start"][b]:
                    bad[pg.table_h[b, j // S], j % S] = False
        where = torch.nonzero(bad)
        junk = [float("nan"), float("inf"), -float("inf")]
        for n, (ph, s) in enumerate(where.tolist()):
            if q4:
                pair = torch.full((2,), junk[n % 3], dtype=BF, device="cuda").view(torch.uint8)
                for part in (0, 1):
                    at = 16 * d + 4 * (part * 16 + s % 16)
                    dirty[ph, :, s // 16, at: at + 4] = pair
            else:
                for x in dirty:
                    x[ph, :, s] = junk[n % 3]
        q = pg.randn(3, T, 8, d)
        clean = _decode(pg, q, opts, q4=q4, pools=pools)
        check_decode(clean[0], clean[1], clean[2])
        got = _decode(pg, q, opts, q4=q4, pools=dirty)
        assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])


@pytest.mark.parametrize("G,T", [(2, 4), (8, 2), (8, 4), (16, 4)])
def test_a_later_tokens_nan_stays_with_the_rows_that_see_it(G, T):
    lens, d = [37, 64], 128
    pg = Paged(lens, 2, d, 16, seed=410)
    k, v = pg.pools()
    q = pg.randn(2, T, 2 * G, d)
    clean = _decode(pg, q, {}, q4=False, pools=(k, v))
    check_decode(*clean)
    for b, L in enumerate(lens):
        v[pg.table_h[b, (L - 1) // 16], :, (L - 1) % 16, ::3] = float("inf")   # the last token: seen by the last row alone
    got = _decode(pg, q, {}, q4=False, pools=(k, v))[0]
    assert torch.allclose(got[:, :-1], clean[0][:, :-1], rtol=0, atol=0)
    assert torch.isinf(got[:, -1, :, ::3]).all() and torch.isfinite(got[:, -1, :, 1::3]).all()


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
def test_a_nan_seen_is_a_nan(q4):
    pg = Paged([1, 40], 1, 64, 16, seed=411)
    pools = pg.pool_q4() if q4 else pg.pools()
    q = pg.randn(2, 1, 4, 64)
    q[:, :, 1] = float("nan")
    out, lse, _ = _decode(pg, q, {"cap": 10.0}, q4=q4, pools=pools)
    assert torch.isnan(out[:, :, 1]).all() and torch.isnan(lse[:, :, 1]).all()
    keep = [0, 2, 3]
    assert torch.isfinite(out[:, :, keep]).all() and torch.isfinite(lse[:, :, keep]).all()


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
def test_scores_of_every_size(q4):
    """Large and shifting scores: the running maximum moves at every tile; and a uniform softmax over a long cache."""
    pg = Paged([3000], 1, 64, 16, seed=412)
    pools = pg.pool_q4() if q4 else pg.pools()
    q = pg.randn(1, 1, 4, 64)
    ramp = torch.zeros(1, 1, 4, 64, device="cuda").to(BF)
    for x, scale in ((q, 3.0), (q, 1e-4), (ramp, 1.0)):
        out, lse, want = _decode(pg, x, {}, q4=q4, pools=pools, scale=scale)
        check_decode(out, lse, want)
    if not q4:
        k, v = pools
        for j in range(3000):  # rising scores
            k[pg.table_h[0, j // 16], 0, j % 16] = 0.02 * j / 64
        one = torch.ones(1, 1, 4, 64, device="cuda").to(BF)
        out, lse, want = _decode(pg, one, {}, q4=False, pools=(k, v), scale=1.0)
        check_decode(out, lse, want)


def test_decode_faults_are_flagged_and_skipped():
    for q4 in (False, True):
        pg = Paged([100, 50], 1, 64, 16, seed=413)
        q = pg.randn(2, 1, 2, 64)
        pools = pg.pool_q4() if q4 else pg.pools()
        good = _decode(pg, q, {}, q4=q4, pools=pools)[0]
        saved = pg.table.clone()
        pg.table[0, 2] = pg.n_phys + 5
        pg.table[0, 3] = -1
        out = _decode(pg, q, {}, q4=q4, pools=pools)[0]
        assert B.ekv_get_error() == B.EKV_EFLAG_BAD_PAGE
        assert torch.isfinite(out).all() and torch.equal(out[1], good[1]) and not torch.equal(out[0], good[0])
        pg.table.copy_(saved)
        lens = pg.seq_lens.clone()
        pg.seq_lens[0] = -4
        pg.seq_lens[1] = 16 * pg.max_pages + 1
        pg.table[1] = pg.table[0]
        out = _decode(pg, q, {}, q4=q4, pools=pools)[0]
        assert B.ekv_get_error() == B.EKV_EFLAG_BAD_LEN
        assert (out[0] == 0).all() and torch.isfinite(out).all()
        pg.seq_lens.copy_(lens)
        pg.table.copy_(saved)
        sel = torch.tensor([[[0, 7, -1]], [[0, 4, 1]]], dtype=torch.int32, device="cuda")
        n = torch.tensor([[3], [99]], dtype=torch.int32, device="cuda")    # clamped to cap
        cache = B.make_cache_q4(pools, 64) if q4 else B.make_cache(*pools)
        ws = B.workspace(B.ekv_softmax_mod_workspace_bytes(64, 1, 2, 1), "cuda")
        out = torch.full((2, 1, 2, 64), float("nan"), device="cuda")
        call = B.ekv_softmax_decode_q4 if q4 else B.ekv_softmax_decode_mod
        call(cache, B.make_seqs(pg.table, pg.seq_lens), q, 0.125, None, sel, n, 3, out, ws)
        assert B.ekv_get_error() == B.EKV_EFLAG_BAD_SEL
        assert torch.isfinite(out).all()


def test_offsets_past_32_bits():
    """Pools of more than 2³¹ numbers, pages at their ends."""
    d, hkv, S = 128, 8, 16
    n_phys = 2 ** 31 // (d * hkv * S) + 300
    k = torch.empty(n_phys, hkv, S, d, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    pg = Paged([150], hkv, d, S, seed=414)
    at = torch.arange(n_phys - pg.max_pages, n_phys, device="cuda").flip(0)
    small = pg.pools()
    rows = torch.tensor(pg.table_h[0].astype(np.int64), device="cuda")
    k[at], v[at] = small[0][rows], small[1][rows]
    q = pg.randn(1, 1, 32, d)
    want = _decode(pg, q, {}, q4=False, pools=small)
    out = torch.empty(1, 1, 32, d, device="cuda")
    ws = B.workspace(B.ekv_softmax_mod_workspace_bytes(d, hkv, 32, 1), "cuda")
    big = B.make_cache(k, v)
    seqs = B.make_seqs(at.int()[None].contiguous(), pg.seq_lens)
    B.ekv_softmax_decode_mod(big, seqs, q, float(np.float32(1 / np.sqrt(d))), None, None, None, pg.max_pages, out, ws)
    assert torch.equal(out, want[0])
    new = pg.randn(1, hkv, d)
    B.ekv_rope_append(big, seqs, None, B.make_new_tokens(new, new))
    assert torch.equal(k[at[149 // S], :, 149 % S], new[0]) and torch.equal(v[at[149 // S], :, 149 % S], new[0])
    del k, v, big
    n_phys = 2 ** 32 // (hkv * (16 * d + 128)) + 300
    pool = torch.empty(n_phys, hkv, 1, 16 * d + 128, dtype=torch.uint8, device="cuda")
    at = at + (n_phys - 1 - int(at[0]))
    small4 = pg.pool_q4()
    pool[at] = small4[rows]
    want = _decode(pg, q, {}, q4=True, pools=small4)
    seqs = B.make_seqs(at.int()[None].contiguous(), pg.seq_lens)
    big = B.make_cache_q4(pool, d)
    B.ekv_softmax_decode_q4(big, seqs, q, float(np.float32(1 / np.sqrt(d))), None, None, None, pg.max_pages, out, ws)
    assert torch.equal(out, want[0])
    ko = torch.empty(150, hkv, d, device="cuda")
    B.ekv_q4_read(big, seqs, torch.tensor([0, 150], dtype=torch.int32, device="cuda"), ko)
    want_k = q4_values(small4, d)[0]
    assert torch.equal(ko[149].cpu(), torch.tensor(want_k[pg.table_h[0, 149 // S], :, 149 % S].astype(np.float32)))
    assert B.ekv_get_error() == 0


def test_streams_captures_and_repeats_agree():
    """Two streams with a workspace each, a captured and replayed pass, and repeats: the same bits."""
    pg = Paged([900, 31, 4000], 2, 128, 16, seed=415)
    kp, vp = pg.pools()
    pool = pg.pool_q4()
    q, k, v = pg.randn(3, 1, 8, 128), pg.randn(3, 2, 128), pg.randn(3, 2, 128)
    seqs = B.make_seqs(pg.table, pg.seq_lens)
    rope = B.make_rope(rope_table(4000, 128))
    caches = B.make_cache(kp, vp), B.make_cache_q4(pool, 128)
    nbytes = B.ekv_softmax_mod_workspace_bytes(128, 2, 8, 1)
    ws = [B.workspace(nbytes, "cuda") for _ in range(2)]
    q_rot = [torch.empty(3, 8, 128, dtype=BF, device="cuda") for _ in range(2)]
    out = [torch.empty(3, 1, 8, 128, device="cuda") for _ in range(2)]
    new = [B.make_new_tokens(k, v, q[:, 0], x) for x in q_rot]
    mod = B.make_score_mod(softcap=30.0)

    def step(n, stream=None):
        append, decode = ((B.ekv_rope_append, B.ekv_softmax_decode_mod),
                          (B.ekv_rope_append_q4, B.ekv_softmax_decode_q4))[n]
        append(caches[n], seqs, rope, new[n], stream=stream)
        decode(caches[n], seqs, q_rot[n][:, None], 0.08, mod, None, None, pg.max_pages, out[n], ws[n], stream=stream)

    step(0)
    step(1)
    torch.cuda.synchronize()
    first = [x.clone() for x in out]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for n in (0, 1):
            step(n, streams[n])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, out))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(0)
        step(1)
    for x in out:
        x.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, out))
    # a graph sees the lengths and tables of its replay
    pg.seq_lens[0] = 5
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(first[0][0], out[0][0]) and torch.equal(first[0][1:], out[0][1:])
    assert B.ekv_get_error() == 0


@pytest.mark.parametrize("q4", [False, True])
def test_appends_and_reads_at_the_last_positions(q4):
    """The longest sequence of 32-bit positions (all of its pages one physical page),
    with unused rows behind its token: the items of pages past its end do nothing."""
    d, S, rows, pages = 64, 16, 200, 2 ** 27 - 1
    L = pages * S
    g = torch.Generator(device="cuda").manual_seed(9)
    k, v = (torch.randn(rows, 1, d, generator=g, device="cuda").to(BF) for _ in range(2))
    seqs = B.make_seqs(torch.zeros(1, pages, dtype=torch.int32, device="cuda"),
                       torch.tensor([L], dtype=torch.int32, device="cuda"))
    indptr = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    new = B.make_new_tokens(k, v, indptr=indptr)
    if not q4:
        kp, vp = (torch.zeros(1, 1, S, d, dtype=BF, device="cuda") for _ in range(2))
        c = B.make_cache(kp, vp)
        c.box = c.mom = None
        B.ekv_rope_append(c, seqs, None, new)
        assert torch.equal(kp[0, :, -1], k[0]) and torch.equal(vp[0, :, -1], v[0])
        assert not kp[0, :, :-1].any() and not vp[0, :, :-1].any()
    else:
        pool = torch.zeros(1, 1, 1, 16 * d + 128, dtype=torch.uint8, device="cuda")
        c = B.make_cache_q4(pool, d)
        B.ekv_rope_append_q4(c, seqs, None, new)
        out = [torch.full((rows, 1, d), 7.0, device="cuda") for _ in range(2)]
        B.ekv_q4_read(c, seqs, indptr, *out)
        for got, x in zip(out, (k, v)):
            codes, step, zero = quantise64(np64(x[0, 0]))
            assert (np64(got[0, 0]) == (zero + step * codes).astype(np.float32)).all() and (got[1:] == 7).all()
        codes, step, _ = unpack(pool, d)
        assert not codes[..., :-1, :].any() and not step[..., :-1].any()
    assert B.ekv_get_error() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_q4_codes_of_every_scale(d, dtype):
    """Rows from 1e-36 to 1e37, some far from zero next to their spread: step, zero and
    codes are those of 64 bits, number for number."""
    rows, hkv, S = 16 * 37, 2, 16
    pg = Paged([rows], hkv, d, S, seed=41 + d)
    scale = 10.0 ** torch.linspace(-36, 37, rows, dtype=torch.float64, device="cuda")[:, None, None]
    x = [pg.randn(rows, hkv, d, dtype=torch.float64) for _ in range(2)]
    far = torch.tensor([0.0, 3.0, 200.0, 9e3], dtype=torch.float64, device="cuda")[torch.arange(rows, device="cuda") % 4]
    k, v = ((t / 8 * scale + far[:, None, None] * scale).to(dtype) for t in x)
    k[5::7, 0] = k[5::7, 0, :1]                     # rows of one value
    ok = (k.float().isfinite() & v.float().isfinite()).all()
    if not ok:                                      # 9e3·1e37 is past fp32
        k, v = (t.float().clamp(-3e38, 3e38).to(dtype) for t in (k, v))
    pool = torch.zeros_like(pg.pool_q4())
    seqs = B.make_seqs(pg.table, pg.seq_lens)
    B.ekv_rope_append_q4(B.make_cache_q4(pool, d), seqs, None, B.make_new_tokens(
        k, v, indptr=torch.tensor([0, rows], dtype=torch.int32, device="cuda")))
    assert B.ekv_get_error() == 0
    codes, step, zero = unpack(pool, d)             # [phys, Hkv, tile, K/V, 16, d]
    kv = np64(torch.stack([k, v]))
    for t in range(rows):
        page, slot = int(pg.table_h[0, t // S]), t % S
        for h in range(hkv):
            for i in range(2):
                c, st, z = quantise64(kv[i, t, h])
                at = (page, h, 0, i, slot)
                assert st == step[at] and z == zero[at] and (c == codes[at]).all(), (t, h, i)
