"""The serving operators' refusals (CPU): the C entries return a status before
any launch, the binding raises before any call."""
import ctypes

import pytest
import torch

from sparse_kv_cache_kmax_b200 import binding as B

FAKE = 0x1000  # never dereferenced: validation fails before any launch
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def _cache(**kw):
    c = dict(dtype=B.EKV_BF16, head_dim=128, page_size=16, num_kv_heads=8, num_phys_pages=10,
             k_pool=FAKE, v_pool=FAKE, box=FAKE, mom=FAKE)
    c.update(kw)
    return B.Cache(**c)


def _q4(**kw):
    c = dict(head_dim=128, page_size=16, num_kv_heads=8, num_phys_pages=10, pool=FAKE, box=FAKE, mom=FAKE)
    c.update(kw)
    return B.CacheQ4(**c)


def _seqs(**kw):
    s = dict(page_table=FAKE, seq_lens=FAKE, batch=2, max_pages=5)
    s.update(kw)
    return B.Seqs(**s)


def _rope(**kw):
    r = dict(cos_sin=FAKE, max_pos=100, rot_dim=128, interleaved=0)
    r.update(kw)
    return B.Rope(**r)


def _new(**kw):
    n = dict(q=FAKE, k=FAKE, v=FAKE, q_out=2 * FAKE, q_stride=4096, k_stride=1024, v_stride=1024, indptr=FAKE,
             num_tokens=4, num_q_heads=32, dtype=B.EKV_BF16)
    n.update(kw)
    return B.NewTokens(**n)


def _mod(**kw):
    return B.ScoreMod(**kw)


by = ctypes.byref


def _append(cache=None, seqs=None, rope=None, new=None):
    cache = _cache() if cache is None else cache
    fn = B.lib().ekv_rope_append_q4 if isinstance(cache, B.CacheQ4) else B.lib().ekv_rope_append
    return fn(by(cache), by(seqs or _seqs()), by(rope or _rope()), by(new or _new()), None)


APPEND_REFUSALS = [
    (dict(seqs=_seqs(batch=0)), INVALID), (dict(seqs=_seqs(page_table=None)), INVALID),
    (dict(seqs=_seqs(max_pages=2 ** 27)), UNSUPPORTED),                        # positions past 2³¹
    (dict(rope=_rope(cos_sin=None)), INVALID), (dict(rope=_rope(cos_sin=FAKE + 4)), INVALID),
    (dict(rope=_rope(max_pos=0)), INVALID), (dict(rope=_rope(rot_dim=0)), INVALID),
    (dict(rope=_rope(rot_dim=24)), INVALID), (dict(rope=_rope(rot_dim=144)), INVALID),
    (dict(new=_new(k=None)), INVALID), (dict(new=_new(v=None)), INVALID), (dict(new=_new(q_out=None)), INVALID),
    (dict(new=_new(k=FAKE + 8)), INVALID), (dict(new=_new(v_stride=1028)), INVALID),
    (dict(new=_new(k_stride=1016)), INVALID), (dict(new=_new(q_stride=0)), INVALID),
    (dict(new=_new(num_tokens=0)), INVALID), (dict(new=_new(indptr=None, num_tokens=1)), INVALID),
    (dict(new=_new(num_q_heads=12)), INVALID), (dict(new=_new(num_q_heads=24)), UNSUPPORTED),
    (dict(new=_new(q_out=FAKE, q_stride=8192)), INVALID), (dict(new=_new(dtype=5)), UNSUPPORTED),
]


@pytest.mark.parametrize("n", range(len(APPEND_REFUSALS)))
def test_append_refuses(n):
    kw, status = APPEND_REFUSALS[n]
    assert _append(**kw) == status
    assert _append(cache=_q4(), **kw) == status


def test_append_refuses_caches():
    assert _append(cache=_cache(head_dim=96)) == UNSUPPORTED
    assert _append(cache=_cache(page_size=8)) == UNSUPPORTED
    assert _append(cache=_cache(v_pool=None)) == INVALID
    assert _append(cache=_cache(box=None)) == INVALID            # one of the two
    assert _append(cache=_cache(k_pool=FAKE + 8)) == INVALID
    assert _append(new=_new(dtype=B.EKV_F32)) == INVALID          # not the cache's type
    assert _append(cache=_q4(pool=FAKE + 8)) == INVALID
    assert _append(cache=_q4(pool=None)) == INVALID
    assert _append(cache=_q4(mom=None)) == INVALID
    assert _append(cache=_q4(head_dim=80)) == UNSUPPORTED
    L = B.lib()
    assert L.ekv_rope_append(None, by(_seqs()), None, by(_new()), None) == INVALID
    assert L.ekv_rope_append_q4(None, by(_seqs()), None, by(_new()), None) == INVALID
    assert L.ekv_rope_append(by(_cache()), by(_seqs()), None, None, None) == INVALID
    assert L.ekv_rope_append(by(_cache()), None, None, by(_new()), None) == INVALID


def _read(cache=None, seqs=None, indptr=FAKE, n=4, dtype=B.EKV_F32, k=FAKE, v=FAKE):
    return B.lib().ekv_q4_read(by(cache or _q4()), by(seqs or _seqs()), indptr, n, dtype, k, v, None)


def test_read_refuses():
    assert _read(indptr=None) == INVALID and _read(n=0) == INVALID
    assert _read(k=None, v=None) == INVALID and _read(k=FAKE + 4) == INVALID
    assert _read(dtype=3) == UNSUPPORTED and _read(cache=_q4(page_size=64)) == UNSUPPORTED
    assert _read(seqs=_seqs(max_pages=0)) == INVALID and _read(seqs=_seqs(max_pages=2 ** 27)) == UNSUPPORTED
    assert B.lib().ekv_q4_read(None, by(_seqs()), FAKE, 4, 0, FAKE, FAKE, None) == INVALID


def _decode(cache=None, seqs=None, q=FAKE, Hq=32, T=1, scale=0.1, mod=None, sel=None, n_sel=None, cap=5, out=FAKE,
            ws=0x100000, ws_bytes=1 << 40):
    cache = _cache() if cache is None else cache
    fn = B.lib().ekv_softmax_decode_q4 if isinstance(cache, B.CacheQ4) else B.lib().ekv_softmax_decode_mod
    return fn(by(cache), by(seqs or _seqs()), q, Hq, T, scale, None if mod is None else by(mod), sel, n_sel, cap, out,
              None, ws, ws_bytes, None)


DECODE_REFUSALS = [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(q=FAKE + 2), INVALID), (dict(out=FAKE + 4), INVALID),
    (dict(Hq=12), INVALID), (dict(Hq=24), UNSUPPORTED), (dict(Hq=256), UNSUPPORTED),
    (dict(T=0), INVALID), (dict(T=17), UNSUPPORTED), (dict(T=2 ** 30), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(mod=_mod(softcap=-1.0)), INVALID), (dict(mod=_mod(softcap=float("inf"))), INVALID),
    (dict(mod=_mod(softcap=float("nan"))), INVALID), (dict(mod=_mod(window=-1)), INVALID),
    (dict(sel=FAKE), INVALID), (dict(n_sel=FAKE), INVALID), (dict(cap=4), INVALID), (dict(cap=0), INVALID),
    (dict(seqs=_seqs(batch=-1)), INVALID), (dict(seqs=_seqs(max_pages=2 ** 27), cap=2 ** 27), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(ws=0x100010), WORKSPACE), (dict(ws_bytes=1000), WORKSPACE),
]


@pytest.mark.parametrize("n", range(len(DECODE_REFUSALS)))
def test_decode_refuses(n):
    kw, status = DECODE_REFUSALS[n]
    assert _decode(**kw) == status
    assert _decode(cache=_q4(), **kw) == status


def test_decode_refuses_lists_past_32_bits():
    # 32 sequences of 2²⁶ (token tile, KV head) pairs: their number needs 32 bits and a sign
    for cache in (_cache(), _q4()):
        assert _decode(cache=cache, seqs=_seqs(max_pages=2 ** 23), cap=2 ** 23) == UNSUPPORTED
        assert _decode(cache=cache, sel=FAKE, n_sel=FAKE, cap=2 ** 26) == UNSUPPORTED
        # one page less passes this check and meets the next
        assert _decode(cache=cache, seqs=_seqs(max_pages=2 ** 23 - 1), cap=2 ** 23, ws=None) == WORKSPACE
        assert _decode(cache=cache, sel=FAKE, n_sel=FAKE, cap=2 ** 26 - 1, ws=None) == WORKSPACE


def test_decode_refuses_caches():
    assert _decode(cache=_cache(dtype=B.EKV_F32)) == UNSUPPORTED
    assert _decode(cache=_cache(head_dim=256)) == UNSUPPORTED
    assert _decode(cache=_cache(num_phys_pages=2 ** 24 + 1)) == UNSUPPORTED   # rows past 2³¹
    assert _decode(cache=_q4(num_phys_pages=2 ** 24 + 1)) == UNSUPPORTED
    assert _decode(cache=_cache(v_pool=FAKE + 8)) == INVALID
    assert B.lib().ekv_softmax_decode_mod(None, by(_seqs()), FAKE, 32, 1, 0.1, None, None, None, 5, FAKE, None,
                                          0x100000, 1 << 40, None) == INVALID


def test_workspace_bytes():
    size = B.ekv_softmax_mod_workspace_bytes
    assert size(128, 8, 32, 1) > 0 and size(128, 8, 32, 1) % 256 == 0
    assert size(128, 8, 32, 16) > size(128, 8, 32, 1) == size(128, 2, 8, 1)
    assert size(96, 8, 32, 1) == size(128, 8, 12, 1) == size(128, 8, 24, 1) == size(128, 8, 32, 17) == 0
    assert size(128, 0, 32, 1) == size(128, 8, 0, 1) == size(128, 8, 32, 0) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device error path")
def test_valid_calls_without_a_device_report_a_cuda_error():
    assert _append() == _append(cache=_q4()) == _read() == _decode() == _decode(cache=_q4()) == 4


def test_binding_refuses():
    bf = torch.bfloat16
    pool = torch.zeros(3, 2, 1, B.q4_record_bytes(64), dtype=torch.uint8)
    box = torch.zeros(2, 3, 2, 64, dtype=bf)
    B.make_cache_q4(pool, 64, box, box.clone())
    for bad in (lambda: B.make_cache_q4(pool, 128), lambda: B.make_cache_q4(pool.int(), 64),
                lambda: B.make_cache_q4(pool, 64, box), lambda: B.make_cache_q4(pool, 64, box.float(), box.float()),
                lambda: B.make_cache_q4(pool.transpose(0, 1), 64),
                lambda: B.make_rope(torch.zeros(4, 64, dtype=bf)), lambda: B.make_rope(torch.zeros(64)),
                lambda: B.make_score_mod(slopes=torch.zeros(4, dtype=bf)),
                lambda: B.make_score_mod(starts=torch.zeros(4)),
                lambda: B.make_new_tokens(torch.zeros(4, 2, 64), torch.zeros(4, 2, 64, dtype=bf)),
                lambda: B.make_new_tokens(torch.zeros(4, 2, 64), torch.zeros(4, 1, 64)),
                lambda: B.make_new_tokens(torch.zeros(4, 64, 2).transpose(1, 2), torch.zeros(4, 2, 64)),
                lambda: B.make_new_tokens(torch.zeros(4, 2, 64), torch.zeros(4, 2, 64), torch.zeros(4, 8, 64)),
                lambda: B.make_new_tokens(torch.zeros(4, 2, 64), torch.zeros(4, 2, 64),
                                          indptr=torch.zeros(3))):
        with pytest.raises(ValueError):
            bad()
    # another device than the current one, or none
    cache = B.make_cache_q4(pool, 64)
    seqs = B.make_seqs(torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32))
    q = torch.zeros(1, 1, 4, 64, dtype=bf)
    with pytest.raises(ValueError):
        B.ekv_softmax_decode_q4(cache, seqs, q, 0.1, None, None, None, 2, torch.zeros(1, 1, 4, 64),
                                torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError):
        B.ekv_rope_append_q4(cache, seqs, None, B.make_new_tokens(torch.zeros(1, 2, 64), torch.zeros(1, 2, 64)))
    with pytest.raises(ValueError):
        B.ekv_q4_read(cache, seqs, torch.zeros(2, dtype=torch.int32), torch.zeros(1, 2, 64))


def test_descriptions_refuse_strided_tables_and_take_single_rows():
    table = torch.zeros(4, 8, dtype=torch.int32)
    lens = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.make_seqs(table[:, :3], lens)               # a view of a wider table would be read at the wrong places
    with pytest.raises(ValueError):
        B.make_seqs(table, torch.zeros(8, dtype=torch.int32)[::2])
    with pytest.raises(ValueError):
        B.make_seqs(table, torch.zeros(4, dtype=torch.int32, device="meta"))
    assert B.make_seqs(table[:, :8], lens).max_pages == 8
    # one row, or one head: its stride says nothing
    k = torch.zeros(1, 2, 64).as_strided((1, 2, 64), (1, 64, 1))
    n = B.make_new_tokens(k, k, torch.zeros(1, 4, 64), torch.zeros(1, 4, 64))
    assert (n.k_stride, n.v_stride, n.q_stride) == (128, 128, 256)
    one = torch.zeros(3 * 256).as_strided((3, 1, 64), (256, 1, 1))
    assert B.make_new_tokens(one, one).k_stride == 256
    with pytest.raises(ValueError):
        B.make_new_tokens(*[torch.zeros(3 * 256).as_strided((3, 2, 64), (256, 1, 1))] * 2)
