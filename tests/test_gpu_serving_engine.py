"""The serving operators as a program uses them together: prompts enter a cache
in chunks, steps follow, selections and checks of several tokens at once, over
a bf16 cache and one held in 4 bits, against 64-bit references of the whole."""
import numpy as np
import pytest
import torch

from sparse_kv_cache_kmax_b200 import binding as B
from sparse_kv_cache_kmax_b200.engine import DecodeEngine, Q4Engine

from serving_helpers import Paged, check_decode, decode64, np64, q4_values, rope_table, rotate64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HKV, G, D = 2, 4, 128
PROMPTS, STEPS = [70, 33, 161], 3


def _program(S, seed):
    """Final lengths, and tokens for chunks of the prompts and for steps."""
    pg = Paged([p + STEPS for p in PROMPTS], HKV, D, S, seed=seed)
    table = rope_table(max(pg.lens), D)
    q, k, v = ([pg.randn(n, h, D) for n in pg.lens] for h in (HKV * G, HKV, HKV))
    return pg, table, q, k, v


def _phases():
    """(length after, new tokens) per sequence: two chunks, then single tokens."""
    first = [p // 2 for p in PROMPTS]
    yield first, first
    yield PROMPTS, [p - f for p, f in zip(PROMPTS, first)]
    for s in range(STEPS):
        yield [p + s + 1 for p in PROMPTS], [1] * len(PROMPTS)


def _rows(x, after, new):
    return torch.cat([t[L - n: L] for t, L, n in zip(x, after, new)])


def _indptr(new):
    return torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")


def _keys64(pg, table, k, lens):
    """The rotated keys of every sequence, 64 bits, not rounded."""
    return [rotate64(np64(x[:L]), np64(table), np.arange(L), False) for x, L in zip(k, lens)]


@pytest.mark.parametrize("S", [16, 32])
def test_rotated_prompts_and_steps_over_a_bf16_cache(S):
    pg, table, q, k, v = _program(S, 500 + S)
    kp, vp = pg.pools()
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    eng = DecodeEngine(kp, vp, pg.table, lens, HKV * G, policy="topk", k=4, alpha=1.5, cos_sin=table)
    plain = DecodeEngine(kp, vp, pg.table, lens, HKV * G, policy="topk", k=4, alpha=1.5)  # the same pools, no table
    for after, new in _phases():
        lens.copy_(torch.tensor(after, dtype=torch.int32))
        qs, ks, vs = (_rows(x, after, new) for x in (q, k, v))
        if max(new) > 1:
            turned = eng.append(ks, vs, qs, _indptr(new))
            assert turned.shape == qs.shape
            continue
        out = eng.step(qs, ks, vs).clone()
        # the same step from its parts: metadata built afresh, queries rotated by hand
        plain.build_meta()
        q64 = np.concatenate([rotate64(np64(qs[b:b + 1]), np64(table), np.array([after[b] - 1]), False) for b in range(3)])
        turned = torch.tensor(q64, dtype=torch.float32, device="cuda").to(BF)
        again = plain.step(turned)
        assert torch.equal(eng.sel, plain.sel) and torch.allclose(out, again, rtol=2e-2, atol=2e-2)
    assert B.ekv_get_error() == 0
    # the cache holds the rotated keys: one rounding to bf16, and fp32's in the rotation
    keys = _keys64(pg, table, k, pg.lens)
    for b, L in enumerate(pg.lens):
        got = np64(kp[pg.table[b].long()].transpose(1, 2).reshape(-1, HKV, D)[:L])
        size = 2 * np.abs(np64(k[b])).max()
        assert np.abs(got - keys[b]).max() <= 2.0 ** -8 * np.abs(keys[b]).max() + 2.0 ** -22 * size
        assert torch.equal(vp[pg.table[b].long()].transpose(1, 2).reshape(-1, HKV, D)[:L], v[b])
    # the last three tokens checked at once, over what the cache holds, capped and windowed
    T = 3
    qq = torch.stack([x[L - T: L] for x, L in zip(q, pg.lens)])
    out, lse = eng.softmax(qq, softcap=20.0, window=50)
    check_decode(out, lse, decode64(pg, np64(kp), np64(vp), qq, float(np.float32(eng.scale)), cap=20.0, window=50))
    # over the last step's selection
    out, lse = eng.softmax(qq[:, -1:].contiguous(), selected=True)
    check_decode(out, lse, decode64(pg, np64(kp), np64(vp), qq[:, -1:], float(np.float32(eng.scale)),
                                    sel=eng.sel.cpu().numpy(), n_sel=eng.n_sel.cpu().numpy()))
    # the adaptive decode rotates and appends too
    a, _ = eng.decode_adaptive(qs, ks, vs, k0=2)
    full = DecodeEngine(kp, vp, pg.table, lens, HKV * G, policy="full", alpha=1.5)
    assert torch.allclose(a, full.step(turned), rtol=2e-2, atol=2e-2)


@pytest.mark.parametrize("pick", [None, 4])
def test_rotated_prompts_and_steps_over_a_4_bit_cache(pick):
    pg, table, q, k, v = _program(16, 600)
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    pool = Q4Engine.new_pool(pg.n_phys, HKV, 16, D, "cuda")
    eng = Q4Engine(pool, D, pg.table, lens, HKV * G, k=pick, cos_sin=table)
    slopes = torch.tensor(0.5 ** (np.arange(1, HKV * G + 1)), dtype=torch.float32, device="cuda")
    for after, new in _phases():
        lens.copy_(torch.tensor(after, dtype=torch.int32))
        qs, ks, vs = (_rows(x, after, new) for x in (q, k, v))
        if max(new) > 1:
            eng.append(ks, vs, qs, _indptr(new))
            continue
        out, lse = eng.step(qs, ks, vs, softcap=30.0, slopes=slopes)
        now = Paged.__new__(Paged)
        now.__dict__.update(pg.__dict__)
        now.lens, now.pages = after, [-(-L // 16) for L in after]
        q64 = np.concatenate([rotate64(np64(qs[b:b + 1]), np64(table), np.array([after[b] - 1]), False) for b in range(3)])
        turned = torch.tensor(q64, dtype=torch.float32, device="cuda").to(BF)
        K, V = q4_values(pool, D)
        want = decode64(now, K, V, turned[:, None], float(np.float32(eng.scale)), cap=30.0, slopes=slopes.cpu().numpy(),
                        sel=None if pick is None else eng.sel.cpu().numpy(),
                        n_sel=None if pick is None else eng.n_sel.cpu().numpy())
        # the query is rotated in fp32 before its rounding: at most one step of bf16 apart
        off = np.abs(np64(out[:, None]) - want[0]).max()
        assert off <= 0.05 * np.abs(want[0]).max()
        again, _ = eng.softmax(turned[:, None], selected=pick is not None, softcap=30.0, slopes=slopes)
        check_decode(again, _, want)
    # what the cache holds is within half a step of what went in, and of its bf16 parameters' roundings
    total = sum(pg.lens)
    kr, vr = eng.read(_indptr(pg.lens), total, dtype=torch.float32)
    keys = np.concatenate(_keys64(pg, table, k, pg.lens))
    for got, x in ((np64(kr), keys), (np64(vr), np.concatenate([np64(t) for t in v]))):
        span = x.max(-1, keepdims=True) - x.min(-1, keepdims=True)
        room = span / 15 / 2 * (1 + 2.0 ** -8) + 2.0 ** -8 * (np.abs(x).max(-1, keepdims=True) + span)
        assert (np.abs(got - x) <= room).all()
    assert B.ekv_get_error() == 0


def test_engine_refusals():
    pg = Paged([20], 1, 64, 16, seed=1)
    eng = Q4Engine(Q4Engine.new_pool(pg.n_phys, 1, 16, 64, "cuda"), 64, pg.table, pg.seq_lens, 4)
    q = torch.zeros(1, 1, 4, 64, dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        eng.select(q[:, 0])
    with pytest.raises(ValueError):
        eng.softmax(q, selected=True)
    with pytest.raises(ValueError):
        eng.softmax(torch.zeros(1, 17, 4, 64, dtype=BF, device="cuda"))
    with pytest.raises(ValueError):
        eng.softmax(q, slopes=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError):
        eng.append(torch.zeros(1, 2, 64, device="cuda"), torch.zeros(1, 2, 64, device="cuda"))


def test_another_stream_than_the_current_one():
    """What an engine allocates for a call belongs to the call's stream: its zeros come
    before the rows, and nobody gets a rotated q's memory while a step still reads it."""
    pg, table, q, k, v = _program(16, 77)
    lens = torch.tensor(PROMPTS, dtype=torch.int32, device="cuda")
    engines = [Q4Engine(Q4Engine.new_pool(pg.n_phys, HKV, 16, D, "cuda"), D, pg.table, lens, HKV * G, cos_sin=table)
               for _ in range(2)]
    ks, vs, ip = _rows(k, PROMPTS, PROMPTS), _rows(v, PROMPTS, PROMPTS), _indptr(PROMPTS)
    for e in engines:
        e.append(ks, vs, None, ip)
    want = engines[0].read(ip, sum(PROMPTS))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(40_000_000)                     # the current stream is behind
    got = engines[1].read(ip, sum(PROMPTS), stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    after, new = [p + 1 for p in PROMPTS], [1] * len(PROMPTS)
    lens.copy_(torch.tensor(after, dtype=torch.int32))
    qs, k1, v1 = (_rows(x, after, new) for x in (q, k, v))
    out, lse = engines[0].step(qs, k1, v1)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)                 # the step's stream is behind
    out2, lse2 = engines[1].step(qs, k1, v1, stream=side)
    other = [torch.full_like(qs, float("nan")) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and len(other) == 4
    assert B.ekv_get_error() == 0
