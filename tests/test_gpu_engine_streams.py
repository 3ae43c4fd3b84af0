"""One engine's masked softmax decodes on two streams, after work that still uses
freed memory, and in two captured graphs: every call computes what it does alone."""
import pytest
import torch

from sparse_kv_cache_kmax_b200 import binding as B
from sparse_kv_cache_kmax_b200.engine import DecodeEngine, Q4Engine

from serving_helpers import Paged

pytestmark = pytest.mark.gpu
HKV, G, D = 2, 4, 128


def _engine(q4, seed, T):
    """An engine over sequences long enough that units are cut, and two sets of queries."""
    pg = Paged([5000, 31, 9000], HKV, D, 16, seed=seed)
    if q4:
        eng = Q4Engine(pg.pool_q4(), D, pg.table, pg.seq_lens, HKV * G)
    else:
        eng = DecodeEngine(*pg.pools(), pg.table, pg.seq_lens, HKV * G, k=4)
    return eng, [pg.randn(3, T, HKV * G, D) for _ in range(2)]


BOTH = pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])


@BOTH
@pytest.mark.parametrize("T", [1, 4])
def test_two_streams_at_once(q4, T):
    eng, qs = _engine(q4, 800 + T, T)
    want = [eng.softmax(q, softcap=30.0) for q in qs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for i in (0, 1):
            got[i].append(eng.softmax(qs[i], softcap=30.0, stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(a, b) for pair in got[i] for a, b in zip(pair, want[i]))
    assert B.ekv_get_error() == 0


@BOTH
def test_the_first_call_on_a_side_stream_leaves_freed_memory_to_its_users(q4):
    eng, (q, _) = _engine(q4, 810, 1)
    want = [x.clone() for x in eng.softmax(q)]
    eng2, (q2, _) = _engine(q4, 810, 1)              # the same inputs, no call so far
    nbytes = B.ekv_softmax_mod_workspace_bytes(D, HKV, HKV * G, 1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    src = [torch.full((nbytes + 256,), n, dtype=torch.uint8, device="cuda") for n in range(8)]
    dst = [torch.empty_like(x) for x in src]
    torch.cuda.synchronize()
    torch.cuda._sleep(40_000_000)                    # the current stream is behind
    for s, d in zip(src, dst):
        t = s.clone()                                # freed at once, its copies still queued
        d.copy_(t)
        del t
    got = eng2.softmax(q2, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(bool((d == n).all()) for n, d in enumerate(dst))
    assert B.ekv_get_error() == 0


@BOTH
def test_two_graphs_replayed_at_once(q4):
    eng, qs = _engine(q4, 820, 1)
    want = [[x.clone() for x in eng.softmax(q, window=4000)] for q in qs]
    graphs, got = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(eng.softmax(q, window=4000))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(30):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eng.softmax(qs[0], softcap=5.0)              # an eager call beside them
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))
    assert B.ekv_get_error() == 0
