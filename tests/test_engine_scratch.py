"""The engines' masked softmax decode takes its scratch for one call, on the call's
stream (CPU: the streams and the kernel are stand-ins)."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

from sparse_kv_cache_kmax_b200 import binding as B
from sparse_kv_cache_kmax_b200 import engine as E


@pytest.fixture
def calls(monkeypatch):
    """Runs E._softmax on stand-ins; what each call was given, and the stream each buffer was made on."""
    made, on, seen = {}, ["current"], []

    @contextlib.contextmanager
    def stream(s):
        on.append(on[-1] if s is None else s)
        yield
        on.pop()

    def workspace(nbytes, device):
        t = torch.empty(nbytes, dtype=torch.uint8)
        made[t.data_ptr()] = on[-1]
        return t

    empty = torch.empty

    def note(*a, **kw):
        t = empty(*a, **kw)
        made[t.data_ptr()] = on[-1]
        return t

    def kernel(cache, seqs, q, scale, mod, sel, n_sel, cap, out, ws, *, lse, stream):
        seen.append(SimpleNamespace(stream=stream or "current", ws=ws, out=out, lse=lse))

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(B, "workspace", workspace)
    monkeypatch.setattr(B, "ekv_softmax_mod_workspace_bytes", lambda d, hkv, hq, t: 0 if t > 8 else 1024 * t)
    monkeypatch.setattr(torch, "empty", note)
    eng = SimpleNamespace(d=64, Hkv=2, Hq=4, scale=0.1, device="cpu", cache=None, seqs=None, mod_bytes={})

    def run(T, s):
        E._softmax(kernel, eng, torch.zeros(3, T, 4, 64), None, None, 5, {}, s)
        return seen[-1]

    return run, made


def test_scratch_belongs_to_the_calls_stream(calls):
    run, made = calls
    for s in (None, "side", "other", None):
        c = run(2, s)
        for t in (c.ws, c.out, c.lse):
            assert made[t.data_ptr()] == c.stream


def test_no_two_calls_in_flight_share_scratch(calls):
    """On two streams, and on one that is captured into two graphs: nothing is kept from
    one call for the next, so the allocator alone decides when memory is used again."""
    run, _ = calls
    both = [run(2, s) for s in (None, "side", None, "side")]     # all held, as calls in flight are
    assert len({c.ws.data_ptr() for c in both}) == 4
    assert run(3, "side").ws.numel() >= 1024 * 3


def test_unsupported_query_tokens_are_refused_every_time(calls):
    run, _ = calls
    for _ in range(2):
        with pytest.raises(ValueError):
            run(9, None)


def test_the_adaptive_decodes_buffers_belong_to_the_first_calls_stream(monkeypatch):
    on, made = ["current"], []

    @contextlib.contextmanager
    def stream(s):
        on.append(on[-1] if s is None else s)
        yield
        on.pop()

    for name in ("empty", "zeros"):
        def note(*a, make=getattr(torch, name), **kw):
            made.append(on[-1])
            return make(*a, **kw)
        monkeypatch.setattr(torch, name, note)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(B, "ekv_decode_adaptive", lambda *a: 1)
    pools = [torch.randn(4, 1, 16, 64).bfloat16() for _ in range(2)]
    eng = E.DecodeEngine(*pools, torch.arange(4, dtype=torch.int32)[None], torch.tensor([50], dtype=torch.int32), 4, k=2)
    made.clear()
    eng.decode_adaptive(torch.randn(1, 4, 64).bfloat16(), stream="side")
    assert made and set(made) == {"side"}
