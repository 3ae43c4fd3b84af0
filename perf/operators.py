"""The serving operators around the paged cache: their cases, their plain forms
and the calls a user makes of them.

Five operators over one paged layout (page table [B, max_pages], lengths [B],
pools of pages of S tokens):

append     new tokens of every sequence are rotated by their positions and
           written into the K/V pages; the touched pages' metadata is refreshed
append_q4  the same into a cache held in 4 bits; the appended tokens are then
           read back as values
read_q4    whole sequences of a 4-bit cache read back as values
decode     softmax decode with scores capped by a tanh, a bias on distance, a
           window, a prefix and a document start, one to eight query tokens
decode_q4  the same decode over a 4-bit cache

Rotation: pairs (x1, x2) of the first ``rot`` coordinates, (j, j + rot/2) or
(2j, 2j + 1), become (x1 c - x2 s, x2 c + x1 s) with the cosine and sine of the
token's position from a table [positions, rot] (cosines, then sines).

4-bit cache: one uint8 record per 16 tokens of a (page, KV head): the K codes
[16, d/2] (element 2i in the low half of byte i), the V codes [16, d/2], then 16
pairs (step, zero) in bfloat16 for K and 16 for V.  A row x of d numbers (for K
the rotated row, not rounded before) has zero = bf16(min x), step =
bf16((max x - min x) / 15) (0 where that is below 1e-30), codes n =
clamp(round((x - zero) / step), 0, 15), halves to the even code, and stands for
zero + step·n.

Decode: token j is visible to the query at position i when j >= start and
(j < prefix or (j <= i and i - j < window)); its score is
cap·tanh(scale·q·k / cap) - slope·|i - j|.
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------- the cases
def _case(name, op, **kw):
    c = {"name": name, "op": op, "batch": 1, "hkv": 8, "group": 4, "d": 128, "page": 16, "dtype": "bf16",
         "context": 1024, "spread": 0.0, "ragged": 1, "new": 1, "rot": 128, "interleaved": False, "packed": True,
         "pad": 0, "tokens": 1, "cap": 0.0, "slopes": 0, "window": 0, "prefix": 0, "start": 0, "pages": 0}
    c.update(kw)
    return c


def listed():
    return [
        # one new token in each of 64 sequences of a shared pool: every layer of every decode step
        _case("append_decode_b64", "append", batch=64, context=16384, spread=0.75, pad=3),
        # four prompts enter the cache at once, straight from one fused projection's output
        _case("append_prompts_16k", "append", batch=4, context=0, new=4096, spread=0.2),
        # chunks of prompts behind earlier chunks, fp32, partial rotation in neighbouring pairs, odd sizes
        _case("append_chunk_f32", "append", batch=3, hkv=4, group=2, d=64, page=32, dtype="f32", context=3001,
              spread=0.5, new=517, rot=32, interleaved=True, packed=False, pad=5),
        # the same moments of a 4-bit cache: a decode step, and prompts
        _case("append_q4_decode_b64", "append_q4", batch=64, context=16384, spread=0.75),
        _case("append_q4_prompts_8k", "append_q4", batch=2, context=100, new=4096, spread=0.1),
        # sequences leave their 4-bit cache (for another precision, or for the host)
        _case("read_q4_4k", "read_q4", context=4001, dtype="f32"),
        _case("read_q4_b8_16k", "read_q4", batch=8, context=16384, spread=0.5),
        # four proposed tokens checked at once in one short chat: latency, every mask
        _case("decode_verify_2k", "decode", context=2003, tokens=4, cap=50.0, window=1024, prefix=64, start=7),
        # many sequences of a scattered pool, bias on distance
        _case("decode_bias_b64", "decode", batch=64, context=16384, spread=0.75, slopes=1),
        # long contexts of four sequences, capped scores: the whole cache is read
        _case("decode_cap_128k", "decode", batch=4, context=131072, cap=30.0),
        # 4 bits: pages picked for each KV head out of long contexts, and the whole of them
        _case("decode_q4_pages_128k", "decode_q4", batch=4, context=131072, pages=256, cap=50.0),
        _case("decode_q4_128k", "decode_q4", batch=4, context=131072, slopes=1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["append", "append_q4", "read_q4", "decode", "decode_q4"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 16, 32])
    hkv = rng.choice([1, 2, 4, 8, 8])
    group = rng.choice([1, 2, 4, 4, 8, 16])
    c = _case("", op, d=d, page=page, hkv=hkv, group=group, ragged=rng.randrange(1, 1 << 20), spread=rng.random(),
              rot=rng.choice([d, d, d // 2, 32]), interleaved=rng.random() < 0.3, packed=rng.random() < 0.6)
    del c["name"]
    if op in ("append", "append_q4"):
        c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
        c["pad"] = rng.choice([0, 0, 1, 17])
        if rng.random() < 0.5:
            c["batch"], c["new"] = _log_int(rng, 1, 128), 1
            c["context"] = _log_int(rng, 1, max(1, min(16384, 786432 // c["batch"])))
        else:
            c["batch"] = _log_int(rng, 1, 8)
            c["group"] = rng.choice([1, 2, 4])
            c["new"] = _log_int(rng, 2, 8192 // c["batch"])
            c["context"] = rng.choice([0, _log_int(rng, 1, 8192)])
    elif op == "read_q4":
        c["dtype"] = rng.choice(["bf16", "f32"])
        c["batch"] = _log_int(rng, 1, 32)
        c["context"] = _log_int(rng, 1, 65536 // c["batch"])
    else:
        c["batch"] = _log_int(rng, 1, 64)
        c["context"] = _log_int(rng, 1, 262144 // c["batch"])
        c["tokens"] = rng.choice([1, 1, 1, 1, 2, 3, 4])
        c["cap"] = rng.choice([0.0, 30.0, 50.0])
        c["slopes"] = rng.choice([0, 0, 1])
        if rng.random() < 0.4:
            c["window"] = _log_int(rng, 1, max(1, c["context"]))
            c["prefix"] = rng.choice([0, _log_int(rng, 1, max(1, c["context"] // 4))])
        if rng.random() < 0.3:
            c["start"] = _log_int(rng, 1, max(1, c["context"] // 2))
        if rng.random() < 0.3:
            c["pages"] = _log_int(rng, 1, 512)
    return c


def _lens(c):
    """[(length with the new tokens, new tokens)] of the case's sequences."""
    r = random.Random(c["ragged"])
    u = [(0.0, 0.0)] + [(r.random(), r.random()) for _ in range(c["batch"] - 1)]
    grow = c["op"] in ("append", "append_q4")
    new = [max(1, round(c["new"] * (1 - c["spread"] * y))) if grow else 0 for _, y in u]
    old = [round(c["context"] * (1 - c["spread"] * x)) for x, _ in u]
    return [(max(o + n, 1), n) for o, n in zip(old, new)]


def _dtype(c):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[c["dtype"]]


def _q4_bytes(d):
    return 16 * d + 128  # one record: 16 tokens, K and V


# ---------------------------------------------------------------- the inputs
def _rope_table(positions, rot, device):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    ang = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    lens = _lens(c)
    B, Hkv, G, d, S = c["batch"], c["hkv"], c["group"], c["d"], c["page"]
    Hq = Hkv * G
    pages = [-(-L // S) for L, _ in lens]
    P, n_phys = max(pages), sum(pages) + 3
    perm = torch.randperm(n_phys, generator=g, device=dev).int()
    table = torch.zeros(B, P, dtype=torch.int32, device=dev)
    mine = torch.arange(P, device=dev)[None] < torch.tensor(pages, device=dev)[:, None]
    table[mine] = perm[: sum(pages)]
    s = {"case": c, "table": table, "lens": torch.tensor([L for L, _ in lens], dtype=torch.int32, device=dev),
         "max_pages": P, "scale": d ** -0.5}
    q4 = c["op"].endswith("q4")
    dt = torch.bfloat16 if c["op"].startswith("decode") else _dtype(c)
    randn = lambda *shape, dtype=dt: torch.randn(*shape, generator=g, device=dev, dtype=dtype)  # noqa: E731
    if q4:
        pool = torch.randint(0, 256, (n_phys, Hkv, S // 16, _q4_bytes(d)), generator=g, device=dev, dtype=torch.uint8)
        sz = torch.empty(n_phys, Hkv, S // 16, 32, 2, device=dev)
        sz[..., 0] = 0.25 + 0.2 * torch.rand(n_phys, Hkv, S // 16, 32, generator=g, device=dev)
        sz[..., 1] = -8.0 * sz[..., 0] + 0.3 * torch.randn(n_phys, Hkv, S // 16, 32, generator=g, device=dev)
        pool[..., 16 * d:] = sz.bfloat16().view(n_phys, Hkv, S // 16, 64).view(torch.uint8)
        s["pool"] = pool
    else:
        s["k_pool"], s["v_pool"] = randn(n_phys, Hkv, S, d), randn(n_phys, Hkv, S, d)
    if c["op"].startswith("append"):
        meta = torch.bfloat16 if q4 else dt
        s["box"] = torch.zeros(Hkv, n_phys, 2, d, dtype=meta, device=dev)
        s["mom"] = torch.zeros_like(s["box"])
        N = sum(n for _, n in lens)
        rows = N + c["pad"]
        if c["packed"]:
            qkv = randn(rows, Hq + 2 * Hkv, d)
            s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        else:
            s["q"], s["k"], s["v"] = randn(rows, Hq, d), randn(rows, Hkv, d), randn(rows, Hkv, d)
        s["q_out"] = torch.zeros(rows, Hq, d, dtype=dt, device=dev)
        s["cos_sin"] = _rope_table(max(L for L, _ in lens), c["rot"], dev)
    if c["op"].startswith("append") or c["op"] == "read_q4":
        counts = [n if c["op"] != "read_q4" else L for L, n in lens]
        s["total"] = sum(counts)
        s["indptr"] = torch.tensor([0] + counts, device=dev).cumsum(0).int()
    if q4 and not c["op"].startswith("decode"):
        out = torch.float32 if c["op"] == "append_q4" else dt
        s["k_read"] = torch.zeros(s["total"], Hkv, d, dtype=out, device=dev)
        s["v_read"] = torch.zeros_like(s["k_read"])
    if c["op"].startswith("decode"):
        T = c["tokens"]
        s["q"] = randn(B, T, Hq, d)
        s["out"] = torch.zeros(B, T, Hq, d, device=dev)
        s["lse"] = torch.zeros(B, T, Hq, device=dev)
        full = lambda x: torch.full((B,), x, dtype=torch.int32, device=dev)  # noqa: E731
        s["slopes"] = (0.5 ** (8.0 * (1 + torch.arange(Hq, device=dev)) / Hq)).float() if c["slopes"] else None
        s["prefix"] = full(c["prefix"]) if c["prefix"] else None
        s["start"] = full(c["start"]) if c["start"] else None
        s["sel"] = s["n_sel"] = None
        if c["pages"]:
            k = min(c["pages"], P)
            r = torch.rand(B, Hkv, P, generator=g, device=dev).masked_fill(~mine[:, None], 2.0)
            idx = r.topk(k, largest=False).indices
            idx = idx.masked_fill(r.gather(2, idx) > 1, P).sort(-1).values
            s["sel"] = idx.masked_fill(idx == P, 0).int().contiguous()
            s["n_sel"] = (idx < P).sum(-1).int()
    return s


# ---------------------------------------------------------------- the plain forms
def _rotate(x, cs, rot, interleaved):
    """x [rows, heads, d], cs [rows, rot]."""
    c, s = cs[:, None, : rot // 2], cs[:, None, rot // 2:]
    x1, x2 = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., : rot // 2], x[..., rot // 2: rot])
    y1, y2 = x1 * c - x2 * s, x2 * c + x1 * s
    y = torch.stack([y1, y2], -1).flatten(-2) if interleaved else torch.cat([y1, y2], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _rows(s):
    """The cache position of every row that indptr counts: (sequence, position, physical page, slot)."""
    S = s["case"]["page"]
    n = s["indptr"].diff().long()
    b = torch.repeat_interleave(torch.arange(n.numel(), device=n.device), n)
    pos = torch.arange(b.numel(), device=n.device) - s["indptr"][b] + s["lens"][b] - n[b]
    return b, pos, s["table"][b, pos // S].long(), pos % S


def _touched(s):
    """Pages that the new tokens touch: (physical page, valid tokens)."""
    S = s["case"]["page"]
    L, n = s["lens"].long(), s["indptr"].diff().long()
    page = torch.arange(s["max_pages"], device=L.device)[None]
    hit = (page >= ((L - n) // S)[:, None]) & (page * S < L[:, None]) & (n > 0)[:, None]
    return s["table"][hit].long(), (L[:, None] - page * S).clamp(max=S)[hit]


def _away(x, up):
    """fp32 -> bf16, toward +inf (up) or -inf."""
    bits = x.contiguous().view(torch.int32)
    grow = (bits >= 0) if up else (bits < 0)
    bits = torch.where(grow, bits + 0xFFFF, bits)
    return (bits & -65536).view(torch.float32).bfloat16()


def _write_meta(s, keys, phys, n, outward):
    """keys [touched, Hkv, S, d] as the cache holds them; box and moments over the first n of each page."""
    ok = (torch.arange(keys.shape[2], device=n.device)[None] < n[:, None])[:, None, :, None]
    mx = keys.masked_fill(~ok, -math.inf).amax(2)
    mn = keys.masked_fill(~ok, math.inf).amin(2)
    k64, m = keys.double().masked_fill(~ok, 0.0), n[:, None, None].double()
    mean = k64.sum(2) / m
    var = ((k64 - mean[:, :, None]).square() * ok).sum(2) / m
    dt = s["box"].dtype
    box = torch.stack([_away(mx, True), _away(mn, False)] if outward else [mx.to(dt), mn.to(dt)], 2)
    s["box"][:, phys] = box.transpose(0, 1)
    s["mom"][:, phys] = torch.stack([mean, var], 2).to(dt).transpose(0, 1)


def _plain_rotated(s, dtype):
    c = s["case"]
    N = s["total"]
    cs = s["cos_sin"][_rows(s)[1]]
    turn = lambda x, t: _rotate(x[:N].to(t), cs.to(t), c["rot"], c["interleaved"])  # noqa: E731
    s["q_out"][:N] = turn(s["q"], torch.float32).to(s["q_out"].dtype)
    return turn(s["k"], dtype), s["v"][:N].to(dtype)


def _plain_append(s):
    k, v = _plain_rotated(s, torch.float32)
    _, _, phys, slot = _rows(s)
    s["k_pool"][phys, :, slot] = k.to(s["k_pool"].dtype)
    s["v_pool"][phys, :, slot] = v.to(s["v_pool"].dtype)
    page, n = _touched(s)
    _write_meta(s, s["k_pool"][page].float(), page, n, False)


def _quantise(x):
    """Rows of d numbers (64 bits) -> codes (uint8), (step, zero) in bf16."""
    mn, mx = x.amin(-1), x.amax(-1)
    step, zero = ((mx - mn) / 15).bfloat16(), mn.bfloat16()
    step = step.masked_fill(step < 1e-30, 0.0)
    by = step.double().masked_fill(step == 0, math.inf)
    codes = ((x - zero.double()[..., None]) / by[..., None]).round().clamp(0, 15).to(torch.uint8)
    return codes, torch.stack([step, zero], -1)


def _plain_append_q4(s):
    c, S, d = s["case"], s["case"]["page"], s["case"]["d"]
    k, v = _plain_rotated(s, torch.float64)  # values next to a border between two codes
    _, _, phys, slot = _rows(s)
    rec = s["pool"]
    tile, r = slot // 16, slot % 16
    for_k, for_v = _quantise(k), _quantise(v)
    codes = rec[..., : 16 * d].view(*rec.shape[:3], 32, d // 2)
    sz = rec[..., 16 * d:].view(*rec.shape[:3], 32, 4)
    codes[phys, :, tile, r] = for_k[0][..., 0::2] | (for_k[0][..., 1::2] << 4)
    codes[phys, :, tile, 16 + r] = for_v[0][..., 0::2] | (for_v[0][..., 1::2] << 4)
    sz[phys, :, tile, r] = for_k[1].view(torch.uint8)
    sz[phys, :, tile, 16 + r] = for_v[1].view(torch.uint8)
    page, n = _touched(s)
    _write_meta(s, _q4_values(rec[page], d)[0], page, n, True)


def _q4_values(rec, d):
    """Records [..., Hkv, S/16, R] -> K and V [..., Hkv, S, d] in fp32."""
    codes = rec[..., : 16 * d].unflatten(-1, (32, d // 2))
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    sz = rec[..., 16 * d:].contiguous().view(torch.bfloat16).unflatten(-1, (32, 2)).float()
    x = (sz[..., 1:].double() + sz[..., :1].double() * n).float()
    return x[..., :16, :].flatten(-3, -2), x[..., 16:, :].flatten(-3, -2)


def _plain_read_q4(s):
    _, _, phys, slot = _rows(s)
    d = s["case"]["d"]
    rec = s["pool"][phys, :, slot // 16]                       # [rows, Hkv, R]
    r, rows = slot % 16, torch.arange(slot.numel(), device=slot.device)
    codes = rec[..., : 16 * d].unflatten(-1, (32, d // 2))
    sz = rec[..., 16 * d:].contiguous().view(torch.bfloat16).unflatten(-1, (32, 2))
    pick = lambda x, at: x[rows, :, at]  # noqa: E731
    value = lambda at: (pick(sz, at)[..., 1:].double() + pick(sz, at)[..., :1].double() * torch.stack(  # noqa: E731
        [pick(codes, at) & 15, pick(codes, at) >> 4], -1).flatten(-2)).float()
    s["k_read"].copy_(value(r))
    s["v_read"].copy_(value(16 + r))


def _plain_decode(s):
    c = s["case"]
    B, T, Hkv, G, d, S = c["batch"], c["tokens"], c["hkv"], c["group"], c["d"], c["page"]
    dev = s["lens"].device
    L = s["lens"].long()
    if s["sel"] is None:
        page = torch.arange(s["max_pages"], device=dev).expand(B, 1, -1)
        phys = s["table"].long()[:, None]
        held = page * S < L[:, None, None]
    else:
        page = s["sel"].long()
        phys = s["table"].long()[:, None].expand(-1, Hkv, -1).gather(2, page)
        held = torch.arange(page.shape[-1], device=dev) < s["n_sel"][..., None]
    head = torch.arange(Hkv, device=dev)[:, None]
    if c["op"] == "decode":
        K, V = (s[x][phys, head].flatten(2, 3).float() for x in ("k_pool", "v_pool"))
    else:
        K, V = (x.flatten(2, 3) for x in _q4_values(s["pool"][phys, head], d))
    j = (page[..., None] * S + torch.arange(S, device=dev)).flatten(2)           # [B, 1 or Hkv, N]
    held = held.repeat_interleave(S, -1) & (j < L[:, None, None])
    q = s["q"].float().view(B, T, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, d)
    z = (q @ K.transpose(2, 3)).view(B, Hkv, G, T, -1) * s["scale"]
    if c["cap"]:
        z = c["cap"] * torch.tanh(z / c["cap"])
    i = (L[:, None] - T + torch.arange(T, device=dev))[:, None, :, None]          # [B, 1, T, 1]
    gap = i - j[:, :, None]                                                       # [B, 1 or Hkv, T, N]
    seen = gap >= 0
    if c["window"]:
        seen = seen & (gap < c["window"])
    if s["prefix"] is not None:
        seen = seen | (j < s["prefix"][:, None, None])[:, :, None]
    if s["start"] is not None:
        seen = seen & (j >= s["start"][:, None, None])[:, :, None]
    seen = seen & held[:, :, None] & (i >= 0)
    if s["slopes"] is not None:  # far positions: the bias passes what 32 bits hold to a unit
        z = z.double() - s["slopes"].double().view(1, Hkv, G, 1, 1) * gap.abs()[:, :, None]
    z = z.masked_fill(~seen[:, :, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    w = (z - m.clamp(min=-1e30)).float().exp()
    den = w.sum(-1)
    o = (w.flatten(2, 3) @ V).view(B, Hkv, G, T, d) / den.clamp(min=1e-30)[..., None]
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(B, T, Hkv * G, d))
    s["lse"].copy_((m[..., 0] + den.log()).permute(0, 3, 1, 2).reshape(B, T, Hkv * G))


# ---------------------------------------------------------------- the framework's calls
def _handles(s):
    """What a user's program makes once: descriptions of the cache, the batch and the call."""
    from sparse_kv_cache_kmax_b200 import binding as Bd

    c = s["case"]
    h = {"Bd": Bd, "seqs": Bd.make_seqs(s["table"], s["lens"])}
    if c["op"].endswith("q4"):
        h["cache"] = Bd.make_cache_q4(s["pool"], c["d"], s.get("box"), s.get("mom"))
    else:
        h["cache"] = Bd.make_cache(s["k_pool"], s["v_pool"], s.get("box"), s.get("mom"))
    if c["op"].startswith("append"):
        h["rope"] = Bd.make_rope(s["cos_sin"], interleaved=c["interleaved"])
        one = c["new"] == 1
        h["new"] = Bd.make_new_tokens(s["k"], s["v"], s["q"], s["q_out"], indptr=None if one else s["indptr"])
    if c["op"].startswith("decode"):
        h["mod"] = Bd.make_score_mod(softcap=c["cap"], slopes=s["slopes"], window=c["window"],
                                     prefix_lens=s["prefix"], starts=s["start"])
        h["ws"] = Bd.workspace(Bd.ekv_softmax_mod_workspace_bytes(c["d"], c["hkv"], c["hkv"] * c["group"],
                                                                  c["tokens"]), s["q"].device)
        h["cap"] = s["max_pages"] if s["sel"] is None else s["sel"].shape[-1]
    return h


def _own(s):
    h = s.get("handles")
    if h is None:
        h = s["handles"] = _handles(s)
    Bd, op = h["Bd"], s["case"]["op"]
    if op == "append":
        Bd.ekv_rope_append(h["cache"], h["seqs"], h["rope"], h["new"])
    elif op == "append_q4":
        Bd.ekv_rope_append_q4(h["cache"], h["seqs"], h["rope"], h["new"])
        Bd.ekv_q4_read(h["cache"], h["seqs"], s["indptr"], s["k_read"], s["v_read"])
    elif op == "read_q4":
        Bd.ekv_q4_read(h["cache"], h["seqs"], s["indptr"], s["k_read"], s["v_read"])
    elif op == "decode":
        Bd.ekv_softmax_decode_mod(h["cache"], h["seqs"], s["q"], s["scale"], h["mod"], s["sel"], s["n_sel"], h["cap"],
                                  s["out"], h["ws"], lse=s["lse"])
    else:
        Bd.ekv_softmax_decode_q4(h["cache"], h["seqs"], s["q"], s["scale"], h["mod"], s["sel"], s["n_sel"], h["cap"],
                                 s["out"], h["ws"], lse=s["lse"])


_PLAIN = {"append": _plain_append, "append_q4": lambda s: (_plain_append_q4(s), _plain_read_q4(s)),
          "read_q4": _plain_read_q4, "decode": _plain_decode, "decode_q4": _plain_decode}
_RETURNS = {"append": ("q_out", "k_pool", "v_pool", "box", "mom"), "append_q4": ("q_out", "k_read", "v_read", "box", "mom"),
            "read_q4": ("k_read", "v_read"), "decode": ("out", "lse"), "decode_q4": ("out", "lse")}


def run(state):
    op = state["case"]["op"]
    if own:
        _own(state)
    else:
        _PLAIN[op](state)
    return {x: state[x] for x in _RETURNS[op]}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    lens = _lens(c)
    B, Hkv, G, d, S, T = c["batch"], c["hkv"], c["group"], c["d"], c["page"], c["tokens"]
    Hq = Hkv * G
    el = 2 if c["dtype"] == "bf16" else 4
    q4_row = d + 8                                        # K and V codes of one (token, KV head), with their pairs
    if c["op"].startswith("append"):
        N = sum(n for _, n in lens)
        touched = sum(-(-L // S) - (L - n) // S for L, n in lens)
        before = sum((L - n) % S for L, n in lens)        # tokens already in the touched pages
        bytes_ = N * (Hq + 2 * Hkv) * d * el + N * Hq * d * el + N * c["rot"] * 4
        q4 = c["op"] == "append_q4"
        bytes_ += N * Hkv * (q4_row if q4 else 2 * d * el)
        bytes_ += before * Hkv * (d // 2 + 4 if q4 else d * el) + touched * (Hkv * 4 * d * (2 if q4 else el) + 4)
        if q4:
            bytes_ += N * Hkv * (q4_row + 2 * d * 4)
        return {"bytes": bytes_, "flops": N * (Hq + Hkv) * c["rot"] * 3 + (N + before) * Hkv * d * 6}
    if c["op"] == "read_q4":
        N = sum(L for L, _ in lens)
        return {"bytes": N * Hkv * (q4_row + 2 * d * el), "flops": N * Hkv * d * 4}
    if c["pages"]:
        seen = sum(min(c["pages"] * S, L) for L, _ in lens)
    else:
        lo = [max(0, L - T - c["window"] + 1) if c["window"] else 0 for L, _ in lens]
        seen = sum(max(0, L - max(a, c["start"])) + max(0, min(c["prefix"], a) - c["start"]) for (L, _), a in zip(lens, lo))
    row = q4_row if c["op"] == "decode_q4" else 4 * d
    bytes_ = seen * Hkv * row + -(-seen // S) * 4 + B * T * Hq * (d * 2 + d * 4 + 4)
    return {"bytes": bytes_, "flops": seen * Hq * T * d * 4}


# ---------------------------------------------------------------- the definition, in 64 bits
def _exact_turn(x, pos, rot, interleaved, table):
    y = x.double().clone()
    half = rot // 2
    a = [2 * j for j in range(half)] if interleaved else list(range(half))
    b = [2 * j + 1 for j in range(half)] if interleaved else list(range(half, rot))
    z = torch.complex(x[..., a].double(), x[..., b].double()) * torch.complex(
        table[pos, :half].double(), table[pos, half:].double())[:, None]
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_row16(x):
    """The values that rows of d numbers stand for in 4 bits."""
    lo, hi = x.min(-1).values, x.max(-1).values
    step = ((hi - lo) / 15).to(torch.bfloat16).double()
    zero = lo.to(torch.bfloat16).double()
    n = torch.where(step[..., None] > 1e-30, torch.round((x - zero[..., None]) / step[..., None]), 0.0 * x).clamp(0, 15)
    return zero[..., None] + step[..., None] * n


def _exact_unpack(rec, d):
    """[..., R] uint8 -> K, V [..., 16, d] in 64 bits."""
    sz = rec[..., 16 * d:].contiguous().view(torch.bfloat16).double().unflatten(-1, (2, 16, 2))
    both = rec[..., : 16 * d].unflatten(-1, (2, 16, d // 2))
    x = torch.empty(*both.shape[:-1], d, dtype=torch.float64, device=rec.device)
    x[..., 0::2], x[..., 1::2] = both % 16, both // 16
    x = x * sz[..., :1] + sz[..., 1:]
    return x[..., 0, :, :], x[..., 1, :, :]


def _exact_append(s, lens):
    c, S = s["case"], s["case"]["page"]
    q4 = c["op"] == "append_q4"
    q_out = torch.zeros_like(s["q_out"], dtype=torch.float64)
    box, mom = s["box"].double(), s["mom"].double()
    if q4:
        k_read, v_read = s["k_read"].double(), s["v_read"].double()
    else:
        kp, vp = s["k_pool"].double(), s["v_pool"].double()
    at = 0
    for b, (L, n) in enumerate(lens):
        pos = torch.arange(L - n, L, device=q_out.device)
        rows = slice(at, at + n)
        turn = lambda x: _exact_turn(x[rows], pos, c["rot"], c["interleaved"], s["cos_sin"])  # noqa: B023, E731
        q_out[rows] = turn(s["q"])
        k, v = turn(s["k"]), s["v"][rows].double()
        first = (L - n) // S
        ids = s["table"][b, first: -(-L // S)].long()
        old = L - n - first * S
        if q4:
            k, v = _exact_row16(k), _exact_row16(v)
            k_read[rows], v_read[rows] = k, v
            keys = _exact_unpack(s["pool"][ids], c["d"])[0].flatten(2, 3).transpose(1, 2).reshape(-1, c["hkv"], c["d"])
        else:
            keys = kp[ids].transpose(1, 2).reshape(-1, c["hkv"], c["d"])
            vals = vp[ids].transpose(1, 2).reshape(-1, c["hkv"], c["d"])
            vals[old: old + n] = v
            vp[ids] = vals.unflatten(0, (-1, S)).transpose(1, 2)
        keys[old: old + n] = k
        if not q4:
            kp[ids] = keys.unflatten(0, (-1, S)).transpose(1, 2)
            keys[old: old + n] = k.to(s["k_pool"].dtype).double()  # metadata is of the keys as the cache holds them
        for p in range(ids.numel()):
            part = keys[p * S: min((p + 1) * S, old + n)]
            box[:, ids[p], 0], box[:, ids[p], 1] = part.max(0).values, part.min(0).values
            mom[:, ids[p], 0], mom[:, ids[p], 1] = part.mean(0), part.var(0, unbiased=False)
        at += n
    if q4:
        return {"q_out": q_out, "k_read": k_read, "v_read": v_read, "box": box, "mom": mom}
    return {"q_out": q_out, "k_pool": kp, "v_pool": vp, "box": box, "mom": mom}


def _exact_read(s, lens):
    c = s["case"]
    k, v = s["k_read"].double(), s["v_read"].double()
    at = 0
    for b, (L, _) in enumerate(lens):
        both = _exact_unpack(s["pool"][s["table"][b, : -(-L // c["page"])].long()], c["d"])
        for to, x in zip((k, v), both):
            to[at: at + L] = x.flatten(2, 3).transpose(1, 2).reshape(-1, c["hkv"], c["d"])[:L]
        at += L
    return {"k_read": k, "v_read": v}


def _exact_decode(s, lens):
    c = s["case"]
    S, T, G, d = c["page"], c["tokens"], c["group"], c["d"]
    dev = s["q"].device
    out = torch.zeros_like(s["out"], dtype=torch.float64)
    lse = torch.zeros_like(s["lse"], dtype=torch.float64)
    for b, (L, _) in enumerate(lens):
        for h in range(c["hkv"]):
            pages = torch.arange(-(-L // S), device=dev) if s["sel"] is None else s["sel"][b, h, : int(s["n_sel"][b, h])].long()
            ids = s["table"][b, pages].long()
            if c["op"] == "decode":
                K, V = s["k_pool"][ids, h].double(), s["v_pool"][ids, h].double()
            else:
                K, V = _exact_unpack(s["pool"][ids, h], d)
            K, V = K.reshape(-1, d), V.reshape(-1, d)
            j = (pages[:, None] * S + torch.arange(S, device=dev)).reshape(-1)
            K, V, j = K[j < L], V[j < L], j[j < L]
            for t in range(T):
                i = L - T + t
                see = (j <= i) & ((i - j < c["window"]) if c["window"] else True) | (j < c["prefix"])
                see = see & (j >= c["start"]) & (i >= 0)
                z = s["q"][b, t, h * G: (h + 1) * G].double() @ K[see].T * s["scale"]
                z = c["cap"] * torch.tanh(z / c["cap"]) if c["cap"] else z
                if s["slopes"] is not None:
                    z = z - s["slopes"][h * G: (h + 1) * G, None].double() * (i - j[see]).abs()
                lse[b, t, h * G: (h + 1) * G] = torch.logsumexp(z, -1)
                if bool(see.any()):
                    out[b, t, h * G: (h + 1) * G] = torch.softmax(z, -1) @ V[see]
    return {"out": out, "lse": lse}


def exact(case, seed):
    s, lens = prepare(case, seed), _lens(case)
    if case["op"].startswith("append"):
        return _exact_append(s, lens)
    return _exact_read(s, lens) if case["op"] == "read_q4" else _exact_decode(s, lens)
