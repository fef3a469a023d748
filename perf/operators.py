"""Timed cases of the operators around a 4-bit paged KV cache.

The operators, in the order a serving or training step meets them:

    rope              rotation of q and k by positions with several axes, and its backward
    kv4_append        K and V rows quantised to 4 bits and written into the pages of a cache
    kv4_read          rows of the cache as bf16 again
    attn_decode_kv4   attention of the newest token(s) of each sequence over the cache
    copy_pages        pages of a pool copied to others (forked sequences, a compacted pool)

run() is one pass through one of them: in elementary torch operations where
`own` is false, through the package where it is true.  prepare() makes the
inputs (the packed cache among them) in the same way for both.

The page format.  A page holds `page` tokens (16, 32, 64, 128 or 256) of every
KV head, head by head, each head's part a run of 16-token tiles.  A group is
32 channels of one token and head; its scale s is bf16, its codes c are in
0..15 and stand for (c - 8) * s.  A tile of 16 tokens x d channels is

    K codes   16 * d / 2 bytes   [tok][t][group][4 bytes]
    V codes   16 * d / 2 bytes   [tok / 8][g][t][group][tok % 2][2 bytes], tok = 8 h + 2 t + (tok % 2)
    K scales  16 * d / 32 bf16   [tok][group]
    V scales  16 * d / 32 bf16   [tok][group]

with channel 32 group + 8 t + n of K in nibble n of its four bytes, and channel
32 group + 4 g + i of V in nibble i of its two bytes (low nibbles first).
Quantisation: s = bf16(m / 7) for the group's largest magnitude m (s = 0 below
m = 2^-100, s = NaN where the group holds an infinity or a NaN), and
c = 8 + floor(x / s + 1/2), limited to 1..15 (c = 8 where s is 0 or NaN).
"""
import math
import random

import numpy as np
import torch

own = False

if torch.cuda.is_available():
    torch.backends.cuda.matmul.allow_tf32 = False


# ------------------------------------------------------------------ cases
def listed():
    return [
        # The rotation before a decode step: one token per sequence, far positions, three axes on one ladder.
        dict(name="rope token", op="rope", way="fwd", B=64, N=1, Hq=32, Hkv=8, d=128, s0=16, s1=24, s2=24, shared=True,
             interleaved=False, far=1000000, dtype="bf16"),
        # A training step of the GPT-2 workload's shape (one axis): forward and backward.
        dict(name="rope gpt2 train", op="rope", way="train", B=8, N=1024, Hq=12, Hkv=12, d=64, s0=32, s1=0, s2=0,
             shared=False, interleaved=False, far=1024, dtype="bf16"),
        # The frame workload: 24 frames of 26 x 40 patches, axes (time, height, width) with a ladder each.
        dict(name="rope frames", op="rope", way="fwd", B=1, N=24960, Hq=24, Hkv=24, d=128, s0=22, s1=21, s2=21,
             shared=False, interleaved=True, far=0, dtype="bf16"),
        # The new token of each sequence written to the cache and read back.
        dict(name="append token", op="append", B=64, N=1, Hkv=8, d=128, page=64, lens=5, lo=1024, hi=8192, ragged=False),
        # A padded batch of prompt chunks of unlike lengths, pages that end inside them.
        dict(name="append chunks d64", op="append", B=7, N=1021, Hkv=12, d=64, page=16, lens=6, lo=1, hi=2500, ragged=True),
        # The long-context prompt written to the cache and read back for a prefill over it.
        dict(name="append prompt", op="append", B=1, N=16384, Hkv=8, d=128, page=64, lens=7, lo=16384, hi=16384,
             ragged=False),
        # One short sequence with as many KV heads as query heads: latency.
        dict(name="decode one d64", op="decode", B=1, Sq=1, Hq=12, Hkv=12, d=64, page=16, lens=1, lo=1000, hi=1000),
        # The decode workload: lengths spread over [1024, 8192].
        dict(name="decode batch", op="decode", B=64, Sq=1, Hq=32, Hkv=8, d=128, page=64, lens=2005, lo=1024, hi=8192),
        # Several tokens at once over a ragged batch; one sequence is shorter than its tokens.
        dict(name="decode tokens", op="decode", B=19, Sq=4, Hq=32, Hkv=8, d=128, page=32, lens=3, lo=2, hi=6000),
        # One very long sequence: the split along the keys and its joining.
        dict(name="decode long", op="decode", B=1, Sq=1, Hq=32, Hkv=8, d=128, page=128, lens=4, lo=524287, hi=524287),
        # The last pages of a few sequences copied as they are forked: latency.
        dict(name="fork pages", op="pages", pages=512, moves=8, Hkv=8, d=128, page=64),
        # A fragmented pool made dense.
        dict(name="compact pool", op="pages", pages=8192, moves=4000, Hkv=8, d=128, page=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "decode", "pages"])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "rope":
        Hkv = rng.choice([1, 2, 3, 4, 5, 8, 12])
        Hq = Hkv * rng.choice([1, 1, 2, 4, 7])
        n = d // 2
        axes = rng.choice([1, 2, 3])
        s0 = rng.randint(1, n) if axes == 1 else rng.randint(1, n // 2)
        s1 = 0 if axes < 2 else rng.randint(1, (n - s0) // 2 or 1)
        s2 = 0 if axes < 3 else rng.randint(1, n - s0 - s1)
        B, way, dtype = rng.choice([1, 2, 3, 8]), rng.choice(["fwd", "train"]), rng.choice(["bf16", "f32"])
        most = 24960 * 48 * 128 // (2 if way == "train" else 1) // (2 if dtype == "f32" else 1)
        N = _log(rng, 1, max(1, most // (B * (Hq + Hkv) * d)))
        return dict(op="rope", way=way, B=B, N=N, Hq=Hq, Hkv=Hkv, d=d, s0=s0, s1=s1, s2=s2,
                    shared=rng.random() < 0.5, interleaved=rng.random() < 0.5, far=_log(rng, 16, 2000000),
                    dtype=dtype)
    if op == "append":
        B = rng.choice([1, 2, 5, 16, 64])
        Hkv = rng.choice([1, 2, 3, 8, 12])
        N = _log(rng, 1, max(1, 16384 * 8 * 128 // (B * Hkv * d)))
        return dict(op="append", B=B, N=N, Hkv=Hkv, d=d, page=page, lens=rng.randint(0, 1 << 20), lo=N if rng.random() < 0.5 else 1,
                    hi=N + _log(rng, 1, 3000), ragged=rng.random() < 0.5)
    if op == "decode":
        B = rng.choice([1, 2, 3, 7, 16, 33])
        Hkv = rng.choice([1, 2, 3, 8])
        G = rng.choice([1, 2, 3, 4, 5, 7, 8])
        Sq = rng.choice([1, 1, 1, 2, 3, 5, 8])
        hi = _log(rng, 16, max(16, 524287 * 8 * 128 // (B * Hkv * d * Sq)))
        return dict(op="decode", B=B, Sq=Sq, Hq=G * Hkv, Hkv=Hkv, d=d, page=page, lens=rng.randint(0, 1 << 20),
                    lo=rng.choice([0, 1, hi // 8]), hi=hi)
    Hkv = rng.choice([1, 2, 5, 8])
    pages = _log(rng, 4, max(4, 8192 * 8 * 64 * 128 // (Hkv * page * d)))
    return dict(op="pages", pages=pages, moves=_log(rng, 1, max(1, pages // 2)), Hkv=Hkv, d=d, page=page)


def _lens(c):
    """The sequences' lengths; the shortest one is there in every batch."""
    r = random.Random(c["lens"])
    return [c["lo"]] * (c["B"] > 1) + [r.randint(c["lo"], c["hi"]) for _ in range(c["B"] - (c["B"] > 1))]


def _new(c, lens):
    """How many tokens each sequence appends: all N, or fewer where the batch is padded."""
    r = random.Random(c["lens"] + 1)
    return [min(n, r.randint(0, c["N"]) if c["ragged"] else c["N"]) for n in lens]


def _sections(c):
    return [s for s in (c["s0"], c["s1"], c["s2"]) if s]


def _row_bytes(d):
    """One token and head in the cache: codes and scales of K and V."""
    return 2 * (d // 2 + d // 32 * 2)


def work(c):
    d = c["d"]
    if c["op"] == "rope":
        e = 2 if c["dtype"] == "bf16" else 4
        x = c["B"] * c["N"] * (c["Hq"] + c["Hkv"]) * d
        passes = 2 if c["way"] == "train" else 1
        return {"bytes": passes * (2 * x * e + 4 * c["B"] * c["N"] * len(_sections(c))), "flops": passes * 3 * x}
    if c["op"] == "append":
        lens = _lens(c)
        n = sum(_new(c, lens)) * c["Hkv"]
        pad = c["B"] * c["N"] * c["Hkv"] * 2 * d * 2  # the rows that the read gives back, padding included
        return {"bytes": n * (2 * d * 2 + 2 * _row_bytes(d)) + pad, "flops": n * 2 * d * 5}
    if c["op"] == "decode":
        n, cols = sum(_lens(c)), c["B"] * c["Sq"] * c["Hq"]
        table = 4 * sum(-(-x // c["page"]) for x in _lens(c))
        return {"bytes": n * c["Hkv"] * _row_bytes(d) + cols * (2 * d * 2 + 4) + table + 4 * c["B"],
                "flops": 4 * d * n * c["Hq"] * c["Sq"]}
    return {"bytes": 2 * c["moves"] * c["page"] * c["Hkv"] * _row_bytes(d), "flops": 0}


# ------------------------------------------------------------------ the page format in torch
def _quant(x):
    """Codes (uint8, 0..15) [..., d] and scales (bf16) [..., d / 32] of x [..., d]."""
    g = x.float().unflatten(-1, (-1, 32))
    m = g.abs().amax(-1)
    s = (m / 7).to(torch.bfloat16)
    s = torch.where(m < 2.0 ** -100, torch.zeros_like(s), s)
    s = torch.where(torch.isfinite(m), s, torch.full_like(s, math.nan))
    sf = s.float()[..., None]
    c = torch.floor(g / sf + 0.5).clamp(-7, 7) + 8
    c = torch.where((sf > 0) & torch.isfinite(sf), c, torch.full_like(c, 8.0))
    return c.to(torch.uint8).flatten(-2), s


def _pack(ck, sk, cv, sv):
    """Tiles [n, Hkv, tile bytes] from codes [n, 16, Hkv, d] and scales [n, 16, Hkv, d / 32]."""
    n, _, H, d = ck.shape
    G = d // 32
    k = ck.view(n, 16, H, G, 4, 4, 2)  # group, t, byte, nibble
    k = (k[..., 0] | (k[..., 1] << 4)).permute(0, 2, 1, 4, 3, 5).reshape(n, H, 8 * d)
    v = cv.view(n, 2, 4, 2, H, G, 8, 2, 2)  # h, t, parity, head, group, g, byte, nibble
    v = (v[..., 0] | (v[..., 1] << 4)).permute(0, 4, 1, 6, 2, 5, 3, 7).reshape(n, H, 8 * d)
    s = [x.permute(0, 2, 1, 3).contiguous().view(torch.uint8).reshape(n, H, 32 * G) for x in (sk, sv)]
    return torch.cat([k, v, *s], -1)


def _unpack(tiles, d):
    """K and V, fp32 [n, 16, Hkv, d], of tiles [n, Hkv, tile bytes]."""
    n, H, _ = tiles.shape
    G = d // 32
    k, v, sk, sv = tiles.split([8 * d, 8 * d, 32 * G, 32 * G], -1)
    k = torch.stack([k & 15, k >> 4], -1).view(n, H, 16, 4, G, 8).permute(0, 2, 1, 4, 3, 5).reshape(n, 16, H, G, 32)
    v = torch.stack([v & 15, v >> 4], -1).view(n, H, 2, 8, 4, G, 2, 4).permute(0, 2, 4, 6, 1, 5, 3, 7)
    v = v.reshape(n, 16, H, G, 32)
    sk, sv = (x.contiguous().view(torch.bfloat16).view(n, H, 16, G, 1).transpose(1, 2).float() for x in (sk, sv))
    return ((k.float() - 8) * sk).flatten(-2), ((v.float() - 8) * sv).flatten(-2)


def _tile_bytes(d):
    return 16 * _row_bytes(d)


def _cache(c, lens, g, room=0):
    """A pool of pages in a random order with stale bytes in them, and the table of its sequences' pages."""
    page, Hkv, d = c["page"], c["Hkv"], c["d"]
    per = [-(-n // page) for n in lens]
    total, width = sum(per), max(1, max(per)) + room
    n_pages = total + 3
    pool = torch.randint(0, 256, (n_pages, Hkv, page // 16 * _tile_bytes(d)), dtype=torch.uint8, device="cuda", generator=g)
    order = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32)
    own_row = torch.tensor([b for b, p in enumerate(per) for _ in range(p)], dtype=torch.long, device="cuda")
    own_col = torch.tensor([j for p in per for j in range(p)], dtype=torch.long, device="cuda")
    table = torch.zeros(len(lens), width, dtype=torch.int32, device="cuda")
    table[own_row, own_col] = order[:total]
    return pool, table, order[:total]


def _rows(shape, g, shift=0.0):
    """Rows of K or V as a layer gives them: normal, with some channels that lie off zero."""
    x = torch.randn(shape, device="cuda", generator=g)
    if shift:
        x += shift * torch.randn(shape[-2:], device="cuda", generator=g)
    return x.to(torch.bfloat16)


# ------------------------------------------------------------------ prepare
def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    s = {"case": c}
    if c["op"] == "rope":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        B, N, d, sec = c["B"], c["N"], c["d"], _sections(c)
        for name, H in (("q", c["Hq"]), ("k", c["Hkv"])):
            s[name] = torch.randn(B, N, H, d, device="cuda", generator=g).to(dt)
            s["d" + name] = torch.randn(B, N, H, d, device="cuda", generator=g).to(dt)
        if c["far"]:
            s["pos"] = torch.randint(0, c["far"], (B, N, len(sec)), dtype=torch.int32, device="cuda", generator=g)
        else:  # frames of 26 x 40 patches, the first frame anywhere in the video
            i = torch.arange(N, device="cuda")
            first = torch.randint(0, 1000, (B, 1, 1), device="cuda", generator=g)
            grid = torch.stack([i // 1040, i % 1040 // 40, i % 40], -1).expand(B, N, 3)
            s["pos"] = (grid + first * torch.tensor([1, 0, 0], device="cuda")).to(torch.int32).contiguous()
        n = d // 2
        axes = np.repeat(np.arange(len(sec)), sec).astype(np.uint8)
        if c["shared"]:
            freq = 10000.0 ** (-np.arange(sum(sec)) / n)
        else:
            freq = np.concatenate([10000.0 ** (-np.arange(m) / m) for m in sec])
        s["axes"], s["freq"] = axes, freq
        return s
    if c["op"] == "append":
        lens = _lens(c)
        new = _new(c, lens)
        pool, table, _ = _cache(c, lens, g)
        s.update(pool=pool, table=table, k=_rows((c["B"], c["N"], c["Hkv"], c["d"]), g, 2.0),
                 v=_rows((c["B"], c["N"], c["Hkv"], c["d"]), g),
                 lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 new=torch.tensor(new, dtype=torch.int32, device="cuda"))
        s["start"] = s["lens"] - s["new"]
        return s
    if c["op"] == "decode":
        lens = _lens(c)
        pool, table, pages = _cache(c, lens, g)
        page, Hkv, d = c["page"], c["Hkv"], c["d"]
        per = max(1, (1 << 26) // (page * Hkv * d))  # pages packed at once
        for i in range(0, len(pages), per):
            p = pages[i:i + per].long()
            shape = (len(p) * page // 16, 16, Hkv, d)
            tiles = _pack(*_quant(_rows(shape, g, 2.0)), *_quant(_rows(shape, g)))
            pool[p] = tiles.view(len(p), page // 16, Hkv, -1).transpose(1, 2).reshape(len(p), Hkv, -1)
        # what lies behind a sequence's end is stale
        q = torch.randn(c["B"], c["Sq"], c["Hq"], d, device="cuda", generator=g).to(torch.bfloat16)
        s.update(pool=pool, table=table, q=q, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        return s
    size = (c["pages"], c["Hkv"], c["page"] // 16 * _tile_bytes(c["d"]))
    s["pool"] = torch.randint(0, 256, size, dtype=torch.uint8, device="cuda", generator=g)
    order = random.Random(seed).sample(range(c["pages"]), 2 * c["moves"])
    s["src"] = np.array(order[:c["moves"]], dtype=np.int32)
    s["dst"] = np.array(order[c["moves"]:], dtype=np.int32)
    return s


# ------------------------------------------------------------------ run
def _rotate(x, pos, axes, freq, interleaved, sign):
    """x [B, N, H, d] rotated pair by pair; pairs behind the table's stay."""
    n, half = len(freq), x.shape[-1] // 2
    ax = torch.from_numpy(axes.astype(np.int64)).to(x.device)
    ang = pos.double()[..., ax] * torch.from_numpy(freq).to(x.device)
    cos, sin = ang.cos().float()[:, :, None], (sign * ang.sin()).float()[:, :, None]
    y = x.float().unflatten(-1, (half, 2) if interleaved else (2, half))
    if not interleaved:
        y = y.transpose(-1, -2)
    a, b = y[..., :n, 0], y[..., :n, 1]
    y = torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1), y[..., n:, :]], -2)
    if not interleaved:
        y = y.transpose(-1, -2)
    return y.flatten(-2).to(x.dtype)


def _where(table, page, pos):
    """(page, 16-token tile of the page) of token positions pos [B, n]."""
    return table.gather(1, (pos // page).long()).long(), (pos % page // 16).long()


def _tiles_of(pool, page):
    """The pool as [pages, tiles of a page, Hkv, tile bytes] (a view)."""
    return pool.unflatten(-1, (page // 16, -1)).transpose(1, 2)


def _plain_append(s):
    c, pool, table = s["case"], s["pool"], s["table"]
    B, N, H, d = s["k"].shape
    G, page = d // 32, c["page"]
    (ck, sk), (cv, sv) = _quant(s["k"]), _quant(s["v"])
    n = torch.arange(N, device=pool.device)
    b, i = torch.nonzero(n[None] < s["new"][:, None], as_tuple=True)
    pos = s["start"].long()[b] + i
    at = table[b, pos // page].long()
    tile, tok = pos % page // 16, pos % 16
    tiles = _tiles_of(pool, page)
    k = ck[b, i].view(-1, H, G, 4, 4, 2)
    tiles[..., :8 * d].unflatten(-1, (16, d // 2))[at, tile, :, tok] = (
        (k[..., 0] | (k[..., 1] << 4)).transpose(2, 3).reshape(-1, H, d // 2))
    v = cv[b, i].view(-1, H, G, 8, 2, 2)
    v = (v[..., 0] | (v[..., 1] << 4)).transpose(2, 3)  # [n, H, g, group, 2]
    tiles[..., 8 * d:16 * d].unflatten(-1, (2, 8, 4, G, 2, 2))[at, tile, :, tok // 8, :, tok % 8 // 2, :, tok % 2] = v
    for x, o in ((sk, 16 * d), (sv, 16 * d + 32 * G)):
        tiles[..., o:o + 32 * G].unflatten(-1, (16, 2 * G))[at, tile, :, tok] = x[b, i].contiguous().view(torch.uint8)
    pos = s["start"][:, None] + n
    live = pos < s["lens"][:, None]
    at, tile = _where(table, page, pos.clamp(max=table.shape[1] * page - 1))
    k, v = _unpack(tiles[at, tile].flatten(0, 1), d)
    row = torch.arange(B * N, device=pool.device)
    tok = (pos % 16).flatten()
    return {x: torch.where(live[..., None, None], y[row, tok].view(B, N, H, d), 0.0).to(torch.bfloat16)
            for x, y in (("k", k), ("v", v))}


def _plain_decode(s):
    c, table = s["case"], s["table"]
    B, Sq, Hq, d = s["q"].shape
    H, L = c["Hkv"], table.shape[1] * c["page"]
    k, v = _unpack(_tiles_of(s["pool"], c["page"])[table.long()].flatten(0, 2), d)
    k, v = k.view(B, L, H, d), v.view(B, L, H, d)
    q = s["q"].float().view(B, Sq, H, Hq // H, d)
    x = torch.einsum("bshgd,blhd->bhgsl", q, k) / math.sqrt(d)
    j = torch.arange(L, device=x.device)
    end = s["lens"][:, None] - Sq + torch.arange(Sq, device=x.device) + 1  # keys that token s sees
    seen = (j < end[..., None])[:, None, None]
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    w = p.sum(-1, keepdim=True)
    v = torch.where((j < s["lens"][:, None])[..., None, None], v, 0.0)
    o = torch.einsum("bhgsl,blhd->bshgd", p / torch.where(w == 0, 1.0, w), v)
    return {"o": o.reshape(B, Sq, Hq, d).to(torch.bfloat16), "lse": (m + torch.log(w))[..., 0].view(B, Hq, Sq)}


def run(s):
    c = s["case"]
    if own:
        return _run_own(s)
    if c["op"] == "rope":
        table = (s["pos"], s["axes"], s["freq"], c["interleaved"])
        r = {"q": _rotate(s["q"], *table, 1), "k": _rotate(s["k"], *table, 1)}
        if c["way"] == "train":  # the rotation's transpose is the rotation back
            r |= {"dq": _rotate(s["dq"], *table, -1), "dk": _rotate(s["dk"], *table, -1)}
        return r
    if c["op"] == "append":
        return _plain_append(s)
    if c["op"] == "decode":
        return _plain_decode(s)
    src, dst = (torch.from_numpy(s[x]).to(s["pool"].device).long() for x in ("src", "dst"))
    s["pool"][dst] = s["pool"][src]
    return s["pool"].view(torch.int32)


def _run_own(s):
    import exact_io_aware_sm_b200 as eio
    c = s["case"]
    if c["op"] == "rope":
        if c["way"] == "fwd":
            q, k = eio.rope(s["q"], s["k"], s["pos"], s["axes"], s["freq"], interleaved=c["interleaved"])
            return {"q": q, "k": k}
        from exact_io_aware_sm_b200.autograd import rope
        q, k = s["q"].detach().requires_grad_(), s["k"].detach().requires_grad_()
        yq, yk = rope(q, k, s["pos"], s["axes"], s["freq"], interleaved=c["interleaved"])
        dq, dk = torch.autograd.grad((yq, yk), (q, k), (s["dq"], s["dk"]))
        return {"q": yq.detach(), "k": yk.detach(), "dq": dq, "dk": dk}
    if c["op"] == "append":
        eio.kv4_append(s["k"], s["v"], s["pool"], s["table"], s["lens"], n_new=s["new"])
        k, v = eio.kv4_read(s["pool"], s["table"], s["lens"], c["N"], c["d"], start=s["start"])
        return {"k": k, "v": v}
    if c["op"] == "decode":
        o, lse = eio.attn_decode_kv4(s["q"], s["pool"], s["table"], s["lens"])
        return {"o": o, "lse": lse}
    eio.copy_pages(s["pool"], s["src"], s["dst"])
    return s["pool"].view(torch.int32)


# ------------------------------------------------------------------ exact
def _places(d):
    """Byte and shift of every code of a tile, and byte of every scale: int64 arrays [16, d] (scales [16, d / 32])."""
    G = d // 32
    t, c = np.meshgrid(np.arange(16), np.arange(d), indexing="ij")
    grp, r = c // 32, c % 32
    kb = t * (d // 2) + (r // 8) * 4 * G + grp * 4 + r % 8 // 2
    vb = 8 * d + (t // 8) * 4 * d + (r // 4) * 16 * G + (t % 8 // 2) * 4 * G + grp * 4 + t % 2 * 2 + r % 4 // 2
    t, j = np.meshgrid(np.arange(16), np.arange(G), indexing="ij")
    ks = 16 * d + 2 * (t * G + j)
    return (kb, r % 2 * 4), (vb, r % 2 * 4), ks, ks + 32 * G


def _values(tiles, codes, scales):
    """fp64 [n, H, 16, d] of one of K and V in tiles [n, H, bytes]."""
    at, shift = (torch.from_numpy(x).to(tiles.device) for x in codes)
    low = torch.from_numpy(scales).to(tiles.device)
    bits = tiles[..., low].to(torch.int32) | (tiles[..., low + 1].to(torch.int32) << 8)
    s = (bits << 16).view(torch.float32).double().repeat_interleave(32, -1)
    return ((tiles[..., at].long() >> shift & 15) - 8).double() * s


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    d = c["d"]
    if c["op"] == "rope":
        half, n = d // 2, len(s["freq"])
        names = [("q", "q", 1.0), ("k", "k", 1.0)] + ([("dq", "dq", -1.0), ("dk", "dk", -1.0)] if c["way"] == "train" else [])
        out = {}
        for name, src, sign in names:
            x = s[src].double()
            y = x.clone()
            for p in range(n):
                i, j = (2 * p, 2 * p + 1) if c["interleaved"] else (p, p + half)
                a = s["pos"][:, :, int(s["axes"][p]), None].double() * float(s["freq"][p])
                y[..., i] = x[..., i] * a.cos() - sign * x[..., j] * a.sin()
                y[..., j] = sign * x[..., i] * a.sin() + x[..., j] * a.cos()
            out[name] = y
        return out
    if c["op"] == "append":
        live = torch.arange(c["N"], device="cuda") < s["new"][:, None]
        out = {}
        for name in ("k", "v"):
            x = s[name].double().reshape(*s[name].shape[:-1], d // 32, 32)
            m = x.abs().max(-1, keepdim=True).values
            step = (m / 7).to(torch.bfloat16).double()
            y = torch.where(step > 0, torch.floor(x / step + 0.5).clamp(-7, 7) * step, 0.0)
            out[name] = torch.where(live[..., None, None], y.reshape(s[name].shape), 0.0)
        return out
    if c["op"] == "decode":
        B, Sq, Hq = c["B"], c["Sq"], c["Hq"]
        H, page = c["Hkv"], c["page"]
        G = Hq // H
        kc, vc, ks, vs = _places(d)
        o = torch.zeros(B, Sq, Hq, d, dtype=torch.float64, device="cuda")
        lse = torch.full((B, Hq, Sq), -math.inf, dtype=torch.float64, device="cuda")
        for b, L in enumerate(_lens(c)):
            if not L:
                continue
            ids = s["table"][b, :-(-L // page)].long()
            for h in range(H):
                tiles = s["pool"][ids, h].reshape(len(ids) * page // 16, 1, -1)
                k = _values(tiles, kc, ks).reshape(-1, d)[:L]
                v = _values(tiles, vc, vs).reshape(-1, d)[:L]
                for i in range(Sq):
                    n = L - Sq + i + 1
                    if n < 1:
                        continue
                    x = s["q"][b, i, h * G:(h + 1) * G].double() @ k[:n].T / math.sqrt(d)
                    lse[b, h * G:(h + 1) * G, i] = torch.logsumexp(x, -1)
                    o[b, i, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v[:n]
        return {"o": o, "lse": lse}
    pool = s["pool"].clone()
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        pool[b] = s["pool"][a]
    return pool.view(torch.int32)
