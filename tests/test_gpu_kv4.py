"""Rotary positions and the 4-bit paged cache on the GPU against fp64 (kv4_oracle).

Tolerances, from the arithmetic.  A rounding is off by half a step, eps / 2 of the value.
rope: the angle reaches sincospif as an fp32 fraction of a half turn, at most pi * 2^-24
  = 2^-22.3 rad off; sin and cos are off by 2^-22 more, the two products and their sum by
  3 * 2^-24: below 2^-20.6 (|a| + |b|), and the output's rounding.
append: codes and scales are equal bit for bit.  read: equal bit for bit ((c - 8) s has 11
  significant bits, so one rounding from fp32).
decode: p * s (or p) is rounded to bf16 for the product with V, 2^-8 of each term, and so
  is the output.  A score is a sum of d products and d / 32 scaled parts in fp32 (a tensor core
  may drop, not round: 2^-23 of the running sum a step): off by e = (d + 16) 2^-23 sum|q k|
  scale, which moves p and its sum by 2 e; ex2 and the sum of p add 2^-20.  ex2 gives 0
  below 2^-126 and the largest p is at least 1: each weight may be 2^-126 short as well.
  p sv is an fp16 number in units of 2^-6 of a reference, at most 8 times the group's largest
  sv; below 2^-14 half a step is 2^-25: 2^-28 sv, times a code of 7 at most, and 7 sv = max |v|.
"""
import math

import numpy as np
import pytest
import torch

import exact_io_aware_sm_b200 as eio
from exact_io_aware_sm_b200 import autograd
from exact_io_aware_sm_b200.kv4_cache import Kv4Cache, Kv4Full
from tests import kv4_oracle as ko

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built_lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from exact_io_aware_sm_b200 import build
    build.build()


def f64(t):
    return t.detach().double().cpu().numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(shape, seed, dtype=torch.bfloat16, shift=0.0):
    x = np.random.default_rng(seed).standard_normal(shape) + shift
    return torch.from_numpy(x).to(dtype).cuda()


# ------------------------------------------------------------------ rope
ROPE_CASES = [
    # B, N, Hq, Hk, d, pairs of each axis, interleaved, dtype, positions below
    (1, 1, 1, 1, 32, (16,), 0, "bf16", 4), (1, 1, 12, 12, 64, (32,), 0, "bf16", 1024),
    (2, 37, 4, 2, 128, (16, 24, 24), 0, "bf16", 10 ** 6), (2, 37, 4, 2, 128, (16, 24, 24), 1, "bf16", 10 ** 6),
    (3, 5, 7, 1, 64, (5, 9, 10), 1, "f32", 2 ** 31 - 1), (3, 5, 7, 1, 64, (5, 9, 10), 0, "f32", 2 ** 31 - 1),
    (1, 130, 5, 5, 32, (1,), 0, "f32", 2000), (1, 1041, 3, 1, 128, (1, 1), 1, "bf16", 300),
    (5, 3, 2, 3, 64, (8, 8, 8, 8), 0, "bf16", 99), (64, 1, 32, 8, 128, (16, 24, 24), 0, "bf16", 10 ** 6),
    (2, 9, 40, 8, 128, (64,), 1, "f32", 5000)]


def _rope_table(sections, seed):
    n = sum(sections)
    axes = np.repeat(np.arange(len(sections)), sections).astype(np.uint8)
    np.random.default_rng(seed).shuffle(axes)
    return axes, 10000.0 ** (-np.arange(n) / n)


def _rope_close(y, x, pos, axes, freq, inter, sign=1):
    ref = ko.rope(f64(x), pos, axes, freq, inter, sign)
    half, n = x.shape[-1] // 2, len(freq)
    size = np.abs(f64(x))
    if inter:
        both = np.repeat(size[..., 0::2] + size[..., 1::2], 2, -1)
        both[..., 2 * n:] = 0
    else:
        both = size[..., :half] + size[..., half:]
        both[..., n:] = 0
        both = np.concatenate([both, both], -1)
    err = np.abs(f64(y) - ref)
    tol = torch.finfo(y.dtype).eps / 2 * np.abs(ref) + 2.0 ** -20.6 * both
    assert (err <= tol).all(), (err - tol).max()


@pytest.mark.parametrize("case", ROPE_CASES)
def test_rope_values(case):
    B, N, Hq, Hk, d, sec, inter, dt, far = case
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    axes, freq = _rope_table(sec, N)
    pos = np.random.default_rng(N + d).integers(-far, far, (B, N, len(sec)))
    pos[0, 0, 0] = -far if far < 2 ** 31 - 1 else -2 ** 31
    q, k = randn((B, N, Hq, d), 1, dtype), randn((B, N, Hk, d), 2, dtype)
    yq, yk = eio.rope(q, k, i32(pos), axes, freq, interleaved=bool(inter))
    _rope_close(yq, q, pos, axes, freq, inter)
    _rope_close(yk, k, pos, axes, freq, inter)
    zq, _ = eio.rope(q, None, i32(pos), axes, freq, interleaved=bool(inter), inverse=True)
    _rope_close(zq, q, pos, axes, freq, inter, -1)


def test_rope_strided_inputs_in_place_and_shared_positions():
    """q and k as parts of one fused projection, positions shared by the batch, outputs in place."""
    B, N, Hq, Hk, d = 3, 21, 4, 2, 64
    axes, freq = _rope_table((10, 12), 5)
    qkv = randn((B, N, Hq + 2 * Hk, d), 7)
    before = qkv.clone()
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    pos = np.random.default_rng(1).integers(0, 500, (N, 2))
    yq, yk = eio.rope(q, k, i32(pos), axes, freq)
    full = np.broadcast_to(pos, (B, N, 2))
    _rope_close(yq, q, full, axes, freq, 0)
    _rope_close(yk, k, full, axes, freq, 0)
    eio.rope(q, k, i32(pos), axes, freq, q_out=q, k_out=k)
    assert torch.equal(q, yq) and torch.equal(k, yk) and torch.equal(qkv[:, :, Hq + Hk:], before[:, :, Hq + Hk:])
    # a row that is one batch for all (stride 0) and a token slice
    one = randn((1, N, Hq, d), 8)
    ye, _ = eio.rope(one.expand(B, N, Hq, d)[:, 3:], None, i32(full[:, 3:].copy()), axes, freq)
    _rope_close(ye, one.expand(B, N, Hq, d)[:, 3:], full[:, 3:], axes, freq, 0)


def test_rope_refusals():
    q = randn((1, 4, 2, 64), 1)
    pos = i32(np.zeros((1, 4, 1)))
    ok = dict(axes=[0], freq=[1.0])
    for bad in (dict(q=q.half()), dict(q=q.transpose(1, 2)), dict(k=q.float()), dict(k=q[:, :3]),
                dict(positions=pos.long()), dict(positions=pos[:, :3]), dict(freq=[1.0, 2.0]), dict(q_out=q[:, :3]),
                dict(q_out=q.expand(1, 4, 2, 64).float()), dict(k_out=q)):
        with pytest.raises(ValueError):
            eio.rope(**{**dict(q=q, k=None, positions=pos), **ok, **bad})
    big = randn((1, 8, 2, 64), 1)
    with pytest.raises(ValueError, match="overlaps"):
        eio.rope(big[:, :4], None, pos, q_out=big[:, 2:6], **ok)
    with pytest.raises(eio.AttnError):
        eio.rope(torch.cat([q.flatten(), q.flatten()])[4:516].view(1, 4, 2, 64), None, pos, **ok)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradients(inter):
    """Gradients are the rotation back (shared heads and broadcast inputs sum them), and agree
    with differences of a weighted sum of the outputs."""
    B, N, H, d = 2, 6, 3, 64
    axes, freq = _rope_table((12, 20), 3)
    pos = np.random.default_rng(2).integers(0, 900, (B, N, 2))
    q = randn((B, N, H, d), 1, torch.float32).requires_grad_()
    base = randn((1, N, 1, d), 2, torch.float32).requires_grad_()
    wq, wk = randn((B, N, H, d), 3, torch.float32), randn((B, N, H, d), 4, torch.float32)

    def loss(q, base):
        yq, yk = autograd.rope(q, base.expand(B, N, H, d), i32(pos), axes, freq, interleaved=inter)
        return (yq.double() * wq).sum() + (yk.double() * wk).sum()
    gq, gb = torch.autograd.grad(loss(q, base), (q, base))
    np.testing.assert_allclose(f64(gq), ko.rope(f64(wq), pos, axes, freq, inter, -1), atol=2 ** -20 * 16)
    want = ko.rope(f64(wk), pos, axes, freq, inter, -1).sum((0, 2), keepdims=True)
    np.testing.assert_allclose(f64(gb), want, atol=2 ** -20 * 16 * B * H)
    # the map is linear, so a difference of any size is exact but for rounding: 2^-20 of sum |w| (|a| + |b|)
    e = randn((B, N, H, d), 5, torch.float32)
    with torch.no_grad():
        diff = float(loss(q + e, base) - loss(q, base))
    bound = 2.0 ** -20 * float((wq.abs().sum(-1) * (q.detach().abs() + (q.detach() + e).abs()).amax(-1) * 2).sum()) * 2
    assert abs(diff - float((gq.double() * e).sum())) <= bound


# ------------------------------------------------------------------ append and read
def test_rope_and_its_backward_in_a_graph():
    """Both directions captured and replayed with other rows, positions and gradients give the eager results."""
    axes, freq = _rope_table((12, 20), 3)

    def step(q, k, pos, w):
        yq, yk = autograd.rope(q, k, pos, axes, freq)
        return yq, *torch.autograd.grad((yq * w).sum() + (yk * w[:, :, :1]).sum(), (q, k))
    make = lambda seed: (randn((2, 6, 3, 64), seed, torch.float32).requires_grad_(),  # noqa: E731
                         randn((2, 6, 1, 64), seed + 1, torch.float32).requires_grad_(),
                         i32(np.random.default_rng(seed).integers(0, 900, (2, 6, 2))),
                         randn((2, 6, 3, 64), seed + 2, torch.float32))
    step(*make(1))
    held = make(11)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tuple(x.detach() for x in step(*held))
    for seed in (11, 21, 31):
        new = make(seed)
        with torch.no_grad():
            for x, y in zip(held, new):
                x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, step(*new)))


def _table(lens, page, seed, extra=2, width=1):
    """Pages in a random order: table, the pages of each sequence, and the pool's size."""
    per = [-(-n // page) for n in lens]
    order = np.random.default_rng(seed).permutation(sum(per) + extra)
    table = np.full((len(lens), max(max(per), width)), -7)  # entries behind a sequence's end are never read
    pages, at = [], 0
    for b, n in enumerate(per):
        pages.append(order[at:at + n].tolist())
        table[b, :n] = pages[-1]
        at += n
    return table, pages, len(order)


def _pool(n_pages, H, d, page, seed):
    return torch.from_numpy(np.random.default_rng(seed).integers(0, 256, (n_pages, H, page // 16 * 18 * d), dtype=np.uint8)).cuda()


APPEND_CASES = [
    # lens after, new (None: all N), N, Hkv, d, page
    ([1], None, 1, 1, 64, 16), ([1, 16, 17, 33], None, 1, 2, 128, 16), ([40, 7, 0, 64], [37, 7, 0, 1], 37, 3, 64, 16),
    ([300, 131], [255, 131], 255, 2, 128, 64), ([128], None, 128, 1, 128, 128), ([70, 256, 257], [70, 3, 100], 100, 5, 64, 256),
    ([33, 32, 31], None, 31, 12, 64, 32)]


@pytest.mark.parametrize("case", APPEND_CASES)
def test_append_writes_its_tokens_and_nothing_else(case):
    lens, new, N, H, d, page = case
    B = len(lens)
    table, pages, n_pages = _table(lens, page, N)
    pool = _pool(n_pages, H, d, page, 3)
    want = pool.cpu().numpy().copy()
    k, v = randn((B, N, H, d), 1, shift=0.5), randn((B, N, H, d), 2)
    counts = [N] * B if new is None else new
    for b in range(B):
        for x in (k, v):  # padding is not read
            x[b, counts[b]:] = math.nan
    kn, vn = f64(k), f64(v)
    for b in range(B):
        for i in range(counts[b]):
            t = lens[b] - counts[b] + i
            for h in range(H):
                tile = want[pages[b][t // page], h].reshape(page // 16, 18 * d)[t % page // 16]
                (ck, sk), (cv, sv) = ko.quantise(kn[b, i, h]), ko.quantise(vn[b, i, h])
                full = list(ko.unpack_tile(tile, d))
                for x, row in zip(full, (ck, sk, cv, sv)):
                    x[t % 16] = row
                packed = ko.pack_tile(*full)
                live = ko.pack_tile(*[_only(x, t % 16) for x in (np.full((16, d), 15), np.full((16, d // 32), -1.99),
                                                                 np.full((16, d), 15), np.full((16, d // 32), -1.99))])
                tile[live != 0] = packed[live != 0]
    eio.kv4_append(k, v, pool, i32(table), i32(lens), n_new=None if new is None else i32(new))
    eio.sync_status()
    assert np.array_equal(pool.cpu().numpy(), want)


def _only(x, tok):
    y = np.zeros_like(x)
    y[tok] = x[tok]
    return y


def test_append_of_strided_rows_on_another_stream():
    B, N, H, d, page = 2, 50, 2, 128, 32
    table, _, n_pages = _table([50, 50], page, 1)
    qkv = randn((B, N, 5 * H, d), 4)
    k, v = qkv[:, :, 2 * H:3 * H], qkv[:, :, 4 * H:]
    a, b = _pool(n_pages, H, d, page, 5), _pool(n_pages, H, d, page, 5)
    eio.kv4_append(k.contiguous(), v.contiguous(), a, i32(table), i32([50, 50]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    t, n = i32(table), i32([50, 50])
    torch.cuda.synchronize()
    eio.kv4_append(k, v, b, t, n, stream=side)
    kk, vv = eio.kv4_read(b, t, n, N, d, stream=side)
    side.synchronize()
    assert torch.equal(a, b)
    ka, va = eio.kv4_read(a, t, n, N, d)
    assert torch.equal(ka, kk) and torch.equal(va, vv)


def test_quantiser_extremes():
    """Zeros, values below the smallest scale, the largest finite ones, infinities and NaN, each in a
    group of its own; every bf16 magnitude against maxima next to it."""
    d, page = 64, 256
    rows = np.zeros((256, d), np.float32)
    rows[1, 3] = 2.0 ** -101
    rows[2, :32] = ko.bf16(np.float32(3.3e38))
    rows[3, 5], rows[4, 40], rows[5, 0] = np.inf, np.nan, -np.inf
    rows[6, :32] = np.linspace(-7, 7, 32)
    rows[7, 1], rows[7, 2] = 2.0 ** -100, 2.0 ** -133
    bits = (np.arange(248 * d) * 7 % 0x7f80).astype(np.uint32)  # every kind of bf16 magnitude
    x = (bits << 16).view(np.float32).reshape(248, d)
    rows[8:] = x * np.where(np.arange(d) % 3 == 0, -1, 1)
    rng = np.random.default_rng(3)
    rows[128:] = ko.bf16((rng.standard_normal((128, d)) * 2.0 ** rng.integers(-30, 30, (128, 1))).astype(np.float32))
    k = torch.from_numpy(rows.astype(np.float32)).to(torch.bfloat16).view(1, 256, 1, d).cuda()
    pool = _pool(1, 1, d, page, 1)
    eio.kv4_append(k, k, pool, i32([[0]]), i32([256]))
    kk, vv = eio.kv4_read(pool, i32([[0]]), i32([256]), 256, d)
    eio.sync_status()
    c, s = ko.quantise(f64(k)[0, :, 0])
    tiles = pool.cpu().numpy().reshape(16, 18 * d)
    for t in range(16):
        ck, sk, cv, sv = ko.unpack_tile(tiles[t], d)
        for got_c, got_s in ((ck, sk), (cv, sv)):
            assert np.array_equal(got_s, s[16 * t:16 * t + 16], equal_nan=True)
            assert np.array_equal(got_c, c[16 * t:16 * t + 16])
    want = ko.bf16(ko.value(c, s).astype(np.float32))
    for y in (kk, vv):
        assert np.array_equal(f64(y)[0, :, 0], want, equal_nan=True)


@pytest.mark.parametrize("d,page,N", [(64, 16, 1), (64, 64, 45), (128, 16, 45), (128, 256, 300), (128, 32, 33)])
def test_read_of_any_bytes(d, page, N):
    lens, start, H = [0, 1, 290, 47, 300], [0, 0, 3, 40, 16], 2
    table, pages, n_pages = _table(lens, page, d)
    pool = _pool(n_pages, H, d, page, 9)
    # scales as random bits, but finite
    p = pool.cpu().numpy().reshape(n_pages, H, page // 16, 18 * d)
    sc = p[..., 16 * d:].copy().view(np.uint16) & 0xbf7f
    p[..., 16 * d:] = sc.view(np.uint8)
    pool = torch.from_numpy(p.reshape(n_pages, H, -1)).cuda()
    k, v = eio.kv4_read(pool, i32(table), i32(lens), N, d, start=i32(start))
    eio.sync_status()
    for b, n in enumerate(lens):
        rk, rv = ko.rows(p.reshape(n_pages, H, -1), pages[b], page, n, d)
        for got, ref in ((k, rk), (v, rv)):
            want = np.zeros((N, H, d))
            part = ref[start[b]:start[b] + N]
            want[:len(part)] = ko.bf16(part.astype(np.float32))
            assert np.array_equal(f64(got)[b], want)


# ------------------------------------------------------------------ decode
def _cache_of(lens, H, d, page, seed, width=1):
    """A pool with random tokens in its sequences' pages, garbage (NaN scales among it) elsewhere."""
    table, pages, n_pages = _table(lens, page, seed, width=width)
    pool = _pool(n_pages, H, d, page, seed + 1)
    pool.view(n_pages, H, page // 16, 18 * d)[..., 16 * d:] = 0xff  # NaN scales wherever nothing is written
    N = max(max(lens), 1)
    k, v = randn((len(lens), N, H, d), seed + 2, shift=0.3), randn((len(lens), N, H, d), seed + 3)
    eio.kv4_append(k, v, pool, i32(table), i32(lens), n_new=i32(lens))
    host = pool.cpu().numpy()
    kv = [ko.rows(host, pages[b], page, n, d) for b, n in enumerate(lens)]
    return pool, i32(table), i32(lens), [x[0] for x in kv], [x[1] for x in kv]


def _decode_close(o, lse, q, ks, vs, scale):
    d = q.shape[-1]
    ro, rl, w, a = ko.decode(f64(q), ks, vs, scale)
    e = (d + 16) * 2.0 ** -23 * a + 2.0 ** -20
    rel = 2 * e.transpose(0, 2, 1)[..., None]
    G = q.shape[2] // ks[0].shape[1]
    gone = 2.0 ** -126 * np.stack([np.nan_to_num(np.abs(v)).sum(0).repeat(G, 0) for v in vs])[:, None]
    # len 2^-28 of the largest |v| of the channel's group of 32
    tiny = 2.0 ** -28 * np.stack([len(v) * np.nan_to_num(np.abs(v)).reshape(len(v), v.shape[1], d // 32, 32).max((0, 3), initial=0.0)
                                  .repeat(32, 1).repeat(G, 0) for v in vs])[:, None]
    tol = 2.0 ** -8 * (w + np.abs(ro)) * (1 + rel) + rel * w + gone + tiny + 2.0 ** -133
    err = np.abs(f64(o) - ro)
    assert (err <= tol).all(), (float((err - tol).max()), float((err / (tol + 1e-300)).max()))
    if lse is not None:
        live = np.isfinite(rl)
        l = f64(lse)
        assert np.array_equal(l[~live], rl[~live])
        terr = np.abs(l[live] - rl[live]) - (e + 2.0 ** -22 * np.abs(rl))[live]
        assert terr.size == 0 or (terr <= 0).all(), terr.max()


DECODE_CASES = [
    # lens, Sq, G, Hkv, d, page
    ([1], 1, 1, 1, 64, 16), ([1000], 1, 1, 12, 64, 16), ([0, 1, 15, 16, 17, 31, 32, 33], 1, 4, 2, 128, 16),
    ([0, 0], 1, 2, 1, 64, 32), ([65, 300, 2], 4, 4, 2, 128, 32), ([513, 64, 127, 1], 2, 3, 3, 64, 64),
    ([900, 3], 8, 8, 1, 128, 128), ([777], 5, 7, 2, 64, 256), ([1500, 20], 3, 5, 1, 128, 64),
    ([700, 0, 48], 1, 8, 2, 128, 256), ([260] * 40, 1, 2, 3, 64, 16), ([90, 41], 17, 1, 2, 64, 16),
    ([3000], 1, 16, 1, 128, 64), ([130, 70], 1, 12, 1, 64, 32), ([2049], 2, 6, 1, 128, 16),
    # one unit over every CTA; many short sequences, empty ones among them; more columns than one block
    ([20000], 1, 3, 1, 64, 64), ([(7 * i) % 50 * (i % 3 > 0) for i in range(150)], 1, 2, 2, 64, 16),
    ([33, 1, 64], 9, 2, 1, 64, 32), ([100, 31], 8, 8, 1, 128, 64)]


@pytest.mark.parametrize("case", DECODE_CASES)
def test_decode_values(case):
    lens, Sq, G, H, d, page = case
    pool, table, n, ks, vs = _cache_of(lens, H, d, page, 11 + d + Sq)
    q = randn((len(lens), Sq, G * H, d), 5)
    o, lse = eio.attn_decode_kv4(q, pool, table, n)
    eio.sync_status()
    _decode_close(o, lse, q, ks, vs, 1 / math.sqrt(d))
    o2, none = eio.attn_decode_kv4(q, pool, table, n, want_lse=False)
    assert none is None and torch.equal(o, o2)  # and nothing depends on timing


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** -8, 30.0, 1000.0])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_of_small_and_large_queries(size, d):
    """Flat and one-hot softmaxes: the running maximum moves, weights vanish."""
    pool, table, n, ks, vs = _cache_of([400, 70], 2, d, 16, 21)
    q = (randn((2, 2, 6, d), 6, torch.float32) * size).to(torch.bfloat16)
    q[0, 0, 1] = 0
    q[0, 1, 2, 1:] = 0
    o, lse = eio.attn_decode_kv4(q, pool, table, n, scale=0.25)
    _decode_close(o, lse, q, ks, vs, 0.25)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_with_a_scale_near_zero(d):
    """Weights are equal whatever the queries, zero rows among them, and masked tokens still have none."""
    lens = [0, 1, 3, 70]
    pool, table, n, ks, vs = _cache_of(lens, 2, d, 16, 23)
    q = randn((4, 3, 4, d), 6)
    q[:, :, 1] = 0
    for scale in (1e-10, 1e-25, 1e-37):
        o, lse = eio.attn_decode_kv4(q, pool, table, n, scale=scale)
        _decode_close(o, lse, q, ks, vs, scale)


def test_decode_masked_tokens_with_nan_do_not_matter():
    """A NaN in a token that only the newest query sees leaves the others as they were; that one is NaN."""
    d, page, H, L = 128, 32, 2, 70
    pool, table, n, ks, vs = _cache_of([L], H, d, page, 31)
    k = randn((1, 1, H, d), 3)
    q = randn((1, 3, 4 * H, d), 4)
    for which in range(2):
        bad = k.clone()
        bad[..., 40] = math.nan if which else math.inf
        eio.kv4_append(k if which else bad, bad if which else k, pool, table, n)
        o, _ = eio.attn_decode_kv4(q, pool, table, n)
        host = pool.cpu().numpy()
        ks, vs = ko.rows(host, table[0].tolist(), page, L - 1, d)
        part, lpart = eio.attn_decode_kv4(q[:, :2].contiguous(), pool, table, n - 1)
        _decode_close(part, lpart, q[:, :2], [ks], [vs], 1 / math.sqrt(d))
        _decode_close(o[:, :2], None, q[:, :2], [ks], [vs], 1 / math.sqrt(d))
        last = o[0, 2]
        assert torch.isnan(last[:, 32:64]).all()
        assert torch.isnan(last).all() == (which == 0)


def test_decode_query_rows_with_nan_or_infinity_stay_apart():
    pool, table, n, ks, vs = _cache_of([100], 1, 64, 16, 41)
    q = randn((1, 1, 6, 64), 4)
    clean, lc = eio.attn_decode_kv4(q, pool, table, n)
    q2 = q.clone()
    q2[0, 0, 2, 5], q2[0, 0, 4, 63] = math.nan, math.inf
    o, lse = eio.attn_decode_kv4(q2, pool, table, n)
    for h in range(6):
        if h in (2, 4):
            assert torch.isnan(o[0, 0, h]).all() and torch.isnan(lse[0, h]).all()
        else:
            assert torch.equal(o[0, 0, h], clean[0, 0, h]) and torch.equal(lse[0, h], lc[0, h])


def test_bad_device_arguments_are_latched():
    """Lengths, counts, starts and page numbers out of range: a latched error, zeros or rows left out, no fault."""
    d, page, H = 64, 16, 2
    pool, table, n, ks, vs = _cache_of([40, 40, 40], H, d, page, 51)
    q = randn((3, 1, 4, d), 4)
    good, gl = eio.attn_decode_kv4(q, pool, table, n)
    eio.sync_status()

    def latched():
        with pytest.raises(eio.AttnError) as e:
            eio.sync_status()
        assert e.value.code == 9
    for lens in ([-1, 40, 40], [49, 40, 40], [2 ** 31 - 1, 40, 40]):
        o, lse = eio.attn_decode_kv4(q, pool, table, i32(lens))
        latched()
        assert (o[0] == 0).all() and (lse[0] == -math.inf).all() and torch.equal(o[1:], good[1:])
        k, v = eio.kv4_read(pool, table, i32(lens), 8, d)
        latched()
        assert (k[0] == 0).all() and (v[0] == 0).all()
    for page_id in (-1, pool.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[0, 1] = page_id
        good, gl = eio.attn_decode_kv4(q, pool, table, n)  # the appends below change sequences 1 and 2
        o, lse = eio.attn_decode_kv4(q, pool, t, n)
        latched()
        keep = np.r_[0:16, 32:40]
        _decode_close(o[:1], lse[:1], q[:1], [ks[0][keep]], [vs[0][keep]], 1 / math.sqrt(d))
        assert torch.equal(o[1:], good[1:]) and torch.equal(lse[1:], gl[1:])
        k, v = eio.kv4_read(pool, t, n, 40, d)
        latched()
        assert (k[0, 16:32] == 0).all() and np.array_equal(f64(v)[0, keep], ko.bf16(vs[0][keep].astype(np.float32)))
        before = pool.clone()
        rows = randn((3, 1, H, d), 7)
        eio.kv4_append(rows, rows, pool, t, i32([17, 40, 40]))
        latched()
        for p in range(pool.shape[0]):
            same = torch.equal(pool[p], before[p])
            assert same or p in (int(table[1, 2]), int(table[2, 2]))
    before = pool.clone()
    for new in (-1, 2, 2 ** 31 - 1):
        rows = randn((3, 1, H, d), 8)
        eio.kv4_append(rows, rows, pool, table, n, n_new=i32([new, 0, 0]))
        latched()
        assert torch.equal(pool, before)
    k, v = eio.kv4_read(pool, table, n, 8, d, start=i32([-1, 0, 2 ** 31 - 1]))
    latched()
    assert (k[0] == 0).all() and (k[2] == 0).all() and (k[1] != 0).any()


def test_binding_refusals():
    pool, table, n, _, _ = _cache_of([40], 2, 64, 16, 61)
    q = randn((1, 1, 4, 64), 4)
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(q=q.expand(2, 1, 4, 64).contiguous()), dict(pool=pool[:, :, 4:]),
                dict(pool=pool[:, :, :1000].contiguous()), dict(table=table.long()), dict(table=table[0]),
                dict(seqlens=n.long()), dict(seqlens=i32([1, 2])), dict(o=q[:, :, :2]), dict(lse=torch.zeros(1, 4, device="cuda"))):
        with pytest.raises(ValueError):
            eio.attn_decode_kv4(**{**dict(q=q, pool=pool, table=table, seqlens=n), **bad})
    with pytest.raises(eio.AttnError):
        eio.attn_decode_kv4(q[:, :, :3].contiguous(), pool, table, n)
    k = randn((1, 1, 2, 64), 1)
    for bad in (dict(k=k[..., :32]), dict(v=k.float()), dict(k=k.transpose(2, 3)), dict(n_new=n.long())):
        with pytest.raises(ValueError):
            eio.kv4_append(**{**dict(k=k, v=k, pool=pool, table=table, seqlens=n), **bad})
    with pytest.raises(ValueError):
        eio.kv4_read(pool, table, n, 4, 128)
    with pytest.raises(eio.AttnError):
        eio.kv4_read(pool, table, n, 0, 64)


def test_calls_on_two_streams_and_in_graphs():
    """Two decodes at once do not share scratch; a captured one can be replayed beside others and
    follows the lengths in its buffers."""
    d, page, H = 128, 64, 2
    pool, table, n, ks, vs = _cache_of([900, 333], H, d, page, 71)
    q1, q2 = randn((2, 1, 8, d), 1), randn((2, 4, 8, d), 2)
    want1, want2 = eio.attn_decode_kv4(q1, pool, table, n), eio.attn_decode_kv4(q2, pool, table, n)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        got.append((eio.attn_decode_kv4(q1, pool, table, n, stream=s1), want1))
        got.append((eio.attn_decode_kv4(q2, pool, table, n, stream=s2), want2))
    torch.cuda.synchronize()
    for (o, lse), (wo, wl) in got:
        assert torch.equal(o, wo) and torch.equal(lse, wl)
    lens = n.clone()
    graphs = []
    for q in (q1, q2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, q, eio.attn_decode_kv4(q, pool, table, lens)))
    for step in range(3):
        lens.copy_(n - 50 * step)
        torch.cuda.synchronize()
        for (g, _, _), s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for g, q, (o, lse) in graphs:
            wo, wl = eio.attn_decode_kv4(q, pool, table, lens)
            assert torch.equal(o, wo) and torch.equal(lse, wl)


def test_decode_equals_attention_over_the_rows_read_back():
    """A prefill over the cached rows (kv4_read and attn_fwd, causal, bottom-right) gives the decode's
    answer; the rows are rounded to bf16 there: 2^-8 of each, in the scores too."""
    d, page, H, L, Sq = 128, 32, 2, 500, 6
    pool, table, n, ks, vs = _cache_of([L], H, d, page, 81)
    q = randn((1, Sq, 4 * H, d), 4)
    o, lse = eio.attn_decode_kv4(q, pool, table, n)
    k, v = eio.kv4_read(pool, table, n, L, d)
    of, lf = eio.attn_fwd(q, k, v, mask_kind=eio.MASK_CAUSAL)
    _, _, w, a = ko.decode(f64(q), ks, vs, 1 / math.sqrt(d))
    e = 2.0 ** -8 * a.transpose(0, 2, 1)[..., None]
    assert (np.abs(f64(o) - f64(of)) <= (4 * 2.0 ** -8 + 2 * (np.exp(2 * e) - 1)) * w).all()
    assert (np.abs(f64(lse) - f64(lf)) <= 2.0 ** -8 * a + 1e-3).all()


def test_a_step_in_a_graph_follows_its_buffers():
    """Rotation, append, page copy, read and decode captured once and replayed with other rows, positions
    and lengths in the same buffers."""
    B, H, G, d, page = 2, 2, 4, 64, 16
    axes, freq = _rope_table((16, 16), 2)
    table, pages, n_pages = _table([64, 64], page, 3, extra=4)
    free = sorted(set(range(n_pages)) - set(sum(pages, [])))
    pool = _pool(n_pages, H, d, page, 4)
    t, lens = i32(table), i32([40, 10])
    q, k, v = (randn((B, 1, h, d), 5 + h) for h in (G * H, H, H))
    pos = i32(np.zeros((B, 1, 2)))

    def step():
        rq, rk = eio.rope(q, k, pos, axes, freq)
        eio.kv4_append(rk, v, pool, t, lens)
        eio.copy_pages(pool, [pages[0][0]], [free[0]])
        return (rq, rk, *eio.attn_decode_kv4(rq, pool, t, lens), *eio.kv4_read(pool, t, lens, 7, d))
    eio.kv4_append(randn((B, 64, H, d), 1), randn((B, 64, H, d), 2), pool, t, i32([64, 64]))
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for i, n in enumerate(([41, 11], [64, 1], [17, 16])):
        for x, seed in ((q, 30), (k, 40), (v, 50)):
            x.copy_(randn(x.shape, seed + i))
        lens.copy_(i32(n))
        pos.fill_(7 + 1000 * i)
        before = pool.clone()
        g.replay()
        torch.cuda.synchronize()
        got, after = [x.clone() for x in out], pool.clone()
        pool.copy_(before)
        for x, y in zip(got, step()):
            assert torch.equal(x, y)
        assert torch.equal(after, pool) and torch.equal(pool[free[0]], pool[pages[0][0]])
    eio.sync_status()


def test_first_call_on_a_device_inside_a_capture_is_refused():
    """The error word is allocated by the first call: inside a capture that is an error, not a broken capture."""
    pool, table, n, _, _ = _cache_of([20], 1, 64, 16, 91)
    q = randn((1, 1, 1, 64), 1)
    want = eio.attn_decode_kv4(q, pool, table, n)
    torch.cuda.synchronize()
    eio.shutdown()
    x = torch.zeros(4, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(eio.AttnError) as e:
            eio.kv4_append(q, q, pool, table, n)
        x += 1
    assert e.value.code == 8
    g.replay()
    assert (x == 1).all()
    got = eio.attn_decode_kv4(q, pool, table, n)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_pools_past_four_gigabytes():
    """Pages whose bytes lie past 2^32 are written, read, decoded and copied like the first ones."""
    H, d, page, n_pages = 8, 128, 256, 16000
    pool = eio.kv4_pool(n_pages, H, d, page)
    assert (n_pages - 8) * pool[0].numel() > 2 ** 32
    far, near = [n_pages - 1, n_pages - 3], [1, 0]
    lens = [300]
    k, v = randn((1, 300, H, d), 1), randn((1, 300, H, d), 2)
    q = randn((1, 2, 2 * H, d), 3)
    got = []
    for pages in (far, near):
        t, n = i32([pages]), i32(lens)
        eio.kv4_append(k, v, pool, t, n)
        got.append((*eio.kv4_read(pool, t, n, 300, d), *eio.attn_decode_kv4(q, pool, t, n)))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    eio.copy_pages(pool, far, [n_pages - 7, 2])
    assert torch.equal(pool[2], pool[far[1]]) and torch.equal(pool[n_pages - 7], pool[far[0]])
    assert torch.equal(eio.attn_decode_kv4(q, pool, i32([[n_pages - 7, 2]]), i32(lens))[0], got[0][2])
    eio.sync_status()


# ------------------------------------------------------------------ pages
@pytest.mark.parametrize("n_pages,page_elems,dtype,moves", [
    (4, 16, torch.uint8, 1), (9, 18 * 64, torch.uint8, 4), (3000, 64, torch.uint8, 1500), (40, 4096, torch.bfloat16, 20),
    (11, 1000 * 16, torch.uint8, 3), (9000, 16, torch.uint8, 4400)])
def test_copy_pages(n_pages, page_elems, dtype, moves):
    pool = torch.from_numpy(np.random.default_rng(moves).integers(0, 100, (n_pages, page_elems))).to(dtype).cuda()
    order = np.random.default_rng(moves + 1).permutation(n_pages)
    src, dst = order[:moves], order[moves:2 * moves]
    want = pool.clone()
    want[torch.from_numpy(dst).cuda()] = pool[torch.from_numpy(src).cuda()]
    eio.copy_pages(pool, src, dst)
    assert torch.equal(pool, want)
    same = np.full(min(moves, 3), src[0])
    eio.copy_pages(pool, same, dst[:len(same)])  # a source may repeat
    assert all(torch.equal(pool[int(i)], want[src[0]]) for i in dst[:len(same)])


def test_copy_pages_refusals():
    pool = torch.zeros(8, 32, dtype=torch.uint8, device="cuda")
    eio.copy_pages(pool, [], [])
    for src, dst, err in (([0], [1, 2], ValueError), ([[0]], [[1]], ValueError), ([0.5], [1], ValueError),
                          ([0], [2 ** 32], ValueError), ([0], [8], ValueError), ([0, 1], [2, 2], eio.AttnError),
                          ([0, 1], [1, 2], eio.AttnError)):
        with pytest.raises(err):
            eio.copy_pages(pool, src, dst)
    with pytest.raises(eio.AttnError):
        eio.copy_pages(pool.view(32, 8), [0], [1])  # 8-byte pages
    with pytest.raises(ValueError):
        eio.copy_pages(pool[:, ::2], [0], [1])


# ------------------------------------------------------------------ together
def test_serving_run():
    """A prompt, forks, drafts taken back and a compaction, two layers: rotated keys appended, every
    decode against fp64 over the tokens each sequence should hold."""
    H, G, d, page, layers = 2, 3, 64, 16, 2
    cache = Kv4Cache(24, H, d, page=page, layers=layers)
    axes, freq = _rope_table((16, 16), 1)
    seed = [100]
    held = {}  # id -> per layer list of (k, v) rows, quantised, fp64

    def step(ids, counts, Sq):
        batch = cache.extend(ids, counts)
        N = max(counts)
        first = [cache.length(i) - c for i, c in zip(ids, counts)]
        pos = np.stack([np.stack([f + np.arange(N), (f + np.arange(N)) // 7], -1) for f in first])
        for layer in range(layers):
            seed[0] += 3
            q, k, v = (randn((len(ids), N, h, d), seed[0] + j) for j, h in enumerate((G * H, H, H)))
            q, k = eio.rope(q, k, i32(pos), axes, freq)
            cache.append(layer, k, v, batch)
            for b, i in enumerate(ids):
                for x, rows in ((k, held[i][layer][0]), (v, held[i][layer][1])):
                    rows.extend(ko.value(*ko.quantise(f64(x)[b, t])) for t in range(counts[b]))
            qs = q[:, :Sq].contiguous()
            o, lse = cache.decode(layer, qs, batch)
            ks, vs = ([np.array(held[i][layer][j]) for i in ids] for j in range(2))
            _decode_close(o, lse, qs, ks, vs, 1 / math.sqrt(d))

    def fork(i):
        j = cache.fork(i)
        held[j] = [[list(x) for x in layer] for layer in held[i]]
        return j
    a = cache.add()
    held[a] = [[[], []] for _ in range(layers)]
    step([a], [37], 1)
    b, c = fork(a), fork(a)
    step([a, b, c], [1, 1, 1], 1)
    step([b, a], [4, 2], 2)
    cache.truncate(b, 38)
    for layer in held[b]:
        for rows in layer:
            del rows[38:]
    cache.free(c)
    del held[c]
    assert cache.compact() > 0
    step([a, b], [3, 30], 3)
    with pytest.raises(Kv4Full):
        cache.extend([a], 16 * 24)
    batch = cache.batch([a, b])
    k, v = cache.read(1, batch, 80)
    eio.sync_status()
    for r, i in enumerate((a, b)):
        n = cache.length(i)
        for got, rows in ((k, held[i][1][0]), (v, held[i][1][1])):
            assert np.array_equal(f64(got)[r, :n], ko.bf16(np.array(rows).astype(np.float32)))
            assert (got[r, n:] == 0).all()
