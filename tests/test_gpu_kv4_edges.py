"""Rotary positions and the 4-bit cache on the GPU where values are not finite or lie far apart,
against fp64 (kv4_oracle and torch).

Tolerance of the decode's O, from the arithmetic, for one row (query token and head) and the keys it
sees, with weights p (their sum is 1), and in terms of the largest |v| of a group of 32 channels (7 sv):
  2^-11 sum p |v|   P sv is rounded to fp16 (half a step of 11 bits); the sums and products around it
                    are in fp32, a tensor core may drop what it adds to: (n / 16 + 64) 2^-23 more
  2 e sum p |v|     the scores' error e moves p and its sum; a score is a sum of d products of q with a
                    code 0 .. 15 (|k| + 8 sk bounds them), of which 8 sum q is taken off, in fp32 sums
                    that may drop 2^-23 a step: (d + 16) 2^-23 sum |q| (|k| + 8 sk) scale; ex2 and the
                    sum of p add 2^-20
  n 2^-30 max p 7 sv   the largest product of a row and a group, when its reference last moved, became a
                    number of at least 2^5 (2^6, or more than half of it after the base has moved); fp16's
                    last step below 2^-14 is 2^-24, half of it 2^-25, times a code of 7 at most
  weights below 2^-110 of the largest may be left out whole (ex2 and products of them end at 2^-126)
  2^-8 |O|          the output is a bf16 number
Nothing of a key that the row does not see enters.
"""
import math

import numpy as np
import pytest
import torch

import exact_io_aware_sm_b200 as eio
from exact_io_aware_sm_b200 import autograd
from exact_io_aware_sm_b200.kv4_cache import Kv4Cache
from tests import kv4_oracle as ko

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built_lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from exact_io_aware_sm_b200 import build
    build.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ rope
def _bits(x):
    return x.contiguous().view(torch.int16 if x.dtype is torch.bfloat16 else torch.int32)


@pytest.mark.parametrize("d,n", [(32, 1), (32, 15), (64, 5), (64, 31), (128, 3), (128, 33), (128, 63)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_copies_channels_without_an_entry_bit_by_bit(dtype, inter, d, n):
    """Infinities, NaNs with any payload and zeros of either sign outside the table stay, and do
    not reach their neighbours; both ways, out of place and in place."""
    rng = np.random.default_rng(d + n)
    bits = rng.integers(0, 1 << 16, (2, 9, 5, d), dtype=np.int64)  # any bf16
    special = np.array([0x7f80, 0xff80, 0x7fc1, 0xffff, 0x7f81, 0x8000, 0x0000, 0x0001])
    bits = np.where(rng.random(bits.shape) < 0.5, special[rng.integers(0, 8, bits.shape)], bits)
    table = np.zeros(d, bool)
    for p in range(n):
        table[[2 * p, 2 * p + 1] if inter else [p, p + d // 2]] = True
    finite = ko.bf16(rng.standard_normal(bits.shape).astype(np.float32)).astype(np.float32)
    word = np.where(table, finite.view(np.uint32) >> 16, bits).astype(np.uint32) << 16
    if dtype is torch.float32:
        word |= np.where(table, 0, rng.integers(0, 1 << 16, bits.shape)).astype(np.uint32)
    x = torch.from_numpy(word.view(np.int32)).cuda().view(torch.float32)
    if dtype is torch.bfloat16:
        x = (torch.from_numpy((word >> 16).astype(np.uint16).view(np.int16)).cuda()).view(torch.bfloat16)
    clean = torch.where(torch.from_numpy(table).cuda(), x, torch.zeros_like(x))
    pos = i32(rng.integers(-1000, 1000, (2, 9, 1)))
    axes, freq = np.zeros(n, np.uint8), 10000.0 ** (-np.arange(n) / n)
    keep, turn = torch.from_numpy(np.flatnonzero(~table)).cuda(), torch.from_numpy(np.flatnonzero(table)).cuda()
    for inverse in (False, True):
        want, _ = eio.rope(clean, None, pos, axes, freq, interleaved=inter, inverse=inverse)
        q, k = x.clone(), x[:, :, :2].clone()
        for q_out, k_out in ((None, None), (q, k)):
            yq, yk = eio.rope(q, k, pos, axes, freq, interleaved=inter, inverse=inverse, q_out=q_out, k_out=k_out)
            for y, h in ((yq, 5), (yk, 2)):
                assert torch.equal(_bits(y[..., keep]), _bits(x[:, :, :h][..., keep]))
                assert torch.equal(_bits(y[..., turn]), _bits(want[:, :, :h][..., turn]))


@pytest.mark.parametrize("dtype,off", [(torch.bfloat16, 4), (torch.bfloat16, 1), (torch.float32, 2)])
def test_rope_takes_gradients_off_a_16_byte_boundary(dtype, off):
    g = torch.Generator(device="cuda").manual_seed(off)
    q = torch.randn(2, 5, 4, 64, device="cuda", generator=g).to(dtype).requires_grad_()
    dq = torch.randn(2, 5, 4, 64, device="cuda", generator=g).to(dtype)
    flat = torch.empty(off + dq.numel(), dtype=dtype, device="cuda")
    other = flat[off:].view(dq.shape)
    other.copy_(dq)
    pos = i32(np.arange(5)[:, None])
    y, _ = autograd.rope(q, None, pos, [0] * 32, 100.0 ** (-np.arange(32) / 32))
    want, = torch.autograd.grad(y, q, dq, retain_graph=True)
    assert other.data_ptr() % 16 and torch.equal(torch.autograd.grad(y, q, other)[0], want)


# ------------------------------------------------------------------ cache
@pytest.mark.parametrize("device", [None, "cuda", "cuda:0", torch.device("cuda")])
def test_a_cache_stays_on_the_device_that_it_was_made_on(device):
    """Its device has a number: "cuda" alone would send a later table to whatever device is current then."""
    cache = Kv4Cache(4, 1, 64, device=device)
    assert cache.device == cache.pool.device and cache.device.index == torch.cuda.current_device()
    batch = cache.extend([cache.add()], 5)
    assert batch.table.device == batch.seqlens.device == cache.pool.device


# ------------------------------------------------------------------ decode
def _quantised(x):
    """Values and scales (repeated over their channels), fp64 on the GPU, of x [B, L, H, d] bf16."""
    vals, scales = [], []
    for part in x.cpu().split(max(1, (1 << 22) // x[0].numel())):
        c, s = ko.quantise(part.double().numpy())
        vals.append(torch.from_numpy(ko.value(c, s)).cuda())
        scales.append(torch.from_numpy(s).cuda().repeat_interleave(32, -1))
    return torch.cat(vals), torch.cat(scales)


def _filled(k, v, B, page=64):
    """Pool, table and lengths of a cache with the rows k, v [B, L, H, d] (or [1, L, H, d], the same for
    every sequence)."""
    _, L, H, d = k.shape
    k, v = k.expand(B, -1, -1, -1), v.expand(B, -1, -1, -1)
    per = -(-L // page)
    pool = eio.kv4_pool(B * per, H, d, page)
    pool.fill_(0xff)
    table = torch.randperm(B * per, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    table = table.to(torch.int32).view(B, per)
    n = i32([L] * B)
    eio.kv4_append(k, v, pool, table, n)
    return pool, table, n


def _check(o, lse, q, k, v, scale):
    """O and LSE of the decode against fp64 over the quantised rows; the bound is the docstring's."""
    B, Sq, Hq, d = q.shape
    L, H = k.shape[1:3]
    kv, sk, vv, sv = (x.expand(B, -1, -1, -1) for x in (*_quantised(k), *_quantised(v)))
    for s in range(Sq):
        n = L - Sq + s + 1
        x = q[:, s].double().view(B, H, -1, d)
        kk, vs, top = kv[:, :n], vv[:, :n], 7 * sv[:, :n]
        score = torch.einsum("bhgd,blhd->bhgl", x, kk) * scale
        e = (d + 16) * 2.0 ** -23 * torch.einsum("bhgd,blhd->bhgl", x.abs(), kk.abs() + 8 * sk[:, :n]).amax(-1) * scale
        e = (e + 2.0 ** -20)[..., None]
        p = torch.softmax(score, -1)
        gone = p < 2.0 ** -110 * p.amax(-1, keepdim=True)
        want = torch.einsum("bhgl,blhd->bhgd", p, vs)
        w = torch.einsum("bhgl,blhd->bhgd", p, vs.abs())
        w0 = torch.einsum("bhgl,blhd->bhgd", p * gone, vs.abs())
        peak = torch.stack([(p * top[..., 32 * i].permute(0, 2, 1)[:, :, None]).amax(-1) for i in range(d // 32)], -1)
        tol = ((2.0 ** -11 + (n / 16 + 64) * 2.0 ** -23) * (1 + 2 * e) + 2 * e) * w + n * 2.0 ** -30 * peak.repeat_interleave(32, -1) + w0
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs() + 2.0 ** -133
        err = (o[:, s].double().view(want.shape) - want).abs()
        assert (err <= tol).all(), (s, float((err / tol).nan_to_num(1e30).max()))
        want = torch.logsumexp(score, -1)
        err = (lse[:, :, s].double().view(want.shape) - want).abs()
        assert (err <= e[..., 0] + 2.0 ** -22 * want.abs()).all(), s


def _inputs(B, L, H, G, Sq, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = (B if B <= 300 else 1, L, H, d)
    q, k, v = (torch.randn(s, device="cuda", generator=g) for s in ((B, Sq, G * H, d), rows, rows))
    q[..., 0] = 4  # the same way in every row, so that k's channel 0 moves every score alike
    return q, k, v


FORMS = [(64, 1), (64, 2), (128, 1), (128, 2), (128, 4)]  # d, heads a KV head: 3, 6 and twice 6 columns
# Sequences, keys, KV heads: every unit cut into many runs; units of 5 stages, some whole in a warp's run; runs of 20
# stages.
RUNS = [(1, 500, 2), (300, 150, 4), (1800, 700, 1)]


@pytest.mark.parametrize("d,G", FORMS)
@pytest.mark.parametrize("B,L,H", RUNS)
@pytest.mark.parametrize("big", [1e4, 1e7, 1e9, 3.0e38])
@pytest.mark.parametrize("where", ["hidden", "weightless early", "weightless late", "seen early", "seen late"])
def test_decode_with_one_token_of_large_values(where, big, B, L, H, d, G):
    """A token whose V is far larger than the others': hidden from all but the newest query, of no
    weight, or seen.  It must not cost the rows that it does not belong to their digits."""
    q, k, v = _inputs(B, L, H, G, 3, d, 5)
    at = L - 1 if where == "hidden" else 3 if where.endswith("early") else L - 6
    v[:, at] *= big / v[:, at].abs().amax()
    if where.startswith("weightless"):
        k[:, at, :, 0] = -1200.0  # e^-400 of the others, or less
    q, k, v = (x.to(torch.bfloat16) for x in (q, k, v))
    pool, table, n = _filled(k, v, B)
    o, lse = eio.attn_decode_kv4(q, pool, table, n)
    eio.sync_status()
    _check(o, lse, q, k, v, 1 / math.sqrt(d))


@pytest.mark.parametrize("d,G", FORMS)
@pytest.mark.parametrize("B,L,H", RUNS)
def test_decode_rows_do_not_depend_on_a_token_that_they_do_not_see(B, L, H, d, G):
    """Bit for bit, whatever finite values the newest token has."""
    q, k, v = (x.to(torch.bfloat16) for x in _inputs(B, L, H, G, 3, d, 8))
    pool, table, n = _filled(k, v, B)
    want, lse = eio.attn_decode_kv4(q, pool, table, n)
    for size in (0.0, 1e4, 1e9, 3.0e38):
        rows = (torch.sign(v[:, -1:]) * size).expand(B, -1, -1, -1)
        eio.kv4_append(k[:, -1:].expand(B, -1, -1, -1), rows, pool, table, n)
        o, l = eio.attn_decode_kv4(q, pool, table, n)
        assert torch.equal(o[:, :2], want[:, :2]) and torch.equal(l[..., :2], lse[..., :2])
    eio.sync_status()


@pytest.mark.parametrize("d,G", FORMS)
@pytest.mark.parametrize("B,L,H", RUNS)
@pytest.mark.parametrize("what", ["stairs", "up", "down", "balanced", "groups", "tiny"])
def test_decode_of_values_that_change_size_along_the_keys(what, B, L, H, d, G):
    """stairs: tokens of no weight, each 512 times larger than the one before; up, down: scores that rise
    all along while V grows or falls by 1e8; balanced: V falls as fast as the weights grow, 100 octaves, so
    that all terms count; groups: channels of V 1e9 apart; tiny: every V below 2^-90."""
    q, k, v = _inputs(B, L, H, G, 3, d, 6)
    i = torch.arange(L, device="cuda")
    if what == "stairs":
        for j, at in enumerate(range(2, L - 3, max(1, L // 9))):
            v[:, at] *= 512.0 ** (j + 1)
            k[:, at, :, 0] = -1200.0
    elif what == "groups":
        v[..., :32] *= 1e9
    elif what == "tiny":
        v *= 2.0 ** -95
    elif what == "balanced":
        k[..., 0] = (i / L * 100 * math.log(2))[None, :, None] * math.sqrt(d) / 4
        v *= (2.0 ** (50 - 100 * i / L))[None, :, None, None]
    else:
        k[..., 0] = (i / L * 40 - 20)[None, :, None] * math.sqrt(d) / 4
        v *= (10.0 ** (8 * i / L) if what == "up" else 10.0 ** (-8 * i / L))[None, :, None, None]
    q, k, v = (x.to(torch.bfloat16) for x in (q, k, v))
    pool, table, n = _filled(k, v, B, 32)
    o, lse = eio.attn_decode_kv4(q, pool, table, n)
    eio.sync_status()
    _check(o, lse, q, k, v, 1 / math.sqrt(d))


@pytest.mark.parametrize("d,G", FORMS)
@pytest.mark.parametrize("B,L,H", RUNS)
def test_decode_of_values_near_the_types_largest(B, L, H, d, G):
    """Every V about 3e38, with weights that add up past it before they are divided by their sum."""
    q, k, v = _inputs(B, L, H, G, 3, d, 7)
    v = torch.where(v < 0, -3.0e38, 3.0e38) * (1 - 0.2 * v.abs().clamp(max=1))
    q, k, v = (x.to(torch.bfloat16) for x in (q, k, v))
    pool, table, n = _filled(k, v, B, 16)
    o, lse = eio.attn_decode_kv4(q, pool, table, n)
    eio.sync_status()
    assert torch.isfinite(o.float()).all()
    _check(o, lse, q, k, v, 1 / math.sqrt(d))


@pytest.mark.parametrize("G", [4, 8])
def test_decode_keeps_its_digits_over_half_a_million_keys(G):
    """The norm of O's error over O's.  The weights are flat, so that O is a mean of n values, sqrt(n) times
    smaller than they are, and an error of every term counts like O itself.  Rounding O to bf16 is
    2^-7 / sqrt(12) of a binade's start, 0.00154 of the norm over a binade; 2^-11 a term (fp16) adds 0.0002,
    where 2^-8 (bf16) would give 0.0022 together, and numbers of 8 sum P sv more.  512 or 1024 outputs
    scatter by 3 %: 2^-9 lies eight such steps above the first and below the others."""
    d, L, page = 128, 500001, 128
    g = torch.Generator(device="cuda").manual_seed(G)
    q = 0.25 * torch.randn(1, 1, G, d, device="cuda", generator=g)
    k, v = (torch.randn(1, L, 1, d, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    q = q.to(torch.bfloat16)
    pool, table, n = _filled(k, v, 1, page)
    o, lse = eio.attn_decode_kv4(q, pool, table, n)
    eio.sync_status()
    x, w, want = [], [], []
    for kp, vp in zip(k[0, :, 0].split(1 << 16), v[0, :, 0].split(1 << 16)):
        kk, vv = _quantised(kp[:, None, None])[0][:, 0, 0], _quantised(vp[:, None, None])[0][:, 0, 0]
        x.append(q[0, 0].double() @ kk.T / math.sqrt(d))
        m = x[-1].amax(-1, keepdim=True)
        w.append((m, torch.exp(x[-1] - m).sum(-1, keepdim=True)))
        want.append(torch.exp(x[-1] - m) @ vv)
    lref = torch.logsumexp(torch.cat(x, -1), -1)
    ref = sum(y * torch.exp(m - lref[:, None]) for y, (m, _) in zip(want, w))
    assert (lse[0, :, 0].double() - lref).abs().max() <= 1e-4
    err = (o[0, 0].double() - ref).norm() / ref.norm()
    assert err <= 2.0 ** -9, float(err)


@pytest.mark.parametrize("d,G", FORMS)
@pytest.mark.parametrize("B,L,H", [(1, 500, 2), (300, 150, 4), (40, 2, 3)])
def test_decode_of_query_rows_that_are_not_finite(B, L, H, d, G):
    """Such rows are NaN, O and LSE, if they see a token, and 0 and -inf if not; the others are what they are
    without them, bit for bit.  2^115.9 is a size like any other, 2^116 is not."""
    q, k, v = (x.to(torch.bfloat16) for x in _inputs(B, L, H, G, 3, d, 9))
    pool, table, n = _filled(k, v, B)
    want, lse = eio.attn_decode_kv4(q, pool, table, n)
    q2 = q.clone()
    bad = torch.zeros(q.shape[:3], dtype=torch.bool, device="cuda")
    for i, x in enumerate((math.nan, math.inf, -math.inf, 2.0 ** 116, -3.0e38)):
        h = (i * 7) % (G * H)
        q2[i % B, :, h, (5 + 40 * i) % d] = x
        bad[i % B, :, h] = True
    o, l = eio.attn_decode_kv4(q2, pool, table, n)
    sees = (L - 3 + 1 + torch.arange(3, device="cuda") > 0)[None, :, None] & torch.ones_like(bad)
    assert sees.all() == (L > 2)
    assert torch.equal(torch.isnan(o), (bad & sees)[..., None].expand_as(o))
    assert torch.equal(torch.isnan(l), (bad & sees).transpose(1, 2))
    assert torch.equal(o[~bad], want[~bad]) and torch.equal(l.transpose(1, 2)[~bad], lse.transpose(1, 2)[~bad])
    assert (o[~sees] == 0).all() and (l.transpose(1, 2)[~sees] == -math.inf).all()
    q2 = torch.zeros_like(q)
    q2[..., 3] = 2.0 ** 115.9
    o, l = eio.attn_decode_kv4(q2, pool, table, n, scale=2.0 ** -118)
    eio.sync_status()
    if L > 2:
        _check(o, l, q2, k, v, 2.0 ** -118)
