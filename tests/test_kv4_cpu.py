"""Host side of rotary positions and the 4-bit cache: refusals of the C ABI and of the
binding, the oracle's own consistency, the page accounting of Kv4Cache, and the
differentiable rope with the oracle in place of the library call."""
import ctypes
import math
import random

import numpy as np
import pytest
import torch

import exact_io_aware_sm_b200 as eio
from exact_io_aware_sm_b200 import autograd, build as ebuild, kv4_cache
from tests import kv4_oracle as ko

FAKE = 0x10000  # never dereferenced: every call here fails its checks first


@pytest.fixture(scope="module", autouse=True)
def built_lib():
    ebuild.build()
    return eio.lib()


# ------------------------------------------------------------------ C ABI
def _rope(**kw):
    a = dict(q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, pos=FAKE, axes=[0] * 16, freq=[1.0] * 16, strides=None, B=1, N=4, Hq=2,
             Hk=2, d=64, A=1, n=16, inter=0, inv=0, dt=0)
    a.update(kw)
    axes = None if a["axes"] is None else (ctypes.c_uint8 * len(a["axes"]))(*a["axes"])
    freq = None if a["freq"] is None else (ctypes.c_double * len(a["freq"]))(*a["freq"])
    st = (ctypes.c_int64 * 10)(*(a["strides"] or [512, 128, 512, 128, 512, 128, 512, 128, 4, 1]))
    return eio.lib().attn_rope(a["q"], a["k"], a["qo"], a["ko"], a["pos"], axes, freq, st, a["B"], a["N"], a["Hq"],
                               a["Hk"], a["d"], a["A"], a["n"], a["inter"], a["inv"], a["dt"], None)


@pytest.mark.parametrize("code,kw", [
    (1, dict(q=None)), (1, dict(k=None)), (1, dict(ko=None)), (1, dict(pos=None)), (1, dict(axes=None)),
    (1, dict(freq=None)), (2, dict(B=0)), (2, dict(N=0)), (2, dict(Hq=0)), (2, dict(Hk=-1)), (2, dict(Hq=70000)),
    (2, dict(B=1 << 16, N=1 << 15)), (4, dict(d=96)), (4, dict(dt=2)), (2, dict(A=0)), (2, dict(A=5)), (2, dict(n=0)),
    (2, dict(n=33, axes=[0] * 33, freq=[1.0] * 33)), (2, dict(axes=[0] * 15 + [1])),
    (2, dict(freq=[1.0] * 15 + [math.nan])), (2, dict(freq=[math.inf] + [1.0] * 15)), (2, dict(freq=[70000.0] * 16)),
    (3, dict(q=FAKE + 8)), (3, dict(pos=FAKE + 2)), (3, dict(strides=[516, 128, 512, 128, 512, 128, 512, 128, 4, 1])),
    (3, dict(strides=[512, 128, 512, 128, 512, 128, 512, 132, 4, 1])),
    (3, dict(strides=[512, 128, -512, 128, 512, 128, 512, 128, 4, 1])),
    (2, dict(strides=[512, 128, 512, 128, 512, 128, 512, 128, -4, 1]))])
def test_rope_refusals(code, kw):
    assert _rope(**kw) == code and eio.last_error()


def _append(**kw):
    a = dict(k=FAKE, v=FAKE, pool=FAKE, table=FAKE, lens=FAKE, new=None, st=[512, 128, 512, 128], B=1, N=4, H=2, d=64,
             n_pages=8, page=16, mp=4)
    a.update(kw)
    return eio.lib().attn_kv4_append(a["k"], a["v"], a["pool"], a["table"], a["lens"], a["new"],
                                     (ctypes.c_int64 * 4)(*a["st"]), a["B"], a["N"], a["H"], a["d"], a["n_pages"],
                                     a["page"], a["mp"], None)


def _read(**kw):
    a = dict(k=FAKE, v=FAKE, pool=FAKE, table=FAKE, lens=FAKE, start=None, B=1, N=4, H=2, d=64, n_pages=8, page=16, mp=4)
    a.update(kw)
    return eio.lib().attn_kv4_read(a["k"], a["v"], a["pool"], a["table"], a["lens"], a["start"], a["B"], a["N"], a["H"],
                                   a["d"], a["n_pages"], a["page"], a["mp"], None)


PAGE_REFUSALS = [
    (1, dict(k=None)), (1, dict(pool=None)), (1, dict(table=None)), (1, dict(lens=None)), (2, dict(B=0)), (2, dict(N=0)),
    (2, dict(H=0)), (2, dict(n_pages=0)), (2, dict(mp=0)), (4, dict(d=32)), (4, dict(page=48)), (4, dict(page=8)),
    (4, dict(page=512)), (2, dict(mp=1 << 27)), (2, dict(B=1 << 16, N=1 << 15)), (2, dict(B=1 << 20, N=1, H=1 << 15)), (2, dict(H=1 << 16)),
    (2, dict(B=(1 << 24) + 1)), (3, dict(k=FAKE + 8)),
    (3, dict(pool=FAKE + 16)), (3, dict(table=FAKE + 2))]


@pytest.mark.parametrize("code,kw", PAGE_REFUSALS + [(3, dict(new=FAKE + 1)), (3, dict(st=[512, 4, 512, 128])),
                                                     (3, dict(st=[512, 128, -8, 128]))])
def test_append_refusals(code, kw):
    assert _append(**kw) == code and eio.last_error()


@pytest.mark.parametrize("code,kw", PAGE_REFUSALS + [(3, dict(start=FAKE + 1))])
def test_read_refusals(code, kw):
    assert _read(**kw) == code and eio.last_error()


@pytest.mark.parametrize("kw", [dict(N=(1 << 30) + 1), dict(N=(1 << 31) - 1), dict(N=1 << 21, H=65535),
                                dict(B=8, N=1 << 20, H=5000)])
@pytest.mark.parametrize("call", [_append, _read])
def test_rows_past_32_bits_are_refused(call, kw):
    """Row positions and warps are numbered in 32 bits; broadcast rows reach such sizes without the memory."""
    assert call(**kw) == 2 and eio.last_error()


def _decode(**kw):
    a = dict(q=FAKE, pool=FAKE, table=FAKE, lens=FAKE, o=FAKE, lse=None, work=FAKE, n=1 << 40, B=1, Sq=1, Hq=4, H=2,
             d=64, n_pages=8, page=16, mp=4, scale=0.1)
    a.update(kw)
    return eio.lib().attn_decode_kv4(a["q"], a["pool"], a["table"], a["lens"], a["o"], a["lse"], a["work"], a["n"],
                                     a["B"], a["Sq"], a["Hq"], a["H"], a["d"], a["n_pages"], a["page"], a["mp"],
                                     a["scale"], None)


@pytest.mark.parametrize("code,kw", [
    (1, dict(q=None)), (1, dict(o=None)), (1, dict(lens=None)), (2, dict(Hq=3)), (2, dict(Sq=0)), (2, dict(B=0)),
    (2, dict(scale=0.0)), (2, dict(scale=math.nan)), (4, dict(d=96)), (4, dict(page=24)), (3, dict(q=FAKE + 4)),
    (3, dict(work=FAKE + 4)), (3, dict(lse=FAKE + 2)), (2, dict(Sq=1 << 20, Hq=4096))])
def test_decode_refusals(code, kw):
    assert _decode(**kw) == code and eio.last_error()


def test_decode_workspace_size():
    L = eio.lib()
    n = L.attn_decode_kv4_workspace(2, 1, 8, 2, 128, 64, 100)
    assert n >= 0
    assert L.attn_decode_kv4_workspace(2, 1, 7, 2, 128, 64, 100) == -1
    assert L.attn_decode_kv4_workspace(2, 1, 8, 2, 128, 63, 100) == -1
    if n:
        assert _decode(B=2, Hq=8, H=2, d=128, page=64, mp=100, work=None) == 8
        assert _decode(B=2, Hq=8, H=2, d=128, page=64, mp=100, n=n - 1) == 8


def _moves(src, dst, n_pages=8, nbytes=32, pool=FAKE):
    a, b = (None if x is None else (ctypes.c_int32 * max(1, len(x)))(*x) for x in (src, dst))
    return eio.lib().attn_copy_pages(pool, nbytes, n_pages, a, b, len(src or dst or [0]), None)


@pytest.mark.parametrize("code,args", [
    (1, ([0], [1], 8, 32, None)), (1, (None, [1])), (2, ([0], [8])), (2, ([-1], [1])), (2, ([0, 1], [2, 2])),
    (2, ([0, 1], [2, 0])), (2, ([3], [3])), (2, ([0], [1], 0)), (2, ([0], [1], 8, 24)), (2, ([0], [1], 8, 0)),
    (3, ([0], [1], 8, 32, FAKE + 8))])
def test_copy_pages_refusals(code, args):
    assert _moves(*args) == code and eio.last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_no_device_is_an_error():
    assert _rope() == 6 and _append() == 6 and _read() == 6 and _decode() == 6 and _moves([0], [1]) == 6


def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    pool = torch.zeros(8, 2, 18 * 64, dtype=torch.uint8)
    for call in (lambda: eio.rope(x, x, torch.zeros(1, 4, 1, dtype=torch.int32), [0], [1.0]),
                 lambda: eio.kv4_append(x, x, pool, i[None], i), lambda: eio.kv4_read(pool, i[None], i, 4, 64),
                 lambda: eio.attn_decode_kv4(x, pool, i[None], i), lambda: eio.copy_pages(pool, [0], [1])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    assert eio.kv4_page_bytes(64, 8, 128) == 64 * 8 * 144
    for page, d in ((48, 64), (16, 32)):
        with pytest.raises(ValueError, match="page"):
            eio.kv4_page_bytes(page, 1, d)


# ------------------------------------------------------------------ oracle
@pytest.mark.parametrize("d", [64, 128])
def test_oracle_pack_is_a_bijection_of_nibbles(d):
    rng = np.random.default_rng(d)
    ck, cv = rng.integers(0, 16, (2, 16, d))
    sk, sv = ko.bf16(rng.standard_normal((2, 16, d // 32)).astype(np.float32))
    b = ko.pack_tile(ck, sk, cv, sv)
    for x, y in zip(ko.unpack_tile(b, d), (ck, sk, cv, sv)):
        assert np.array_equal(x, y)


def test_oracle_quantiser_error_bound():
    """|(c - 8) s - x| <= s / 2, and m - 7 s where rounding left 7 s below m: s >= (m / 7)(1 - 2^-8)."""
    x = ko.bf16(np.random.default_rng(1).standard_normal((50, 64)).astype(np.float32) * 3)
    c, s = ko.quantise(x)
    err = np.abs(ko.value(c, s) - x).reshape(50, 2, 32)
    m = np.abs(x).reshape(50, 2, 32).max(-1)
    assert (err <= np.maximum(s / 2, m - 7 * s)[..., None] + 1e-12).all() and c.min() >= 1


# ------------------------------------------------------------------ accounting
class _Model:
    """What a cache holds, token by token: every append writes a fresh number."""

    def __init__(self):
        self.tokens, self.count = {}, 0


def _cache(monkeypatch, n_pages=40, page=16):
    cache = kv4_cache.Kv4Cache(n_pages, 1, 64, page=page, device="cpu")
    slots = np.full((n_pages, page), -1)

    def copy_pages(pool, src, dst, stream=None):
        assert not set(dst) & set(src) and len(set(dst)) == len(dst)
        slots[dst] = slots[src]
    monkeypatch.setattr(eio, "copy_pages", copy_pages)
    return cache, slots


def _write(slots, model, batch, page):
    for b, i in enumerate(batch.ids):
        n, new = int(batch.seqlens[b]), int(batch.n_new[b])
        for t in range(n - new, n):
            slots[int(batch.table[b, t // page]), t % page] = model.count
            model.tokens[i].append(model.count)
            model.count += 1


def _check(cache, slots, model):
    held = {}
    for i, tokens in model.tokens.items():
        assert cache.length(i) == len(tokens)
        s = cache._seqs[i]
        assert len(s.pages) == -(-len(tokens) // cache.page)
        assert [slots[s.pages[t // cache.page], t % cache.page] for t in range(len(tokens))] == tokens
        for p in s.pages:
            held[p] = held.get(p, 0) + 1
    assert {p: int(n) for p, n in enumerate(cache._refs) if n} == held
    assert sorted(cache._free) == sorted(set(range(cache.n_pages)) - set(held))


@pytest.mark.parametrize("seed", range(6))
def test_cache_accounting_against_a_token_model(monkeypatch, seed):
    """Random adds, extensions, forks, truncations, frees and compactions: every sequence
    reads back its own tokens, whatever was shared, copied or moved."""
    rng = random.Random(seed)
    cache, slots = _cache(monkeypatch)
    model = _Model()
    full = 0
    for _ in range(300):
        ids = list(model.tokens)
        what = rng.choice(["add", "extend", "extend", "extend", "fork", "free", "truncate", "compact"])
        if what == "add" and len(ids) < 12:
            model.tokens[cache.add()] = []
        elif what == "extend" and ids:
            some = rng.sample(ids, rng.randint(1, len(ids)))
            counts = [rng.choice([0, 1, 1, 5, 16, 33]) for _ in some]
            before = ([list(cache._seqs[i].pages) for i in ids], cache._refs.copy(), sorted(cache._free))
            try:
                batch = cache.extend(some, counts)
            except kv4_cache.Kv4Full:
                full += 1
                assert before[0] == [cache._seqs[i].pages for i in ids]
                assert np.array_equal(before[1], cache._refs) and before[2] == sorted(cache._free)
                continue
            _write(slots, model, batch, cache.page)
        elif what == "fork" and ids and len(ids) < 12:
            i = rng.choice(ids)
            model.tokens[cache.fork(i)] = list(model.tokens[i])
        elif what == "free" and ids and rng.random() < 0.5:
            i = rng.choice(ids)
            cache.free(i)
            del model.tokens[i]
        elif what == "truncate" and ids:
            i = rng.choice(ids)
            n = rng.randint(0, len(model.tokens[i]))
            cache.truncate(i, n)
            del model.tokens[i][n:]
        elif what == "compact":
            cache.compact()
            assert not cache._refs[cache.pages_used():].any()
        _check(cache, slots, model)
    assert full  # the pool did run out


def test_cache_refusals(monkeypatch):
    cache, _ = _cache(monkeypatch, n_pages=4)
    a = cache.add()
    with pytest.raises(ValueError, match="distinct"):
        cache.extend([a, a], 1)
    with pytest.raises(ValueError, match="distinct"):
        cache.batch([])
    with pytest.raises(ValueError, match="count"):
        cache.extend([a], [-1])
    with pytest.raises(ValueError, match="count"):
        cache.extend([a], [1, 2])
    with pytest.raises(ValueError, match="no sequence"):
        cache.fork(7)
    with pytest.raises(kv4_cache.Kv4Full):
        cache.extend([a], 65)
    old = cache.extend([a], 64)
    with pytest.raises(ValueError, match="length"):
        cache.truncate(a, 65)
    k = torch.zeros(1, 3, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="rows"):
        cache.append(0, k, k, old)
    with pytest.raises(ValueError, match="layer"):
        cache.append(1, k, k, old)
    cache.truncate(a, 10)
    with pytest.raises(ValueError, match="after the batch"):
        cache.append(0, k, k, old)
    new = cache.batch([a])
    cache.free(a)
    with pytest.raises(ValueError, match="after the batch"):
        cache.read(0, new, 4)
    with pytest.raises(ValueError):
        kv4_cache.Kv4Cache(0, 1, 64, device="cpu")


# ------------------------------------------------------------------ differentiable rope
AXES, FREQ = np.array([0, 0, 1, 1, 2], np.uint8), np.array([1.0, 0.1, 0.7, 0.02, 0.3])


def _orope(q, k, positions, axes, freq, interleaved, inverse):
    pos, sign = positions.numpy(), -1 if inverse else 1
    return tuple(None if x is None else torch.from_numpy(ko.rope(x.detach().numpy(), pos, axes, freq, interleaved, sign))
                 for x in (q, k))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradients_against_differences(interleaved):
    g = torch.Generator().manual_seed(3)
    q = torch.randn(2, 3, 2, 16, dtype=torch.float64, generator=g, requires_grad=True)
    k = torch.randn(2, 3, 1, 16, dtype=torch.float64, generator=g, requires_grad=True)
    pos = torch.randint(-50, 50, (2, 3, 3), generator=g)
    f = lambda q, k: autograd.rope(q, k, pos, AXES, FREQ, interleaved=interleaved, call=_orope)  # noqa: E731
    assert torch.autograd.gradcheck(f, (q, k)) and torch.autograd.gradgradcheck(f, (q, k))


def test_rope_gradients_of_one_output_and_of_broadcast_inputs():
    g = torch.Generator().manual_seed(4)
    base = torch.randn(1, 3, 1, 16, dtype=torch.float64, generator=g, requires_grad=True)
    k = torch.randn(2, 3, 2, 16, dtype=torch.float64, generator=g, requires_grad=True)
    pos = torch.randint(0, 50, (2, 3, 3), generator=g)
    q = base.expand(2, 3, 2, 16)
    yq, yk = autograd.rope(q, k, pos, AXES, FREQ, call=_orope)
    w = torch.randn(2, 3, 2, 16, dtype=torch.float64, generator=g)
    gk, = torch.autograd.grad((yk * w).sum(), k, retain_graph=True)
    np.testing.assert_allclose(gk, ko.rope(w.numpy(), pos.numpy(), AXES, FREQ, False, -1), atol=1e-14)
    (yq * w).sum().backward()
    want = ko.rope(w.numpy(), pos.numpy(), AXES, FREQ, False, -1).sum((0, 2), keepdims=True)
    np.testing.assert_allclose(base.grad, want, atol=1e-13)
    assert k.grad is None


@pytest.mark.parametrize("axes", [[256], [-1], [0.5], np.array([256 + 1], np.int64), np.array([True])])
def test_rope_refuses_axes_that_are_no_axis_numbers(axes):
    q = torch.zeros(1, 3, 2, 16, dtype=torch.float64)
    pos = torch.zeros(1, 3, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="axes"):
        autograd.rope(q, None, pos, axes, [1.0], call=_orope)
    for good in ([1], (1,), np.array([1], np.int32), np.array([1], np.uint8)):
        assert autograd.rope(q, None, pos, good, [1.0], call=_orope)[0].shape == q.shape
