"""Host side of rotary positions and the 4-bit cache where a call fails midway, where a
tensor is not laid out as the library reads it, and where sizes pass what is counted in."""
import numpy as np
import pytest
import torch

import exact_io_aware_sm_b200 as eio
from exact_io_aware_sm_b200 import autograd, kv4_cache
from tests import kv4_oracle as ko


# ------------------------------------------------------------------ a cache whose device work fails
def _state(cache):
    return ({i: (list(s.pages), s.length, s.version) for i, s in cache._seqs.items()}, cache._refs.tolist(),
            sorted(cache._free))


def _forked(monkeypatch, layers=1):
    """Two sequences that share a full page and a part-filled one; copies are recorded."""
    copies = []
    monkeypatch.setattr(eio, "copy_pages", lambda pool, src, dst, stream=None: copies.append((list(src), list(dst))))
    cache = kv4_cache.Kv4Cache(12, 1, 64, page=16, layers=layers, device="cpu")
    a = cache.add()
    old = cache.extend([a], 21)
    return cache, a, cache.fork(a), old, copies


@pytest.mark.parametrize("counts", [[1, 1], [16, 0], [40, 3]])
@pytest.mark.parametrize("fails", ["first copy", "second layer's copy", "upload"])
def test_an_extend_that_fails_leaves_the_cache_as_it_was(monkeypatch, fails, counts):
    """A page copy or an upload that raises: no page, length, count or version has changed,
    older batches stay valid, and the same call works once the cause is gone."""
    cache, a, b, old, copies = _forked(monkeypatch, layers=2)
    before, calls = _state(cache), []

    def copy_pages(pool, src, dst, stream=None):
        calls.append((list(src), list(dst)))
        if fails != "upload" and len(calls) == (1 if fails == "first copy" else 2):
            raise eio.AttnError(6, "a copy that fails")

    def no_upload(x):
        raise RuntimeError("out of memory")
    with monkeypatch.context() as m:
        m.setattr(eio, "copy_pages", copy_pages)
        if fails == "upload":
            m.setattr(torch, "from_numpy", no_upload)
        with pytest.raises(RuntimeError):
            cache.extend([a, b], counts)
        assert calls
    assert _state(cache) == before
    assert cache._current(0, old) is not None
    batch = cache.extend([a, b], counts)
    assert copies[0] == ([1], [2]) and copies[1] == copies[0]
    assert [cache.length(i) for i in (a, b)] == [21 + n for n in counts] == batch.seqlens.tolist()
    for r, i in enumerate((a, b)):
        pages = cache._seqs[i].pages
        assert len(pages) == -(-cache.length(i) // 16) and batch.table[r, :len(pages)].tolist() == pages
    assert cache._seqs[a].pages[1] == 2 and cache._seqs[b].pages[1] == 1


def test_a_compaction_that_fails_leaves_the_cache_as_it_was(monkeypatch):
    cache, a, b, old, _ = _forked(monkeypatch)
    c = cache.add()
    cache.extend([c], 5)
    cache.free(a)
    cache.free(b)
    before = _state(cache)

    def copy_pages(pool, src, dst, stream=None):
        raise eio.AttnError(6, "a copy that fails")
    with monkeypatch.context() as m:
        m.setattr(eio, "copy_pages", copy_pages)
        with pytest.raises(eio.AttnError):
            cache.compact()
    assert _state(cache) == before
    assert cache.compact() == 1 and cache._seqs[c].pages == [0]


# ------------------------------------------------------------------ differentiable rope
AXES, FREQ = np.array([0, 0, 1, 1, 2], np.uint8), np.array([1.0, 0.1, 0.7, 0.02, 0.3])


def _off_by(x, n):
    """x's values at element n of a flat buffer: contiguous, but not on a 16-byte boundary."""
    flat = torch.empty(n + x.numel(), dtype=x.dtype)
    y = flat[n:].view(x.shape)
    y.copy_(x)
    return y


def _orope(q, k, positions, axes, freq, interleaved, inverse):
    """The oracle behind the library's own conditions on addresses and strides."""
    for x in (q, k):
        if x is not None:
            B, N, H, d = x.shape
            sb, sn, sh, sd = x.stride()
            assert x.data_ptr() % 16 == 0 and sd == 1 and (H == 1 or sh == d)
            assert all(s * x.element_size() % 16 == 0 for s, n in ((sb, B), (sn, N)) if n > 1)
    return tuple(None if x is None else
                 torch.from_numpy(ko.rope(x.detach().double().numpy(), positions.numpy(), axes, freq, interleaved,
                                          -1 if inverse else 1)).to(x.dtype) for x in (q, k))


@pytest.mark.parametrize("dtype,n", [(torch.bfloat16, 4), (torch.bfloat16, 1), (torch.float32, 2), (torch.float64, 1)])
def test_rope_takes_misaligned_inputs_and_gradients(dtype, n):
    """q, k or a gradient that starts off a 16-byte boundary is copied, not refused: the same answers."""
    g = torch.Generator().manual_seed(n)
    q, k, dq, dk = (torch.randn(2, 3, h, 16, generator=g, dtype=torch.float64).to(dtype) for h in (2, 1, 2, 1))
    pos = torch.randint(0, 50, (2, 3, 3), generator=g)

    def both(put):
        x, y = put(q).requires_grad_(), put(k).requires_grad_()
        out = autograd.rope(x, y, pos, AXES, FREQ, call=_orope)
        return [t.detach() for t in out] + list(torch.autograd.grad(out, (x, y), (put(dq), put(dk))))
    assert _off_by(q, n).data_ptr() % 16
    for got, want in zip(both(lambda x: _off_by(x, n)), both(torch.clone)):
        assert torch.equal(got, want)


def test_rope_computes_only_the_gradients_that_are_wanted():
    g = torch.Generator().manual_seed(9)
    q, k = (torch.randn(2, 3, h, 16, generator=g, dtype=torch.float64) for h in (2, 1))
    w = torch.randn(2, 3, 2, 16, generator=g, dtype=torch.float64)
    pos = torch.randint(0, 50, (2, 3, 3), generator=g)
    calls = []

    def call(q, k, *rest):
        calls.append((q is not None, k is not None))
        return _orope(q, k, *rest)
    want = torch.from_numpy(ko.rope(w.numpy(), pos.numpy(), AXES, FREQ, False, -1))
    for frozen in ("k", "q", None):
        x, y = q.clone().requires_grad_(frozen != "q"), k.clone().requires_grad_(frozen != "k")
        yq, yk = autograd.rope(x, y, pos, AXES, FREQ, call=call)
        calls.clear()
        (yq * w + yk * w).sum().backward()
        assert len(calls) == 1 and sum(calls[0]) == (1 if frozen else 2)
        assert x.grad is None if frozen == "q" else torch.allclose(x.grad, want, atol=1e-14)
        assert y.grad is None if frozen == "k" else torch.allclose(y.grad, want.sum(2, keepdim=True), atol=1e-13)
    # one gradient of two leaves, and a second derivative with k frozen
    x, y = q.clone().requires_grad_(), k.clone().requires_grad_()
    yq, yk = autograd.rope(x, y, pos, AXES, FREQ, call=call)
    assert torch.allclose(torch.autograd.grad((yq * w + yk * w).sum(), x)[0], want, atol=1e-14)
    u = w.clone().requires_grad_()
    yq, yk = autograd.rope(x, k, pos, AXES, FREQ, call=call)
    gx, = torch.autograd.grad((yq * u + yk * u).sum(), x, create_graph=True)
    gu, = torch.autograd.grad((gx * q).sum(), u)
    assert torch.allclose(gu, torch.from_numpy(ko.rope(q.numpy(), pos.numpy(), AXES, FREQ, False)), atol=1e-13)


# ------------------------------------------------------------------ sizes
def _decode(B, Sq, Hq, H, mp, page=256, n=1 << 60):
    fake = 0x10000  # never dereferenced: the calls fail their checks, or find no device
    return eio.lib().attn_decode_kv4(fake, fake, fake, fake, fake, None, fake, n, B, Sq, Hq, H, 64, 8, page, mp, 0.1,
                                     None)


# Columns go in blocks of 8, keys in stages of 32 with three more for a block's start and end.
@pytest.mark.parametrize("B,Sq,Hq,H,mp", [(1, 1 << 20, 1 << 10, 1, 1 << 22), (1, 1 << 20, 1, 1, 1 << 22),
                                          (1 << 10, 1, 1 << 13, 1 << 13, 1 << 21), (1, 8, 1 << 20, 1, 1 << 18)])
def test_decode_refuses_more_work_than_its_counts_hold(B, Sq, Hq, H, mp):
    """A warp's stages are counted in 32 bits; pages may repeat in a table, so little memory reaches past them."""
    assert -(-Hq // H * Sq // 8) * B * H * (mp * 8 + 3) >= 2 ** 41
    assert _decode(B, Sq, Hq, H, mp) == 2 and "work" in eio.last_error()
    assert eio.lib().attn_decode_kv4_workspace(B, Sq, Hq, H, 64, 256, mp) == -1


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")
@pytest.mark.parametrize("B,Sq,Hq,H,mp", [(1, 1, 32, 8, 1 << 22), (4096, 1, 64, 8, 1 << 12), (1, 4096, 64, 8, 1 << 14),
                                          (1 << 20, 1, 8, 1, 1 << 10)])
def test_decode_takes_large_work_that_its_counts_hold(B, Sq, Hq, H, mp):
    assert _decode(B, Sq, Hq, H, mp) == 6  # every check passed: there is no device


# ------------------------------------------------------------------ a cache and rows of another head size
def test_cache_refuses_rows_and_queries_of_another_head_size(monkeypatch):
    """A page of 64 tokens of 128 channels has as many bytes as one of 128 tokens of 64: the pool alone does not
    tell them apart, the cache does."""
    assert eio.kv4_page_bytes(64, 1, 128) == eio.kv4_page_bytes(128, 1, 64)
    called = []
    for name in ("kv4_append", "attn_decode_kv4"):
        monkeypatch.setattr(eio, name, lambda *a, **kw: called.append(a))
    cache = kv4_cache.Kv4Cache(4, 2, 128, page=64, device="cpu")
    a = cache.add()
    batch = cache.extend([a], 3)
    for d in (64, 32):
        k = torch.zeros(1, 3, 2, d, dtype=torch.bfloat16)
        with pytest.raises(ValueError, match="d = 128"):
            cache.append(0, k, k, batch)
        with pytest.raises(ValueError, match="d = 128"):
            cache.decode(0, k[:, :1], batch)
    assert not called
    k = torch.zeros(1, 3, 2, 128, dtype=torch.bfloat16)
    cache.append(0, k, k, batch)
    cache.decode(0, k[:, :1], batch)
    assert len(called) == 2


@pytest.mark.parametrize("d,columns,MB", [(64, 4, 2.7), (64, 8, 5.3), (128, 4, 5.2), (128, 8, 8.0)])
def test_decode_workspace_sizes(d, columns, MB):
    """149 starts of runs, and for each of 148 CTAs a slot a warp (15, or 11 where 8 columns of 128 channels need the
    registers) and two that leave it: fp32 numerators, a maximum and a sum a column.  Longer contexts need no more."""
    size = eio.lib().attn_decode_kv4_workspace
    warps = 11 if columns == 8 and d == 128 else 15
    slot = columns * (d + 2) * 4
    want = 149 * 32 + 148 * (warps + 2) * slot
    assert round(want / 1e6, 1) == MB
    for G, Sq in ((columns, 1), (columns // 4, 4), (2 * columns - 1 if columns == 8 else columns, 1)):
        for B, H, mp in ((64, 8, 128), (1, 8, 8192), (1, 1, 1 << 24)):
            assert size(B, Sq, G * H, H, d, 64, mp) == want
    # fewer stages of 32 keys than SMs: as many CTAs
    assert size(1, 1, columns, 1, d, 16, 3) == 149 * 32 + 2 * (warps + 2) * slot
