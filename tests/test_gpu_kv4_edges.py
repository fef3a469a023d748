"""Rotary positions and the 4-bit cache on the GPU where values are not finite or lie far apart,
against fp64 (kv4_oracle and torch)."""
import numpy as np
import pytest
import torch

import exact_io_aware_sm_b200 as eio
from exact_io_aware_sm_b200 import autograd
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
