"""The e4m3 slots of pa_rotary_append_varlen hold the quotient by the scale, rounded once to fp32 and
once to e4m3: bit by bit what the same two roundings give on the CPU.  Values that do not turn (v) have
no other rounding in front."""

import pytest
import torch

import paged_kv_cache_page_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def stored(x, scale, rot):
    """v [T, Hkv, D] as it comes back from an e4m3 cache."""
    T, hkv, d = x.shape
    pages = -(-T // 16)
    caches = [torch.zeros((pages, 16, hkv, d), dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2)]
    ang = torch.zeros((4, rot // 2), dtype=torch.float32, device=DEV)
    x = x.to(DEV)
    pa.pa_rotary_append_varlen(None, x, x, *caches, torch.arange(T, device=DEV),
                               positions=torch.zeros(T, dtype=torch.int32, device=DEV),
                               rotary_cos=ang.cos(), rotary_sin=ang.sin(),
                               k_scale=scale.to(DEV), v_scale=scale.to(DEV))
    return caches[1].view(torch.uint8).view(-1, hkv, d)[:T].cpu()


def quotient(x, scale):
    return (x.float() / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def same(got, want):
    nan = (want & 0x7f) == 0x7f
    return torch.equal((got & 0x7f) == 0x7f, nan) and torch.equal(got[~nan], want[~nan])


# 64: the kernel that takes 16 features a thread; 20: the one that takes a pair
@pytest.mark.parametrize("rot", [64, 20])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_quotients_next_to_a_midpoint(rot, dtype):
    """Scales that put a quotient onto a midpoint of two e4m3 values, or a step of fp32 beside it, among
    the normal values and among the subnormal ones."""
    g = torch.Generator().manual_seed(rot)
    heads, T, d = 96, 6, 64
    x = (1 + torch.rand(heads, generator=g)).to(dtype)
    j = torch.randint(0, 8, (heads,), generator=g).float()
    mid = torch.where(torch.arange(heads) % 3 == 2, (2 * j + 1) * 2.0 ** -10, 1 + (2 * j + 1) / 16)
    scale = x.float() / mid
    v = x[None, :, None] * (2.0 ** (torch.arange(d) % 7 - 3)).to(dtype) * (1 - 2 * (torch.arange(d) % 2)).to(dtype)
    v = v * (2.0 ** (torch.arange(T) - 2)).to(dtype)[:, None, None]
    assert same(stored(v, scale, rot), quotient(v, scale))


@pytest.mark.parametrize("rot", [64, 20])
def test_any_value_and_scale(rot):
    g = torch.Generator().manual_seed(7 + rot)
    v = torch.randn((70, 8, 128), generator=g) * torch.tensor(2.0) ** torch.randint(-12, 9, (70, 1, 1), generator=g)
    v = v.bfloat16()
    scale = torch.exp(torch.randn(8, generator=g) * 2) * torch.tensor([1.0, -1.0]).repeat(4)
    assert same(stored(v, scale, rot), quotient(v, scale))


@pytest.mark.parametrize("rot", [64, 20])
def test_scales_at_the_ends_of_the_range(rot):
    """Scales whose reciprocal fp32 does not hold, or not with all its bits: a zero stays a zero."""
    inf, nan = float("inf"), float("nan")
    scale = torch.tensor([2.0 ** -130, -(2.0 ** -149), 2.0 ** -127, 1.5 * 2.0 ** 126, -3.0e38, inf, nan, 0.0])
    v = torch.tensor([0.0, -0.0, 1.0, -2.5, 2.0 ** -130, 3.0 * 2.0 ** -133, 3e38, -1e30, 2.0 ** 120, inf, -inf, nan,
                      2.0 ** -126, 2.0 ** -124, 0.375, 7.0]).repeat(4).bfloat16()
    v = v[None, None, :].repeat(3, 8, 1)
    assert same(stored(v, scale, rot), quotient(v, scale))
