"""Arithmetic of paged attention: errors before the rounding to fp16, against sums in float64."""
import random

import pytest

import paged_ref as ref
from test_gpu_paged import _cache, _fill, _i32, _pages, _rows

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def _exact(cache, table, lens, q, scale):
    """[n][Hq][128] float64."""
    H, G = cache.cfg.num_kv_heads, q.shape[1] // cache.cfg.num_kv_heads
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for i, T in enumerate(lens):
        k, v, _, _ = _rows(cache, table, i, T)
        for h in range(H):
            out[i, h * G:(h + 1) * G] = ref.attend(q[i, h * G:(h + 1) * G].double(), k[h], v[h], scale, slice(None))
    return out


@pytest.mark.parametrize("bits, G", [(2, 1), (2, 2), (2, 4), (2, 7), (4, 1), (4, 4)])
def test_error_before_the_rounding(bits, G):
    """Values centred in their groups, so that sum p z takes most of sum p s c back: the output is small beside its terms.

    The 128 tokens of a sum take 8 steps of the tensor cores, each of which may cut the running sum off at 2^-23 of it, half
    of that on average: sum over k / 8 = 4.5 -> 4.5 * 2^-24 of the mean of s c = s (2^bits - 1) / 2.  Logits take 8 steps too;
    a cut of half a unit at each moves a weight by at most 8 * 2^-24 A, A = scale * sum |q| |s c| (natural logarithms), apart
    for every token, so that it moves an output of independent values by that share.  Everything else (operands of 22 bits, sums in
    fp32) is smaller.  The error before the rounding is the difference of the squared errors with and without it."""
    g = torch.Generator("cuda").manual_seed(3 + G)
    H, lens, scale = 4, [8001, 7000, 6100, 7777], 128 ** -0.5
    cache = _cache(num_pages=260, num_seqs=4, max_blocks=64, num_kv_heads=H, bits=bits)
    _fill(cache, g)
    top = 2 ** bits - 1
    for name in ("k", "v"):
        cache.view(name + "_zero").copy_(-0.5 * top * cache.view(name + "_scale"))
    table = _pages(cache, lens, random.Random(1))
    q = torch.randn(4, H * G, 128, generator=g, device="cuda").half()
    want = _exact(cache, table, lens, q, scale)
    got = cache.attend(_i32(lens), q).double()
    size = want.square().mean().sqrt()
    cut = 4.5 * 2.0 ** -24 * (cache.view("v_scale").double().mean() * top / 2) / size
    A = scale * q.abs().double().mean() * 128 * cache.view("k_scale").double().mean() * top / 2
    bound = (cut ** 2 + (8 * 2.0 ** -24 * A) ** 2).sqrt().item()
    rounding = (want.half().double() - want).square().mean()
    own = ((got - want).square().mean() - rounding).clamp(min=0).sqrt() / size
    print(f"own {own.item():.2e} bound {bound:.2e} rounding {(rounding.sqrt() / size).item():.2e}")
    assert own.item() <= bound
