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


@pytest.mark.parametrize("where", ["before", "beside"])
@pytest.mark.parametrize("bits, G", [(2, 1), (4, 1), (2, 2), (2, 4), (4, 3), (2, 7)])
def test_large_values_without_weight(bits, G, where):
    """Groups of V with a scale 2^25 above the others', whose tokens have next to no weight: in blocks before the others, or
    in the same blocks.  A logit's error is below 2^-20 A and a weight's delta = 2 * 2^-20 A + 2^-20 relative, as in
    attend_bound; the output moves by at most 2 delta times the weighted mean of the values' sizes.  700 sequences of the same
    pages, so that a warp goes through several blocks of a head."""
    g = torch.Generator("cuda").manual_seed(bits + G)
    top, R, T, H, n = 2 ** bits - 1, 128, 641, 2, 700
    cache = _cache(num_seqs=n, num_kv_heads=H, bits=bits)
    _fill(cache, g)
    table = _pages(cache, [T], random.Random(2))
    cache.view("block_table").copy_(cache.view("block_table")[:1].expand(n, -1).clone())
    at = torch.from_numpy(table[0, :5]).long().cuda()
    block, tok = torch.arange(5, device="cuda")[:, None], torch.arange(R, device="cuda")[None]
    light = (block < 2).expand(5, R) if where == "before" else ((tok // 32) % 2 == 0).expand(5, R)
    # keys: every channel's code 0 for the light tokens; `top` for the others, but for four channels
    P = 32 // bits
    code = torch.where(light[:, None, :, None], 0, top).expand(5, H, R, 128).clone()
    code[..., :4] = torch.where(light[:, None, :, None], 0, torch.randint(0, top + 1, (5, H, R, 4), generator=g, device="cuda"))
    words = (code.long().view(5, H, R, 128 // P, P) << (torch.arange(P, device="cuda") * bits)).sum(-1)
    cache.view("k_codes")[at] = torch.where(words >= 2 ** 31, words - 2 ** 32, words).int()
    cache.view("k_scale").fill_(3 / top)
    cache.view("k_zero").zero_()
    cache.view("k_res").zero_()
    big = light.view(5, 1, 4, 32)[..., 0].expand(5, H, 4)
    cache.view("v_scale")[at] = torch.where(big, 2.0 ** 13 * 3 / top, 2.0 ** -12).half()
    cache.view("v_zero")[at] = -0.5 * top * cache.view("v_scale")[at]
    cache.view("v_res").zero_()
    q = (0.5 + torch.rand(1, H * G, 128, generator=g, device="cuda")).half()
    scale = 128 ** -0.5
    out = cache.attend(_i32([T] * n), q.expand(n, -1, -1).contiguous())
    k, v, ka, va = _rows(cache, table, 0, T)
    for h in range(H):
        qh = q[0, h * G:(h + 1) * G].double()
        w = torch.softmax(qh @ k[h].T * scale, -1)
        want = w @ v[h]
        A = (qh.abs() @ ka[h].T * scale).max()
        half_step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0 ** -14))) - 11)
        tol = half_step + (2 * A + 4) * 2.0 ** -19 * (w @ va[h])
        err = (out[:, h * G:(h + 1) * G].double() - want).abs()
        assert (err <= tol).all(), (h, (err / tol).max().item(), err.max().item())
