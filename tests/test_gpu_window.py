"""Sliding window and sinks over the contiguous cache, against the formula in float64."""
import pytest

import paged_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from bit_asymmetric_kv_02_b200 import kivi  # noqa: E402

NAN = float("nan")


def _cache(B, H, T, bits, R, gk, gv, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    nq = (T - 1) // R * R
    cache = kivi.KiviCache(B, H, nq + R, bits=bits, group_k=gk, group_v=gv, residual=R)
    k = torch.randn(B, H, T, 128, generator=g, device="cuda").half()
    v = torch.randn(B, H, T, 128, generator=g, device="cuda").half()
    cache.prefill(k, v)
    assert (cache.n_quant, cache.n_res) == (nq, T - nq)
    return cache, g


def _rows(cache, b):
    c, nq, nr = cache.cfg, cache.n_quant, cache.n_res
    R, H, nb, P = c.residual, c.num_kv_heads, nq // c.residual, 32 // c.bits
    parts = ref.dequantised(cache.view("k_codes")[b, :, :nq].reshape(H, nb, R, 128 // P),
                            cache.view("v_codes")[b, :, :nq // P].reshape(H, nb, R // P, 128),
                            *(cache.view(x)[b, :, :nb] for x in ("k_scale", "k_zero")),
                            *(cache.view(x)[b, :, :nq // c.group_v].reshape(H, nb, R // c.group_v) for x in ("v_scale", "v_zero")), c.bits)
    out = []
    for i, (p, res) in enumerate(zip(parts, ("k_res", "v_res") * 2)):
        r = cache.view(res)[b, :, :nr].double()
        out.append(torch.cat([p.reshape(H, nq, 128), r if i < 2 else r.abs()], 1))
    return out


def _check(cache, q, out, window, sinks, scale=128 ** -0.5):
    T, G = cache.n_quant + cache.n_res, q.shape[1] // cache.cfg.num_kv_heads
    keep = torch.from_numpy(ref.visible(T, window, sinks)).cuda()
    for b in range(cache.cfg.batch):
        k, v, ka, va = _rows(cache, b)
        for h in range(cache.cfg.num_kv_heads):
            qh = q[b, h * G:(h + 1) * G].double()
            want = ref.attend(qh, k[h], v[h], scale, keep)
            err = (out[b, h * G:(h + 1) * G].double() - want).abs()
            tol = ref.attend_bound(qh, ka[h], va[h], scale, keep, want)
            assert (err <= tol).all(), (b, h, err.max().item(), (err - tol).max().item())


@pytest.mark.parametrize("window, sinks", [(1, 0), (2, 1), (100, 4), (128, 128), (700, 131), (3000, 5), (0, 0), (40, 5000)])
@pytest.mark.parametrize("T", [1, 128, 129, 1000, 1921])
@pytest.mark.parametrize("bits, G, R, gk, gv", [(2, 1, 128, 32, 32), (2, 5, 256, 128, 64), (4, 4, 128, 64, 128), (2, 2, 1024, 32, 1024)])
def test_window(T, window, sinks, bits, G, R, gk, gv):
    cache, g = _cache(2, 2, T, bits, R, gk, gv, seed=T)
    nq = cache.n_quant
    keep = ref.visible(T, window, sinks)
    for t in range(nq, nq + R):  # residual rows behind the tokens, or hidden
        if t >= T or not keep[t]:
            cache.view("k_res")[:, :, t - nq] = NAN
            cache.view("v_res")[:, :, t - nq] = NAN
    for j in range(nq // R):     # blocks the window hides whole are not read
        if not keep[j * R:(j + 1) * R].any():
            for name in ("k_scale", "k_zero"):
                cache.view(name)[:, :, j] = NAN
            for name in ("v_scale", "v_zero"):
                cache.view(name)[:, :, j * R // gv:(j + 1) * R // gv] = NAN
    q = torch.randn(2, 2 * G, 128, generator=g, device="cuda").half()
    out = cache.attend_window(q, window, sinks=sinks)
    safe = {n: torch.nan_to_num(cache.view(n)) for n in ("k_scale", "k_zero", "v_scale", "v_zero", "k_res", "v_res")}
    for n, x in safe.items():
        cache.view(n).copy_(x)
    _check(cache, q, out, window, sinks)
    assert cache.read_status() == 0


def test_full_residual_and_no_blocks():
    """n_res = R with blocks before it, and residual tokens alone, as append and flush leave them."""
    cache, g = _cache(1, 2, 255, 2, 128, 32, 32)
    x = torch.randn(1, 2, 128, generator=g, device="cuda").half()
    cache.append(x, x)
    assert (cache.n_quant, cache.n_res) == (128, 128)
    q = torch.randn(1, 4, 128, generator=g, device="cuda").half()
    _check(cache, q, cache.attend_window(q, 130, sinks=2), 130, 2)
    cache.flush()
    assert (cache.n_quant, cache.n_res) == (256, 0)
    _check(cache, q, cache.attend_window(q, 130, sinks=2), 130, 2)
    _check(cache, q, cache.attend_window(q, 1), 1, 0)


def test_no_window_is_attend():
    cache, g = _cache(2, 2, 900, 2, 128, 32, 32)
    q = torch.randn(2, 2, 128, generator=g, device="cuda").half()
    a, b = cache.attend(q), cache.attend_window(q, 0)
    # two roundings to fp16 of outputs below 1/2 and 2^-12 of arithmetic
    assert (a.double() - b.double()).abs().max() <= 2.0 ** -11


def test_capture_stream_and_refusals():
    cache, g = _cache(2, 2, 900, 4, 128, 32, 32)
    q = torch.randn(2, 8, 128, generator=g, device="cuda").half()
    out = torch.empty_like(q)
    with pytest.raises(RuntimeError):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            cache.attend_window(q, 100)
    want = cache.attend_window(q, 100, sinks=3)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = cache.attend_window(q, 100, sinks=3, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attend_window(q, 100, sinks=3, out=out)
    q.copy_(torch.randn(q.shape, generator=g, device="cuda").half())
    graph.replay()
    assert torch.equal(out, cache.attend_window(q, 100, sinks=3))
    for bad in (lambda: cache.attend_window(q.float(), 1), lambda: cache.attend_window(q[:1], 1), lambda: cache.attend_window(q, 1 << 31),
                lambda: cache.attend_window(q, 1, out=out[:, :2])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(kivi.KiviError):
        cache.attend_window(q[:, :3].contiguous(), 1)
    with pytest.raises(kivi.KiviError):
        kivi.KiviCache(1, 1, 128).attend_window(q[:1, :1].contiguous(), 1)
    with pytest.raises(kivi.KiviError):
        kivi.KiviCache(1, 1, 128, fine_groups=True).attend_window(q[:1, :1].contiguous(), 1)
