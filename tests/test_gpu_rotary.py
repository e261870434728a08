"""Norms and rotation on the GPU against the formulas in float64."""
import pytest

import paged_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from bit_asymmetric_kv_02_b200 import kivi  # noqa: E402

HALF = 2.0 ** -11  # half a step of fp16


def _bound(want, pair_size):
    """One rounding to fp16 (relative, 2^-25 below the normal range) on values formed in 32 bits from a pair of
    size |a| + |b|: the norm (8 + 3 sum levels, rsqrt, two products), cos and sin (an angle of 2^-24 half turns and
    sincospif), two products and a sum are fewer than 32 roundings of 2^-24."""
    return want.abs() * HALF + 2.0 ** -25 + pair_size * 2.0 ** -19


def _check(rot_args, dtype, tokens, hq, hk, norm, positions, layout4=False, v=False):
    rd = rot_args.get("rotary_dim", 128)
    rot = kivi.Rotary(**rot_args)
    g = torch.Generator("cuda").manual_seed(tokens + hq)
    heads = hq + 2 * hk
    x = torch.randn(tokens, heads, 128, generator=g, device="cuda").to(dtype)
    wq, wk = ((1 + 0.2 * torch.randn(2, 128, generator=g, device="cuda")).to(dtype) if norm else (None, None))
    q, k, vv = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    before = x.clone()
    oq, ok, ov = rot.apply(q, k, vv if v else None, positions=positions, q_weight=wq, k_weight=wk, eps=1e-5)
    assert torch.equal(x, before) and oq.dtype == ok.dtype == torch.float16
    kw = {k_: rot_args[k_] for k_ in ("theta", "scaling", "factor", "low", "high") if k_ in rot_args}
    f, m = ref.frequencies(rd, original=rot_args.get("original_positions", 8192), **kw)
    f = torch.tensor(f, dtype=torch.float64, device="cuda")
    pos = positions if torch.is_tensor(positions) else positions + torch.arange(tokens, device="cuda")
    for got, src, w in ((oq, q, wq), (ok, k, wk)):
        src = src.double()
        want = ref.rotate(src, None if w is None else w.double(), 1e-5, pos, rd, rot_args.get("interleaved", False), f, m)
        base = ref.rotate(src, None if w is None else w.double(), 1e-5, pos * 0, 0, False, f[:0], 1.0)
        size = m * base.abs().amax(-1, keepdim=True) * 2  # a pair's size at most
        err = (got.double() - want).abs()
        assert (err <= _bound(want, size)).all(), (err - _bound(want, size)).max().item()
    if v:
        assert torch.equal(ov, vv.half())
    return oq, ok


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("rd, interleaved", [(128, False), (128, True), (64, False), (48, True), (16, False), (112, False), (0, False)])
def test_layouts(dtype, norm, rd, interleaved):
    _check(dict(rotary_dim=rd, interleaved=interleaved), dtype, 37, 6, 2, norm, 1000, v=True)


@pytest.mark.parametrize("scaling, high", [("none", 4.0), ("linear", 4.0), ("base", 4.0), ("bands", 4.0), ("ramp", 32.0)])
@pytest.mark.parametrize("tokens, hq, hk", [(1, 1, 1), (3, 32, 32), (700, 4, 1), (2000, 3, 1)])
def test_scalings(scaling, high, tokens, hq, hk):
    _check(dict(rotary_dim=128, theta=500000.0, scaling=scaling, factor=8.0, low=1.0, high=high, original_positions=4096),
           torch.bfloat16, tokens, hq, hk, True, 50000)


def test_positions():
    """Any order, repeated, negative, and the far ends of int32."""
    pos = torch.tensor([5, 5, 0, -1, -100000, 2 ** 31 - 1, -2 ** 31, 1 << 20, 77, 3], dtype=torch.int32, device="cuda")
    for inter in (False, True):
        _check(dict(rotary_dim=128, interleaved=inter, theta=10000.0), torch.float16, 10, 3, 1, False, pos)
    with pytest.raises(ValueError):
        _check({}, torch.float16, 10, 3, 1, False, 2 ** 31)
    with pytest.raises(kivi.KiviError):
        _check({}, torch.float16, 10, 3, 1, False, 2 ** 31 - 5)


def test_batched_layout_in_place_and_strides():
    """[B][heads][T][128], as the cache's prefill takes it: rows at position0 + i in every batch entry; fp16 in place."""
    rot = kivi.Rotary(theta=10000.0)
    g = torch.Generator("cuda").manual_seed(0)
    q = torch.randn(2, 5, 33, 128, generator=g, device="cuda").half()
    k = torch.randn(2, 33, 3, 128, generator=g, device="cuda").half().transpose(1, 2)
    oq, ok, _ = rot.apply(q, k, positions=9)
    for b in range(2):
        a, c, _ = rot.apply(q[b].transpose(0, 1), k[b].transpose(0, 1), positions=9)
        assert torch.equal(oq[b], a.transpose(0, 1)) and torch.equal(ok[b], c.transpose(0, 1))
    pos = (9 + torch.arange(33, device="cuda")).int().repeat(2, 1)
    assert torch.equal(rot.apply(q, k, positions=pos)[0], oq)
    q2, k2 = q.clone(), k.clone()
    rot.apply(q2, k2, positions=9, q_out=q2, k_out=k2)
    assert torch.equal(q2, oq) and torch.equal(k2, ok)


def test_zeros_infinities_and_range():
    """A row of zeros under the norm stays zero; what exceeds fp16 becomes infinite; NaN stays in its head row."""
    rot = kivi.Rotary()
    x = torch.zeros(4, 2, 128, device="cuda", dtype=torch.bfloat16)
    x[1, 0] = 1e6
    x[2, 1, 5] = float("nan")
    w = torch.ones(128, device="cuda", dtype=torch.bfloat16)
    q, k, _ = rot.apply(x, x, positions=0, k_weight=w)
    assert not q[0].any() and not k[0].any()
    assert torch.isinf(q[1, 0]).any() and torch.isfinite(k[1, 0]).all()
    assert q[2, 1].isnan().any() and torch.isfinite(q[2, 0]).all() and torch.isfinite(q[3]).all()
    assert k[2, 1].isnan().all() and torch.isfinite(k[2, 0]).all()


def test_refusals():
    rot = kivi.Rotary()
    x = torch.zeros(4, 2, 128, device="cuda", dtype=torch.float16)
    for bad in (lambda: rot.apply(x.float(), x.float()), lambda: rot.apply(x, x.bfloat16()), lambda: rot.apply(x, x[:3]),
                lambda: rot.apply(x, x[..., :64]), lambda: rot.apply(x[0], x[0]), lambda: rot.apply(x.cpu(), x.cpu()),
                lambda: rot.apply(x, x, positions=torch.zeros(4, device="cuda")),
                lambda: rot.apply(x, x, positions=torch.zeros(3, device="cuda", dtype=torch.int32)),
                lambda: rot.apply(x, x, q_weight=torch.ones(64, device="cuda").half()), lambda: rot.apply(x, x, q_out=x.bfloat16()),
                lambda: rot.apply(x, x, q_out=x[:, :1].expand(4, 2, 128)), lambda: rot.apply(x.transpose(1, 2).contiguous().transpose(1, 2), x)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(kivi.KiviError):
        base = torch.zeros(4, 2 * 132, device="cuda", dtype=torch.float16)
        rot.apply(base.view(4, 2, 132)[..., 4:], x)  # head rows that do not start on 16 bytes
    empty = torch.zeros(0, 2, 128, device="cuda", dtype=torch.float16)
    assert rot.apply(empty, empty)[0].shape == (0, 2, 128)


def test_step_rotary_of_the_contiguous_cache():
    rot = kivi.Rotary(rotary_dim=64)
    for dtype in (torch.float16, torch.bfloat16):
        a, b = (kivi.KiviCache(2, 2, 512, num_q_heads=4) for _ in range(2))
        g = torch.Generator("cuda").manual_seed(3)
        k = torch.randn(2, 2, 126, 128, generator=g, device="cuda").half()
        a.prefill(k, k)
        b.prefill(k, k)
        w = torch.rand(128, generator=g, device="cuda").to(dtype)
        for step in range(5):
            q, kn, vn = (torch.randn(2, h, 128, generator=g, device="cuda").to(dtype) for h in (4, 2, 2))
            out = a.step_rotary(rot, kn, vn, q, q_weight=w, k_weight=w)
            pos = torch.full((2,), 126 + step, dtype=torch.int32, device="cuda")
            q2, k2, _ = rot.apply(q, kn, positions=pos, q_weight=w, k_weight=w)
            assert torch.equal(out, b.step(k2, vn.half(), q2))
        # slices of a fused projection are the same rows
        x = torch.randn(2, 8, 128, generator=g, device="cuda").to(dtype)
        q, kn, vn = x[:, :4], x[:, 4:6], x[:, 6:]
        out = a.step_rotary(rot, kn, vn, q)
        assert torch.equal(out, b.step_rotary(rot, kn.contiguous(), vn.contiguous(), q.contiguous()))
        with pytest.raises(ValueError):
            a.step_rotary(rot, kn[:, :1], vn, q)
        assert (a.n_quant, a.n_res) == (b.n_quant, b.n_res) == (128, 4)
        assert torch.equal(a.view("v_res")[:, :, :4], b.view("v_res")[:, :, :4])
        assert torch.equal(a.view("k_codes")[:, :, :128], b.view("k_codes")[:, :, :128])


def test_step_rotary_output_and_stream():
    """A given output is checked before the cache changes; on another stream the step's own tensors are that stream's."""
    g = torch.Generator("cuda").manual_seed(6)
    rot = kivi.Rotary()
    a, b = (kivi.KiviCache(2, 2, 512, num_q_heads=4) for _ in range(2))
    x = torch.randn(2, 8, 128, generator=g, device="cuda").bfloat16()
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    for bad in (torch.zeros(2, 4, 128, device="cuda"), torch.zeros(1, 4, 128, dtype=torch.float16, device="cuda"),
                torch.zeros(2, 8, 128, dtype=torch.float16, device="cuda")[:, ::2], torch.zeros(2, 4, 128, dtype=torch.float16)):
        with pytest.raises(ValueError):
            a.step_rotary(rot, k, v, q, out=bad)
        assert (a.n_quant, a.n_res) == (0, 0)
    out = torch.zeros(2, 4, 128, dtype=torch.float16, device="cuda")
    assert a.step_rotary(rot, k, v, q, out=out) is out
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = b.step_rotary(rot, k, v, q, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, out) and a.read_status() == b.read_status() == 0
