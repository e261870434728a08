"""Paged cache, rotary and windowed attention on the host: what the calls refuse before anything is enqueued, buffer
sizes, and the rotation's fixed-point frequencies.  Pointers are fakes that no call dereferences."""
import ctypes
import math

import pytest

import paged_ref as ref

FAKE = 1 << 20


@pytest.fixture(scope="module")
def kivi():
    from bit_asymmetric_kv_02_b200 import build, kivi as k
    build.build()
    k.load_library()
    return k


def _cfg(kivi, **kw):
    base = dict(num_pages=40, num_seqs=4, max_blocks=8, num_kv_heads=2, head_dim=128, bits=2, group_k=32, group_v=32,
                residual=128)
    base.update(kw)
    return kivi.kivi_paged_config(**base)


def _cache(kivi, **kw):
    c = kivi.kivi_paged_cache(*([FAKE] * len(kivi.PAGED_BUFFERS)))
    for name, value in kw.items():
        setattr(c, name, value)
    return c


def _plan(kivi, **kw):
    p = kivi.kivi_paged_plan(FAKE, FAKE, FAKE, FAKE, 256, 10)
    for name, value in kw.items():
        setattr(p, name, value)
    return p


def _refused(kivi, code, fn, *args):
    with pytest.raises(kivi.KiviError) as e:
        fn(*args)
    assert e.value.code == code


def test_config_rules(kivi):
    check = kivi.kivi_paged_check_config
    assert check(_cfg(kivi)) == 0
    for R in (128, 256, 512):
        assert check(_cfg(kivi, residual=R, group_v=R)) == 0
    assert check(_cfg(kivi, residual=1024)) == 2
    assert check(_cfg(kivi, residual=64)) == 1
    assert check(_cfg(kivi, bits=3)) == 2
    assert check(_cfg(kivi, head_dim=64)) == 2
    assert check(_cfg(kivi, group_k=16)) == 1
    assert check(_cfg(kivi, group_v=256)) == 1
    for name in ("num_pages", "num_seqs", "max_blocks", "num_kv_heads"):
        assert check(_cfg(kivi, **{name: 0})) == 1
    assert check(_cfg(kivi, num_seqs=8192)) == 0
    assert check(_cfg(kivi, num_seqs=8193)) == 2
    assert check(_cfg(kivi, max_blocks=1 << 24)) == 2      # 2^31 tokens a sequence
    assert check(_cfg(kivi, num_pages=1 << 30, num_kv_heads=2)) == 2
    assert kivi.load_library().kivi_paged_check_config(None) == 1


def test_sizes(kivi):
    cfg = _cfg(kivi, bits=4, group_k=64, group_v=128, residual=256)
    got = dict(zip(kivi.PAGED_BUFFERS, kivi.kivi_paged_sizes(cfg)))
    assert got["k_codes"] == got["v_codes"] == 40 * 2 * 256 * 128 // 2
    assert got["k_scale"] == got["k_zero"] == 40 * 2 * 2 * 2
    assert got["v_scale"] == got["v_zero"] == 40 * 2 * 2 * 2
    assert got["k_res"] == got["v_res"] == 4 * 2 * 256 * 128 * 2
    assert (got["block_table"], got["free_pages"], got["queue"]) == (4 * 8 * 4, 40 * 4, 16)
    big = kivi.kivi_paged_sizes(_cfg(kivi, num_pages=1 << 24, num_kv_heads=64))
    assert big[0] == (1 << 24) * 64 * 128 * 32             # past 32 bits
    _refused(kivi, "UNSUPPORTED", kivi.kivi_paged_sizes, _cfg(kivi, bits=8))


def test_build_tables_refusals(kivi):
    cfg, cache, plan = _cfg(kivi), _cache(kivi), _plan(kivi)

    def call(code, cfg=cfg, cache=cache, rows=4, lens=FAKE, new=FAKE, out=FAKE, queue=FAKE, plan=plan, status=None):
        _refused(kivi, code, kivi.kivi_paged_build_tables, cfg, cache, rows, lens, new, out, queue, plan, status, 0)

    call("INVALID_ARG", rows=-1)
    call("INVALID_ARG", rows=5)
    call("INVALID_ARG", lens=0)
    call("INVALID_ARG", new=FAKE + 2)
    call("INVALID_ARG", out=0)
    call("INVALID_ARG", queue=FAKE + 4)
    call("INVALID_ARG", status=FAKE + 1)
    for name in ("block_table", "free_pages", "queue"):
        call("INVALID_ARG", cache=_cache(kivi, **{name: 0}))
    for name in ("cu_tokens", "positions", "runs", "counts"):
        call("INVALID_ARG", plan=_plan(kivi, **{name: FAKE + 4}))
    call("INVALID_ARG", plan=_plan(kivi, max_tokens=0))
    call("INVALID_ARG", plan=_plan(kivi, max_runs=9))      # 2 * 4 + 256 / 128 = 10
    call("UNSUPPORTED", cfg=_cfg(kivi, bits=3))


def test_append_refusals(kivi):
    cfg, cache, plan = _cfg(kivi), _cache(kivi), _plan(kivi)

    def call(code, cfg=cfg, cache=cache, plan=plan, k=FAKE, v=FAKE, st=256, sh=128, status=None):
        _refused(kivi, code, kivi.kivi_paged_append, cfg, cache, plan, k, v, st, sh, status, 0)

    call("INVALID_ARG", k=0)
    call("INVALID_ARG", v=FAKE + 8)
    call("INVALID_ARG", st=252)
    call("INVALID_ARG", sh=4)
    call("INVALID_ARG", status=FAKE + 2)
    call("INVALID_ARG", plan=_plan(kivi, runs=0))
    call("INVALID_ARG", plan=_plan(kivi, max_runs=0))
    for name in ("k_codes", "v_codes", "k_scale", "k_zero", "v_scale", "v_zero", "k_res", "v_res"):
        call("INVALID_ARG", cache=_cache(kivi, **{name: FAKE + 8}))


def test_attention_refusals(kivi):
    cfg, cache = _cfg(kivi), _cache(kivi)
    ws = kivi.kivi_paged_workspace_bytes(cfg, 8)
    assert ws > 0 and ws % 256 == 0
    assert kivi.kivi_paged_workspace_bytes(cfg, 3) == 0
    assert kivi.kivi_paged_workspace_bytes(cfg, 0) == 0
    assert kivi.kivi_paged_workspace_bytes(cfg, 130) == 0     # 65 query heads per KV head

    def call(code, cfg=cfg, cache=cache, rows=4, lens=FAKE, cu=None, q=FAKE, q_rows=4, hq=8, scale=0.1, window=0, sinks=0,
             out=FAKE, ws_ptr=FAKE, ws_bytes=ws, status=None):
        _refused(kivi, code, kivi.kivi_paged_decode_attention, cfg, cache, rows, lens, cu, q, q_rows, hq, scale, window,
                 sinks, out, ws_ptr, ws_bytes, status, 0)

    call("INVALID_ARG", rows=5)
    call("INVALID_ARG", rows=-1)
    call("INVALID_ARG", q_rows=3)
    call("INVALID_ARG", hq=3)
    call("UNSUPPORTED", hq=130)
    call("INVALID_ARG", lens=0)
    call("INVALID_ARG", cu=FAKE + 2)
    call("INVALID_ARG", q=FAKE + 8)
    call("INVALID_ARG", out=FAKE + 2)
    call("INVALID_ARG", scale=float("nan"))
    call("INVALID_ARG", scale=float("inf"))
    call("INVALID_ARG", window=-1)
    call("INVALID_ARG", sinks=-1)
    call("INVALID_ARG", status=FAKE + 1)
    call("INVALID_ARG", cache=_cache(kivi, block_table=0))
    call("INVALID_ARG", cache=_cache(kivi, k_codes=0))
    call("WORKSPACE", ws_ptr=0)
    call("WORKSPACE", ws_ptr=FAKE + 128)
    call("WORKSPACE", ws_bytes=ws - 1)


def test_append_of_no_tokens_refusals(kivi):
    """Without tokens the sources are not used; the rest of the rules hold."""
    cfg, cache = _cfg(kivi), _cache(kivi)
    for kw, st in ((dict(max_tokens=-1), 256), (dict(max_tokens=0), 252), (dict(max_tokens=0, counts=0), 256)):
        _refused(kivi, "INVALID_ARG", kivi.kivi_paged_append, cfg, cache, _plan(kivi, **kw), 0, 0, st, 128, None, 0)
    _refused(kivi, "INVALID_ARG", kivi.kivi_paged_append, cfg, cache, _plan(kivi, max_tokens=1), 0, FAKE, 256, 128, None, 0)


def test_plan_attention_refusals(kivi):
    cfg, cache = _cfg(kivi), _cache(kivi)
    ws = kivi.kivi_paged_workspace_bytes(cfg, 8)

    def call(code, cfg=cfg, cache=cache, rows=4, lens=FAKE, q=FAKE, q_rows=4, hq=8, scale=0.1, window=0, sinks=0, out=FAKE,
             ws_ptr=FAKE, ws_bytes=ws, status=None, **plan):
        _refused(kivi, code, kivi.kivi_paged_plan_attention, cfg, cache, _plan(kivi, **plan), rows, lens, q, q_rows, hq, scale,
                 window, sinks, out, ws_ptr, ws_bytes, status, 0)

    call("INVALID_ARG", cu_tokens=0)
    call("INVALID_ARG", positions=0)
    call("INVALID_ARG", positions=FAKE + 4)
    call("INVALID_ARG", max_tokens=0)
    call("INVALID_ARG", rows=5)
    call("INVALID_ARG", lens=0)
    call("INVALID_ARG", q_rows=-1)
    call("INVALID_ARG", q=FAKE + 8)
    call("INVALID_ARG", hq=3)
    call("INVALID_ARG", scale=float("nan"))
    call("INVALID_ARG", window=-1)
    call("INVALID_ARG", status=FAKE + 1)
    call("WORKSPACE", ws_bytes=ws - 1)


def test_window_refusals(kivi):
    cfg = kivi.kivi_config(2, 3, 128, 2, 32, 32, 128, 1024, 0, 0)
    ws = kivi.kivi_window_workspace_bytes(cfg, 6)
    assert ws > 0
    assert kivi.kivi_window_workspace_bytes(cfg, 7) == 0

    def call(code, cfg=cfg, n_quant=256, n_res=5, q=FAKE, hq=6, scale=0.1, window=64, sinks=4, out=FAKE, ws_ptr=FAKE,
             ws_bytes=ws, k_res=FAKE):
        cache = kivi.kivi_cache(*([FAKE] * 8), n_quant, n_res)
        cache.k_res = k_res
        _refused(kivi, code, kivi.kivi_decode_attention_window, cfg, cache, q, hq, scale, window, sinks, out, ws_ptr,
                 ws_bytes, None, 0)

    call("STATE", n_quant=100)
    call("STATE", n_res=129)
    call("STATE", n_quant=1152)
    call("EMPTY", n_quant=0, n_res=0)
    call("INVALID_ARG", hq=7)
    call("INVALID_ARG", window=-1)
    call("INVALID_ARG", sinks=-5)
    call("INVALID_ARG", scale=float("inf"))
    call("INVALID_ARG", q=0)
    call("INVALID_ARG", k_res=0)
    call("WORKSPACE", ws_ptr=FAKE + 16)
    call("WORKSPACE", ws_bytes=ws - 1)
    call("UNSUPPORTED", cfg=kivi.kivi_config(2, 3, 128, 2, 32, 32, 128, 1024, 1, 0))
    call("UNSUPPORTED", cfg=kivi.kivi_config(2, 3, 128, 2, 32, 32, 128, 1024, 0, 1))


def test_rotary_refusals(kivi):
    init = kivi.kivi_rotary_init
    good = dict(rotary_dim=64, interleaved=0, theta=10000.0, scaling=0, factor=1.0, low=1.0, high=4.0, original_positions=8192)

    def bad(**kw):
        _refused(kivi, "INVALID_ARG", init, *{**good, **kw}.values())

    bad(rotary_dim=72)
    bad(rotary_dim=144)
    bad(rotary_dim=-16)
    bad(interleaved=2)
    bad(theta=1.0)
    bad(theta=float("nan"))
    bad(scaling=5)
    bad(scaling=1, factor=0.5)
    bad(scaling=3, factor=8.0, low=4.0, high=4.0)
    bad(scaling=3, factor=8.0, low=0.0)
    bad(scaling=4, factor=8.0, original_positions=0)
    rot = init(*good.values())
    heads = kivi.kivi_heads(FAKE, FAKE, None, 4, 0, 0, 512, 128, 0, 512, 128)

    def apply(code, dtype=0, batch=1, tokens=5, positions=None, position0=0, eps=1e-6, v=None, **kw):
        h = kivi.kivi_heads(FAKE, FAKE, None, 4, 0, 0, 512, 128, 0, 512, 128)
        for name, value in kw.items():
            setattr(h, name, value)
        _refused(kivi, code, kivi.kivi_rotary_apply, rot, dtype, batch, tokens, positions, position0, h, heads, v, eps, 0)

    apply("UNSUPPORTED", dtype=2)
    apply("INVALID_ARG", tokens=-1)
    apply("INVALID_ARG", batch=-1)
    apply("INVALID_ARG", eps=-1.0)
    apply("INVALID_ARG", eps=float("nan"))
    apply("INVALID_ARG", positions=FAKE + 2)
    apply("INVALID_ARG", position0=0x7fffffff - 4)
    apply("INVALID_ARG", x_dev=FAKE + 8)
    apply("INVALID_ARG", y_dev=0)
    apply("INVALID_ARG", weight_dev=FAKE + 2)
    apply("INVALID_ARG", x_token=516)
    apply("INVALID_ARG", y_head=4)
    apply("INVALID_ARG", num_heads=-1)
    apply("INVALID_ARG", v=kivi.kivi_heads(FAKE, FAKE, FAKE, 4, 0, 0, 512, 128, 0, 512, 128))  # values have no norm
    apply("UNSUPPORTED", batch=1 << 16, tokens=1 << 16, position0=-1)


@pytest.mark.parametrize("scaling", ["none", "linear", "base", "bands", "ramp"])
@pytest.mark.parametrize("rd", [0, 16, 64, 112, 128])
def test_rotary_frequencies(kivi, scaling, rd):
    """turns[i] is the frequency in turns as a 64-bit fraction; double arithmetic leaves a few parts in 2^52."""
    for theta, factor, original in ((10000.0, 8.0, 8192), (500000.0, 32.0, 131072), (1.5, 1.0, 64)):
        for low, high in ((1.0, 4.0), (1.0, 32.0)):
            r = kivi.kivi_rotary_init(rd, 1, theta, kivi.ROPE_SCALINGS[scaling], factor, low, high, original)
            f, m = ref.frequencies(rd, theta, scaling, factor, low, high, original)
            assert (r.rotary_dim, r.interleaved) == (rd, 1)
            assert abs(r.magnitude - m) <= 2.0 ** -23 * m
            for i, x in enumerate(f):
                want = x / (2 * math.pi)
                assert abs(r.turns[i] / 2.0 ** 64 - want) <= 2.0 ** -48 * want + 2.0 ** -63
            assert all(t == 0 for t in r.turns[rd // 2:])


def test_torch_layer_int32(kivi):
    """Python integers that an int32 argument would cut off are refused."""
    for x in (1 << 31, -(1 << 31) - 1, 1 << 40):
        with pytest.raises(ValueError):
            kivi._int32("window", x)
    assert kivi._int32("window", -5) == -5
    with pytest.raises(ValueError):
        kivi.Rotary(scaling="other")


def test_torch_layer_device(kivi):
    """Device 0 by its number is device 0, not whichever one is current."""
    import torch
    assert kivi._device(torch, 0) == torch.device("cuda", 0) == kivi._device(torch, "cuda:0")
    assert kivi._device(torch, 1) == torch.device("cuda", 1) and kivi._device(torch, None) == torch.device("cuda")


def test_struct_sizes(kivi):
    """The ctypes structures have the C layout of include/kivi.h."""
    assert ctypes.sizeof(kivi.kivi_rotary) == 16 + 64 * 8
    assert ctypes.sizeof(kivi.kivi_heads) == 3 * 8 + 8 + 6 * 8
    assert ctypes.sizeof(kivi.kivi_paged_config) == 9 * 4
    assert ctypes.sizeof(kivi.kivi_paged_cache) == 11 * 8
    assert ctypes.sizeof(kivi.kivi_paged_plan) == 4 * 8 + 8
