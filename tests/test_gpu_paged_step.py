"""PagedKiviCache.step as one call: what it refuses changes nothing, and steps of one token or none."""
import pytest

from test_gpu_paged import _cache, _i32

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from bit_asymmetric_kv_02_b200 import kivi  # noqa: E402

F16, BF16 = torch.float16, torch.bfloat16


def _filled(**kw):
    """A cache of two sequences of 127 and 40 tokens, with its plan, lengths and the next step's projection output."""
    g = torch.Generator("cuda").manual_seed(1)
    cache = _cache(num_seqs=2, num_q_heads=4, **kw)
    for name in kivi.BUFFERS:  # rows that nobody writes are compared too, and NaN is not itself
        cache.buffers[name].zero_()
    plan, lens = cache.new_plan(200), _i32([0, 0])
    x = torch.randn(167, 8, 128, generator=g, device="cuda").half()
    cache.step(plan, lens, _i32([127, 40]), x[:, :4], x[:, 4:6], x[:, 6:])
    return cache, plan, lens, torch.randn(2, 8, 128, generator=g, device="cuda").half()


def _state(cache, lens):
    names = ("block_table", "free_pages", "queue", "k_res", "v_res")
    return [lens.clone()] + [cache.view(n).clone() for n in names]


@pytest.mark.parametrize("rotary", [False, True])
def test_a_refused_step_changes_nothing(rotary):
    cache, plan, lens, x = _filled()
    rot, new = kivi.Rotary() if rotary else None, _i32([1, 1])
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    before = _state(cache, lens)
    odd = torch.zeros(2 * 8 * 128 + 8, dtype=F16, device="cuda")[4:4 + 2 * 8 * 128].view(2, 8, 128)  # 8 bytes off
    wide = torch.zeros(2, 2, 130, dtype=F16, device="cuda")
    bad = [dict(q=q.float()), dict(k=k.float()), dict(v=v.float()), dict(q=q[:, :3]), dict(k=k[:, :1]), dict(v=v[:, :1]),
           dict(k=k[:1]), dict(v=v[:1]), dict(q=q[..., :64]), dict(k=wide[..., :128], v=wide[..., :128]), dict(q=q.cpu()),
           dict(k=odd[:, :2], v=odd[:, 2:4]), dict(new=new.long()), dict(new=new[:1]), dict(lens=lens.long()), dict(scale=float("nan")),
           dict(window=-1), dict(window=1 << 31), dict(sinks=-1), dict(out=torch.zeros(1, 4, 128, dtype=F16, device="cuda")),
           dict(out=torch.zeros(2, 4, 128, device="cuda")), dict(plan=_cache(num_seqs=3).new_plan(200)),
           dict(q=torch.zeros(2, 3, 128, dtype=F16, device="cuda")), dict(q=torch.zeros(2, 130, 128, dtype=F16, device="cuda")),
           dict(out=torch.zeros(2 * 4 * 128 + 8, dtype=F16, device="cuda")[4:4 + 2 * 4 * 128].view(2, 4, 128))]
    if rotary:
        w = torch.ones(128, dtype=F16, device="cuda")
        bad += [dict(q=q.bfloat16()), dict(k=k.bfloat16()), dict(q_weight=w.bfloat16()), dict(k_weight=w[:64]), dict(eps=-1.0),
                dict(eps=float("nan")), dict(q=odd[:, :4]), dict(q_weight=torch.ones(136, dtype=F16, device="cuda")[4:132])]
    else:
        bad += [dict(q=q.bfloat16(), k=k.bfloat16(), v=v.bfloat16()), dict(k=k.bfloat16(), v=v.bfloat16())]
    for kw in bad:
        args = dict(plan=plan, lens=lens, new=new, q=q, k=k, v=v)
        args.update(kw)
        more = {n: args.pop(n) for n in list(args) if n not in ("plan", "lens", "new", "q", "k", "v")}
        with pytest.raises((ValueError, kivi.KiviError)):
            cache.step(args["plan"], args["lens"], args["new"], args["q"], args["k"], args["v"], rotary=rot, **more)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(before, _state(cache, lens))), kw.keys()
    # a number of query heads without a workspace, under capture
    more_heads = torch.zeros(2, 8, 128, dtype=F16, device="cuda")
    with pytest.raises(RuntimeError):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            cache.step(plan, lens, new, more_heads, k, v, rotary=rot)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, _state(cache, lens)))
    assert cache.read_status() == 0


@pytest.mark.parametrize("rows, new", [(2, [2, 1]), (1, [1, 1]), (3, [200, 200])])
def test_more_new_tokens_than_rows(rows, new):
    """Nothing is planned, and the status word says so."""
    cache, plan, lens, x = _filled()
    x = torch.cat([x, x])[:rows]
    before = _state(cache, lens)
    out = torch.full((rows, 4, 128), 7.0, dtype=F16, device="cuda")
    cache.step(plan, lens, _i32(new), x[:, :4], x[:, 4:6], x[:, 6:], out=out)
    assert cache.read_status() == 3 and (out == 7.0).all()
    assert all(torch.equal(a, b) for a, b in zip(before, _state(cache, lens)))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads, kv", [(4, 2), (1, 1)])
def test_steps_of_one_token_and_none(dtype, heads, kv):
    """One running sequence in slices of a fused projection, and steps in which requests only finish: as the calls one by one."""
    rot = kivi.Rotary(rotary_dim=64)
    g = torch.Generator("cuda").manual_seed(4)
    a, b = (_cache(num_seqs=2, num_kv_heads=kv, num_q_heads=heads) for _ in range(2))
    lens_a, lens_b, plan_a, plan_b = _i32([0, 0]), _i32([0, 0]), a.new_plan(130), b.new_plan(130)
    for new in ([126, 0], [1, 0], [1, 0], [1, 0], [0, 1], [0, 0], [-1, 0], [0, 1], [-1, -1], [1, 0]):
        rows = sum(max(n, 0) for n in new)
        x = torch.randn(rows, heads + 2 * kv, 128, generator=g, device="cuda").to(dtype)
        q, k, v = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
        out = torch.zeros(rows, heads, 128, dtype=F16, device="cuda")
        got = a.step(plan_a, lens_a, _i32(new), q, k, v, rotary=rot, out=out)
        assert got.shape == (rows, heads, 128)
        b.build_tables(plan_b, lens_b, _i32(new))
        want = torch.zeros_like(out)
        if rows > 0:
            q2, k2, v2 = rot.apply(q, k, v, positions=plan_b.positions[:rows])
            b.append(plan_b, k2.contiguous(), v2.contiguous())
            b.attend(lens_b, q2, plan=plan_b, out=want)
        assert torch.equal(out, want) and torch.equal(lens_a, lens_b), new
    for name in kivi.PAGED_BUFFERS[-3:]:
        assert torch.equal(a.view(name), b.view(name))
    assert a.read_status() == b.read_status() == 0
    # append alone: the strides of a dimension of one entry mean nothing
    x = torch.randn(1, heads + 2 * kv, 128, generator=g, device="cuda").half()
    for cache, lens, plan, k in ((a, lens_a, plan_a, x[:, :kv]), (b, lens_b, plan_b, x[:, :kv].clone())):
        cache.build_tables(plan, lens, _i32([0, 1]))
        cache.append(plan, k, x[:, kv:2 * kv])
    assert torch.equal(a.view("k_res")[1, :, 0], b.view("k_res")[1, :, 0])
    assert a.read_status() == b.read_status() == 0
    a.append(plan_a, x[:0, :kv], x[:0, kv:2 * kv].contiguous())


def test_no_rows_for_a_plan_of_tokens():
    """append() and step() of no rows behind tables that count some: reported, and nothing is read."""
    cache, plan, lens, x = _filled()
    none = x[:0, :2]
    cache.build_tables(plan, lens, _i32([0, 0]))
    cache.append(plan, none, none)
    assert cache.read_status() == 0
    residual = cache.view("k_res").clone()
    cache.build_tables(plan, lens, _i32([1, 1]))
    cache.append(plan, none, none)
    assert cache.read_status() == 11 and torch.equal(cache.view("k_res"), residual)
    cache.status.zero_()
    cache.step(plan, lens, _i32([0, -1]), x[:0, :4], none, none)
    assert cache.read_status() == 0 and lens.tolist() == [128, 0]
    cache.step(plan, lens, _i32([0, 1]), x[:0, :4], none, none)
    assert cache.read_status() == 11


@pytest.mark.parametrize("kind", ["no page", "too long", "not served at all"])
def test_sequences_that_could_not_be_served(kind):
    """Their rows of the output are left as they are: the cache does not hold their new tokens."""
    cache, plan, lens, x = _filled(max_blocks=2)
    new, status, served = _i32([1, 1]), 3, [False, True]
    if kind == "no page":
        cache.view("queue").copy_(torch.tensor([64, 64]))  # sequence 0 fills its block
    elif kind == "too long":
        new = _i32([1, 400])
        x = torch.randn(401, 8, 128, generator=torch.Generator("cuda").manual_seed(2), device="cuda").half()
        plan, served = cache.new_plan(401), [True, False]
    else:
        lens[0] = -5
    rows = [0, len(x) - 1]
    before = lens.tolist()
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    for call in ("step", "attend"):
        out = torch.full((len(x), 4, 128), 7.0, dtype=F16, device="cuda")
        if call == "step":
            cache.step(plan, lens, new, q, k, v, out=out)
            want = cache.attend(lens.clamp(min=0), q[rows].contiguous())
        else:
            cache.attend(lens, q.contiguous(), plan=plan, out=out)
        assert cache.read_status() == status
        for i in (0, 1):
            assert torch.equal(out[rows[i]], want[i] if served[i] else torch.full_like(want[i], 7.0)), (call, i)
            assert lens[i].item() == before[i] + (new[i].item() if served[i] else 0)
        assert (out[1:-1] == 7.0).all()
