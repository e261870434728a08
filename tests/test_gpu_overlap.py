"""Kernels that are launched over the end of the ones before them see what those wrote: steps whose plans differ, with nothing
between the calls, against the same calls with the GPU waited for between them."""
import pytest

from test_gpu_paged import _cache, _i32

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from bit_asymmetric_kv_02_b200 import kivi  # noqa: E402

F16 = torch.float16


def _apart(cache, plan, lens, new, x, heads, kv, rot, w, out):
    """A step, waiting after every call; every call's status."""
    rows = len(x)
    q, k, v = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
    cache.build_tables(plan, lens, new)
    torch.cuda.synchronize()
    q, k, v = rot.apply(q, k, v, positions=plan.positions[:rows], q_weight=w[0], k_weight=w[1])
    torch.cuda.synchronize()
    cache.append(plan, k, v)
    torch.cuda.synchronize()
    cache.attend(lens, q, plan=plan, out=out)
    torch.cuda.synchronize()


def _same(a, b):
    return all(torch.equal(a.view(n), b.view(n)) for n in kivi.PAGED_BUFFERS)


@pytest.mark.parametrize("captured", [True, False])
@pytest.mark.parametrize("n, heads, kv, bits", [(3, 8, 2, 2), (40, 4, 4, 2), (40, 8, 2, 4)])
def test_steps_without_a_gap(n, heads, kv, bits, captured):
    """bf16 steps (the rotation converts the values too, so that tables, rotation, append and attention follow one another),
    single tokens and more of them in turn."""
    g = torch.Generator("cuda").manual_seed(n)
    a, b = (_cache(num_pages=20 * n, num_seqs=n, max_blocks=20, num_kv_heads=kv, bits=bits, num_q_heads=heads) for _ in range(2))
    for cache in (a, b):
        for name in kivi.BUFFERS:
            cache.buffers[name].zero_()
    lens_a, lens_b = _i32([0] * n), _i32([0] * n)
    plan_a, plan_b = a.new_plan(60 * n), b.new_plan(60 * n)
    rot = kivi.Rotary(theta=500000.0)
    w = (1 + 0.1 * torch.randn(2, 128, generator=g, device="cuda")).bfloat16()
    counts = [[1] * n, [20 + i % 7 for i in range(n)], [i % 2 for i in range(n)], [3] * n]
    kinds = []
    for c in counts:
        rows = sum(c)
        x = torch.zeros(rows, heads + 2 * kv, 128, dtype=torch.bfloat16, device="cuda")
        kinds.append((_i32(c), x, torch.zeros(rows, heads, 128, dtype=F16, device="cuda"), torch.zeros(rows, heads, 128, dtype=F16, device="cuda")))

    def step(new, x, out):
        a.step(plan_a, lens_a, new, x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:], rotary=rot, q_weight=w[0], k_weight=w[1], out=out)

    torch.cuda.synchronize()
    graphs = []
    if captured:
        for new, x, out, _ in kinds:
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                step(new, x, out)
    for i in range(48):
        j = (i * i + i // 3) % len(kinds)
        new, x, out, want = kinds[j]
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        if captured:
            graphs[j].replay()
        else:
            step(new, x, out)
        _apart(b, plan_b, lens_b, new, x, heads, kv, rot, w, want)
        assert a.read_status() == b.read_status() == 0, (i, j)
        assert torch.equal(out, want) and torch.equal(lens_a, lens_b), (i, j)
    assert _same(a, b)


def test_steps_back_to_back():
    """Whole graphs one after the other without a wait, each step's plan, rotation and append over the ones before."""
    n, heads, kv = 24, 8, 4
    g = torch.Generator("cuda").manual_seed(2)
    rot = kivi.Rotary()
    w = torch.ones(2, 128, dtype=torch.bfloat16, device="cuda")
    a, b = (_cache(num_pages=12 * n, num_seqs=n, max_blocks=12, num_kv_heads=kv, num_q_heads=heads) for _ in range(2))
    for cache in (a, b):
        for name in kivi.BUFFERS:
            cache.buffers[name].zero_()
    lens_a, lens_b, plan_a, plan_b = _i32([0] * n), _i32([0] * n), a.new_plan(16 * n), b.new_plan(16 * n)
    kinds = []
    for c in ([1] * n, [5 + i % 11 for i in range(n)]):
        x = torch.randn(sum(c), heads + 2 * kv, 128, generator=g, device="cuda").bfloat16()
        kinds.append((_i32(c), x, torch.zeros(sum(c), heads, 128, dtype=F16, device="cuda")))
    torch.cuda.synchronize()
    graphs = []
    for new, x, out in kinds:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            a.step(plan_a, lens_a, new, x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:], rotary=rot, q_weight=w[0], k_weight=w[1], out=out)
    order = [0, 1, 0, 0, 1, 1, 0, 1] * 4
    for j in order:
        graphs[j].replay()
    torch.cuda.synchronize()
    got = [out.clone() for _, _, out in kinds]
    wants = [torch.zeros_like(out) for _, _, out in kinds]
    for j in order:
        new, x, _ = kinds[j]
        _apart(b, plan_b, lens_b, new, x, heads, kv, rot, w, wants[j])
    assert a.read_status() == b.read_status() == 0 and torch.equal(lens_a, lens_b)
    assert _same(a, b) and all(torch.equal(x, y) for x, y in zip(got, wants))
