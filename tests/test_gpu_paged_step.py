"""PagedKiviCache.step as one call: steps of one token or none."""
import pytest

from test_gpu_paged import _cache, _i32

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from bit_asymmetric_kv_02_b200 import kivi  # noqa: E402

F16, BF16 = torch.float16, torch.bfloat16


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
