"""Paged cache on the GPU: tables, append and attention, each against a plain implementation (paged_ref, the oracle), and
the steps of a batch of sequences that come and go."""
import random

import numpy as np
import pytest

import paged_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from bit_asymmetric_kv_02_b200 import kivi  # noqa: E402
import oracle.kivi_oracle as O  # noqa: E402

NAN = float("nan")


def _cache(**kw):
    base = dict(num_pages=64, num_seqs=4, max_blocks=16, num_kv_heads=2, bits=2, group_k=32, group_v=32, residual=128)
    base.update(kw)
    return kivi.PagedKiviCache(**base)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---- tables ---------------------------------------------------------------------------------------
def _check_tables(cache, lens, new, max_tokens, table, ring, queue, in_place=False, want_status=0):
    """One call on the given state against the plain implementation; returns what it left."""
    R = cache.cfg.residual
    cache.view("block_table").copy_(torch.from_numpy(table))
    cache.view("free_pages").copy_(torch.from_numpy(ring))
    cache.view("queue").copy_(torch.tensor(queue))
    plan = cache.new_plan(max_tokens)
    for x in (plan.cu_tokens, plan.positions, plan.runs, plan.counts):
        x.fill_(-77)
    n = len(lens)
    lens_d, out_d = _i32(lens), torch.full((n,), -77, dtype=torch.int32, device="cuda")
    queue_d = torch.full((2,), -77, dtype=torch.int64, device="cuda")
    cache.status.zero_()
    if in_place:
        cache.build_tables(plan, lens_d, _i32(new))
        out_d, queue_d = lens_d, cache.view("queue")
    else:
        cache.build_tables(plan, lens_d, _i32(new), lens_out=out_d, queue_out=queue_d)
        assert lens_d.tolist() == list(lens) and cache.view("queue").tolist() == list(queue)
    table, ring = table.copy(), ring.copy()
    out, queue, cu, positions, runs, failed = ref.build_tables(table, ring, queue, lens, new, R, max_tokens)
    assert cache.read_status() == (3 if failed else 0) == want_status
    assert out_d.tolist() == out and queue_d.tolist() == list(queue)
    assert plan.cu_tokens.tolist() == cu + [-77] * (cache.cfg.num_seqs - n)
    assert plan.positions.tolist() == positions + [-77] * (max_tokens - len(positions))
    assert plan.counts.tolist() == [len(runs), cu[-1]]
    got = plan.runs.cpu().numpy()
    assert np.array_equal(got[:len(runs)], np.array(runs, np.int32).reshape(-1, 8)) and (got[len(runs):] == -77).all()
    assert np.array_equal(cache.view("block_table").cpu().numpy(), table)
    assert np.array_equal(cache.view("free_pages").cpu().numpy(), ring)
    return out, queue, table, ring


def _state(cache, lens, rng, head=0):
    """Tables of sequences that hold those tokens, and the queue of the other pages from `head` on."""
    cfg = cache.cfg
    ids = np.array(rng.sample(range(cfg.num_pages), cfg.num_pages), np.int32)
    table = np.full((cfg.num_seqs, cfg.max_blocks), -1, np.int32)
    used = 0
    for i, length in enumerate(lens):
        k = max(0, length) // cfg.residual
        table[i, :k] = ids[used:used + k]
        used += k
    free = ids[used:]
    ring = np.full(cfg.num_pages, -5, np.int32)
    for j, p in enumerate(free):
        ring[(head + j) % cfg.num_pages] = p
    return table, ring, (head, head + len(free))


@pytest.mark.parametrize("n, num_seqs, R", [(1, 1, 128), (7, 9, 256), (64, 64, 128), (333, 400, 512), (2500, 2500, 128)])
def test_tables(n, num_seqs, R):
    rng = random.Random(n)
    cache = _cache(num_pages=max(64, 8 * n), num_seqs=num_seqs, max_blocks=12, residual=R, num_kv_heads=1)
    for trial in range(4):
        top = 6 * R if n < 1000 else 3 * R
        lens = [rng.choice([0, 1, R - 1, R, R + 1, rng.randrange(top)]) for _ in range(n)]
        new = [rng.choice([-1, -9, 0, 1, 1, 1, R - 1, R, R + 1, rng.randrange(2 * R)]) for _ in range(n)]
        table, ring, queue = _state(cache, lens, rng, head=rng.randrange(3 * cache.cfg.num_pages))
        tokens = sum(max(a, 0) for a in new)
        fits = sum(max(0, (a + b) // R - a // R) for a, b in zip(lens, new) if b > 0) <= queue[1] - queue[0]
        _check_tables(cache, lens, new, tokens + trial, table, ring, queue, in_place=trial % 2 == 1,
                      want_status=0 if fits else 3)


def test_tables_no_rows():
    cache = _cache()
    plan = cache.new_plan(8)
    empty = torch.zeros(0, dtype=torch.int32, device="cuda")
    cache.build_tables(plan, empty, empty)
    assert plan.counts.tolist() == [0, 0] and plan.cu_tokens[0].item() == 0
    assert cache.view("queue").tolist() == [0, 64] and cache.read_status() == 0


@pytest.mark.parametrize("lens, new, max_tokens, free", [
    ([5, 2047, 3, 100], [1, 130, 1, 28], 300, 9),              # row 1 needs more than max_blocks
    ([5, -1, 3, 100], [1, 2, 1, 28], 300, 9),                  # a negative length
    ([5, 2**30, 3, 100], [1, 5, 1, 28], 300, 9),               # a length the table cannot hold
    ([5, 2**31 - 1, 3, 100], [1, 5, 1, 28], 300, 9),
    ([127, 127, 127, 0], [1, 1, 1, 1], 300, 2),                # the third row finds no page
    ([127, 100, 127, 0], [1, 300, 1, 1], 303, 2),              # the second asks for three: later takers fail with it
    ([127, 127, 5, 0], [1, 1, 1, 300], 200, 9),                # more tokens than the plan holds
    ([640, 127, 300, 0], [-1, 1, -1, 1], 300, 0),              # pages that come back are handed out later
])
def test_tables_that_cannot_serve_a_row(lens, new, max_tokens, free):
    rng = random.Random(3)
    cache = _cache(max_blocks=16)
    table, ring, queue = _state(cache, [min(max(x, 0), 2047) for x in lens], rng, head=60)
    queue = (queue[0], min(queue[1], queue[0] + free))
    for in_place in (False, True):
        _check_tables(cache, lens, new, max_tokens, table, ring, queue, in_place=in_place, want_status=3)


# ---- append ---------------------------------------------------------------------------------------
def _oracle_block(k, v, cfg):
    """Code words and scales of one head's R-token block by the oracle."""
    kc, ks, kz = O.quantize_k_block(k, cfg.group_k, cfg.bits)
    vc, vs, vz = O.quantize_v_block(v, cfg.group_v, cfg.bits)
    return {"k_codes": O.pack_k(kc, cfg.bits), "v_codes": O.pack_v(vc, cfg.bits), "k_scale": ks, "k_zero": kz, "v_scale": vs,
            "v_zero": vz}


def _bits(x):
    return np.ascontiguousarray(x).view(np.uint8)


def _check_cache(cache, lens, kv):
    """Every sequence's pages and residual rows against the oracle's of its tokens kv[i] = (k, v) [T][H][128]."""
    R, H = cache.cfg.residual, cache.cfg.num_kv_heads
    host = {name: cache.view(name).cpu().numpy() for name in kivi.PAGED_BUFFERS}
    for i, T in enumerate(lens):
        k, v = kv[i]
        for j in range(T // R):
            page = host["block_table"][i, j]
            for h in range(H):
                want = _oracle_block(k[j * R:(j + 1) * R, h], v[j * R:(j + 1) * R, h], cache.cfg)
                for name, w in want.items():
                    assert np.array_equal(_bits(host[name][page, h]), _bits(w)), (i, j, h, name)
        nq = max(T - 1, 0) // R * R
        for name, x in (("k_res", k), ("v_res", v)):
            assert np.array_equal(_bits(host[name][i, :, :T - nq]), _bits(x[nq:T].transpose(1, 0, 2))), (i, name)


@pytest.mark.parametrize("bits, R, gk, gv, H", [(2, 128, 32, 32, 2), (4, 128, 128, 64, 1), (2, 256, 64, 256, 3), (4, 512, 32, 128, 1),
                                                (2, 512, 128, 32, 1)])
def test_append(bits, R, gk, gv, H):
    """Steps of mixed prompts and single tokens, slices of one projection's output as sources."""
    rng = np.random.default_rng(bits * R + gk)
    n = 5
    cache = _cache(num_pages=40, num_seqs=n + 1, max_blocks=12, num_kv_heads=H, bits=bits, group_k=gk, group_v=gv, residual=R)
    for name in kivi.BUFFERS:
        cache.buffers[name].fill_(0xAB)
    lens = torch.zeros(n, dtype=torch.int32, device="cuda")
    kv = [(np.zeros((0, H, 128), np.float16),) * 2 for _ in range(n)]
    plan = cache.new_plan(5 * R)
    steps = [[R + 3, 1, 0, R, 2 * R - 1], [1, R - 1, 1, 1, 1], [R - 4, 1, R, 0, 2], [2 * R, R + 1, 1, R - 1, 0], [1, 1, 1, 1, 1]]
    for new in steps:
        tokens = sum(new)
        qkv = (rng.standard_normal((tokens + 2, 3 * H, 128)) * np.where(rng.random(128) < 0.05, 10, 1)).astype(np.float16)
        dev = torch.from_numpy(qkv).cuda()
        k, v = dev[:, H:2 * H], dev[:, 2 * H:]
        cache.build_tables(plan, lens, _i32(new))
        cache.append(plan, k, v)
        at = 0
        for i, a in enumerate(new):
            kv[i] = tuple(np.concatenate([old, qkv[at:at + a, lo:lo + H]]) for old, lo in zip(kv[i], (H, 2 * H)))
            at += a
        _check_cache(cache, lens.tolist(), kv)
    assert cache.read_status() == 0
    assert (cache.view("k_res")[n].view(torch.int16) == -21589).all()  # 0xABAB: the sequence that took no part
    assert sorted(set(cache.view("block_table").cpu().numpy().ravel()) - {-1}) == sorted(
        cache.view("free_pages").cpu().numpy()[:cache.view("queue")[0].item()])


@pytest.mark.parametrize("bits, R, H, n", [(2, 128, 8, 70), (4, 256, 5, 60), (2, 512, 17, 40), (4, 128, 3, 120)])
def test_append_many_short_runs(bits, R, H, n):
    """Steps of few tokens for many sequences, some of which fill a block, some with more rows than others; then a bad run
    among good ones, and a count of more runs than there are."""
    rng = np.random.default_rng(bits * R + n)
    cache = _cache(num_pages=2 * n + 8, num_seqs=n, max_blocks=4, num_kv_heads=H, bits=bits, residual=R)
    lens = torch.zeros(n, dtype=torch.int32, device="cuda")
    kv = [(np.zeros((0, H, 128), np.float16),) * 2 for _ in range(n)]
    first = [int(x) for x in rng.integers(0, 3, n) * R // 2 + rng.integers(-3, 1, n)]
    steps = [[max(0, x) for x in first], [1] * n, [int(x) for x in rng.integers(0, 3, n)],
             [int(x) for x in np.where(rng.random(n) < 0.1, rng.integers(8, 30, n), 1)]]
    plans = [cache.new_plan(max(1, sum(steps[0]))), cache.new_plan(4 * n)]
    for j, new in enumerate(steps):
        plan = plans[min(j, 1)]
        kv_new = rng.standard_normal((max(1, sum(new)), 2, H, 128)).astype(np.float16)
        dev = torch.from_numpy(kv_new).cuda()
        cache.build_tables(plan, lens, _i32(new))
        cache.append(plan, dev[:, 0], dev[:, 1])
        at = 0
        for i, a in enumerate(new):
            kv[i] = tuple(np.concatenate([kv[i][e], kv_new[at:at + a, e]]) for e in (0, 1))
            at += a
    _check_cache(cache, lens.tolist(), kv)
    assert cache.read_status() == 0
    plan, x = plans[1], torch.randn(4 * n, H, 128, device="cuda").half()
    runs = [[i, -1, i, 0, 1, 1, 0, 0] for i in range(n)]  # a row each
    runs[n // 2][0] = n
    plan.runs[:n] = _i32(runs)
    for count, want in ((n, 11), (n - 1, 11), (n // 2, 0), (1 << 30, 11)):
        cache.status.zero_()
        cache.view("k_res").zero_()
        plan.runs[n:] = 0  # behind the runs: nothing that could be done
        plan.counts.copy_(_i32([count, n]))
        cache.append(plan, x, x)
        assert cache.read_status() == want, count
        done = cache.view("k_res")[:, :, 0]
        for i in range(n):
            on = i < count and i != n // 2
            assert torch.equal(done[i], x[i] if on else torch.zeros_like(x[i])), (count, i)


def test_append_skips_runs_outside_the_cache():
    """Runs that name sequences, pages or rows outside are left out and reported; the others are done."""
    cache = _cache(num_pages=8, num_seqs=2, max_blocks=4, num_kv_heads=1)
    plan = cache.new_plan(256)
    k = torch.randn(256, 1, 128, device="cuda").half()
    good = [0, 3, 0, 0, 128, 1, 0, 0]
    for bad in ([2, 3, 0, 0, 128, 1, 0, 0], [-1, 3, 0, 0, 128, 1, 0, 0], [0, 8, 0, 0, 128, 1, 0, 0], [0, -2, 0, 0, 128, 1, 0, 0],
                [0, 3, 129, 0, 128, 1, 0, 0], [0, 3, -1, 0, 128, 1, 0, 0], [0, 3, 0, -1, 127, 1, 0, 0], [0, 3, 0, 8, 8, 1, 0, 0],
                [0, 3, 0, 1, 129, 1, 0, 0], [1, 4, 128, 0, 128, 0, 5, 0], [1, 4, 128, 0, 128, 0, -1, 0]):
        for name in kivi.BUFFERS:
            cache.buffers[name].zero_()
        cache.status.zero_()
        plan.runs[:2] = _i32([bad, good])
        plan.counts.copy_(_i32([2, 256]))
        cache.append(plan, k, k)
        assert cache.read_status() == 11, bad
        want = _oracle_block(k[:128, 0].cpu().numpy(), k[:128, 0].cpu().numpy(), cache.cfg)
        assert np.array_equal(_bits(cache.view("k_codes")[3, 0].cpu().numpy()), _bits(want["k_codes"])), bad
        assert torch.equal(cache.view("v_res")[0, 0], k[:128, 0])
        assert not cache.view("k_codes")[5:].any() and not cache.view("k_codes")[:3].any()


def test_append_reads_no_row_past_its_source():
    """A plan of more tokens than k and v have rows: the runs past them are refused."""
    cache = _cache(num_kv_heads=1)
    plan = cache.new_plan(300)
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    cache.build_tables(plan, lens, _i32([100, 100]))
    k = torch.randn(150, 1, 128, device="cuda").half()
    cache.append(plan, k, k)
    assert cache.read_status() == 11
    assert torch.equal(cache.view("k_res")[0, 0, :100], k[:100, 0])


# ---- attention ------------------------------------------------------------------------------------
def _fill(cache, g, outliers=False):
    """Random codes, scales and residual rows everywhere."""
    R, bits = cache.cfg.residual, cache.cfg.bits
    for name in ("k_codes", "v_codes"):
        x = cache.view(name)
        x.copy_(torch.randint(-2 ** 31, 2 ** 31, x.shape, generator=g, device="cuda", dtype=torch.int64).int())
    for name in ("k_scale", "v_scale", "k_zero", "v_zero"):
        x = cache.view(name)
        y = torch.rand(x.shape, generator=g, device="cuda") + 0.2
        y = y * 3 / (2 ** bits - 1) if "scale" in name else -y * 1.5
        if outliers:
            y = y * torch.where(torch.rand(x.shape, generator=g, device="cuda") < 0.2, 12.0, 1.0)
        x.copy_(y)
    for name in ("k_res", "v_res"):
        x = cache.view(name)
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))


def _pages(cache, lens, rng):
    table = np.full((cache.cfg.num_seqs, cache.cfg.max_blocks), -1, np.int32)
    ids = rng.sample(range(cache.cfg.num_pages), cache.cfg.num_pages)
    for i, T in enumerate(lens):
        for j in range(T // cache.cfg.residual):
            table[i, j] = ids.pop()
    cache.view("block_table").copy_(torch.from_numpy(table))
    return table


def _rows(cache, table, i, T):
    """float64 K, V rows of sequence i and the sizes of their terms: [H][T][128] each."""
    R, bits = cache.cfg.residual, cache.cfg.bits
    nb = max(T - 1, 0) // R
    at = torch.from_numpy(table[i, :nb]).long().cuda()
    parts = ref.dequantised(*(cache.view(x)[at] for x in ("k_codes", "v_codes", "k_scale", "k_zero", "v_scale", "v_zero")), bits)
    out = []
    for p, res in zip(parts, ("k_res", "v_res", "k_res", "v_res")):
        r = cache.view(res)[i, :, :T - nb * R].double()
        r = r if p is parts[0] or p is parts[1] else r.abs()
        out.append(torch.cat([p.transpose(0, 1).reshape(p.shape[1], nb * R, 128), r], 1))
    return out


def _check_attention(cache, table, lens, q, out, scale, window=0, sinks=0, rows=None):
    G = q.shape[1] // cache.cfg.num_kv_heads
    for i, T in enumerate(lens):
        row = i if rows is None else rows[i]
        if row is None:
            continue
        k, v, ka, va = _rows(cache, table, i, T)
        keep = torch.from_numpy(ref.visible(T, window, sinks)).cuda()
        for h in range(cache.cfg.num_kv_heads):
            qh = q[row, h * G:(h + 1) * G].double()
            want = ref.attend(qh, k[h], v[h], scale, keep)
            got = out[row, h * G:(h + 1) * G].double()
            err = (got - want).abs()
            tol = ref.attend_bound(qh, ka[h], va[h], scale, keep, want)
            assert (err <= tol).all(), (i, T, h, err.max().item(), (err - tol).max().item(), tol.min().item())


LENS = {128: [0, 1, 16, 17, 127, 128, 129, 256, 257, 300, 511, 1000, 1537, 2000], 256: [1, 255, 256, 257, 512, 700, 1300],
        512: [2, 512, 513, 1025, 1999]}


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8])
@pytest.mark.parametrize("bits, R, gk, gv", [(2, 128, 32, 32), (4, 128, 128, 128), (2, 256, 64, 128), (4, 512, 32, 64), (2, 512, 128, 512)])
def test_attention(bits, R, gk, gv, G):
    g = torch.Generator("cuda").manual_seed(G)
    lens = LENS[R]
    H = 3
    cache = _cache(num_pages=80, num_seqs=len(lens) + 1, max_blocks=16, num_kv_heads=H, bits=bits, group_k=gk, group_v=gv, residual=R)
    _fill(cache, g)
    table = _pages(cache, lens, random.Random(R))
    q = torch.randn(len(lens), H * G, 128, generator=g, device="cuda").half()
    out = cache.attend(_i32(lens), q)
    _check_attention(cache, table, lens, q, out, 128 ** -0.5)
    assert torch.equal(out, cache.attend(_i32(lens), q))  # no order of arrival changes a bit
    assert cache.read_status() == 0


@pytest.mark.parametrize("window, sinks", [(1, 0), (1, 1), (2, 4), (100, 0), (129, 5), (500, 130), (700, 700), (5000, 3), (0, 7), (40, 5000)])
@pytest.mark.parametrize("bits, G", [(2, 1), (2, 4), (4, 6), (4, 2)])
def test_attention_window(bits, G, window, sinks):
    """What the window hides has no effect: rows behind it hold NaN, pages that it hides whole are not read."""
    g = torch.Generator("cuda").manual_seed(window)
    lens = LENS[128]
    cache = _cache(num_pages=80, num_seqs=len(lens), bits=bits)
    _fill(cache, g)
    table = _pages(cache, lens, random.Random(window))
    hidden = table.copy()
    for i, T in enumerate(lens):
        keep = ref.visible(T, window, sinks)
        nq = max(T - 1, 0) // 128 * 128
        for j in range(nq // 128):
            if not keep[j * 128:(j + 1) * 128].any():
                hidden[i, j] = -1  # a page that is read would be reported
        for t in range(T, nq + 128):
            cache.view("k_res")[i, :, t - nq] = NAN
            cache.view("v_res")[i, :, t - nq] = NAN
        for t in range(nq, T):
            if not keep[t]:
                cache.view("k_res")[i, :, t - nq] = NAN
                cache.view("v_res")[i, :, t - nq] = NAN
    q = torch.randn(len(lens), 2 * G, 128, generator=g, device="cuda").half()
    cache.view("block_table").copy_(torch.from_numpy(hidden))
    out = cache.attend(_i32(lens), q, window=window, sinks=sinks)
    _check_attention(cache, table, lens, q, out, 128 ** -0.5, window, sinks)
    assert cache.read_status() == 0


@pytest.mark.parametrize("G", [9, 16, 23, 64])
def test_attention_many_queries(G):
    g = torch.Generator("cuda").manual_seed(G)
    lens = [700, 3, 129]
    cache = _cache(num_seqs=3, num_kv_heads=1, bits=4 if G == 16 else 2)
    _fill(cache, g)
    table = _pages(cache, lens, random.Random(G))
    q = torch.randn(3, G, 128, generator=g, device="cuda").half()
    out = cache.attend(_i32(lens), q, window=600, sinks=3)
    _check_attention(cache, table, lens, q, out, 128 ** -0.5, 600, 3)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("scale, qfactor, kfactor, vfactor", [(0.0, 1, 1, 1), (-0.1, 1, 1, 1), (0.5, 3, 1, 100), (1e-4, 300, 40, 1e-3),
                                                              (0.088, 1e-6, 1, 1), (0.088, 1, 1e-4, 300), (30.0, 1, 1, 1)])
def test_attention_ranges(bits, scale, qfactor, kfactor, vfactor):
    """Large and small scales, queries, keys and values; one group's range far from the others'."""
    g = torch.Generator("cuda").manual_seed(5)
    lens = [129, 1000, 77, 1920]
    cache = _cache(num_seqs=4, bits=bits)
    _fill(cache, g, outliers=True)
    for name in ("k_scale", "k_zero", "k_res"):
        cache.view(name).mul_(kfactor)
    for name in ("v_scale", "v_zero", "v_res"):
        cache.view(name).mul_(vfactor)
    cache.view("k_scale")[:, :, 1].mul_(2.0 ** -8)
    cache.view("v_scale")[::3].mul_(2.0 ** -8)
    cache.view("v_scale")[1::5] = 0
    cache.view("k_scale")[2::7] = 0
    table = _pages(cache, lens, random.Random(1))
    q = (torch.randn(4, 8, 128, generator=g, device="cuda") * qfactor).half()
    q[:, 3] = 0  # every logit alike
    out = cache.attend(_i32(lens), q, scale=scale)
    _check_attention(cache, table, lens, q, out, scale)


def test_attention_one_sharp_key():
    """A logit far above the rest, early, late and in the residual: the running maximum moves once or at every block."""
    g = torch.Generator("cuda").manual_seed(9)
    cache = _cache(num_seqs=4, num_kv_heads=1)
    _fill(cache, g)
    lens = [1500] * 4
    table = _pages(cache, lens, random.Random(4))
    for i, j in ((0, 0), (1, 10), (2, None)):
        if j is None:
            cache.view("k_res")[i, 0, 50] = 6.0
        else:
            cache.view("k_zero")[table[i, j].item()] = 4.0
    for j in range(11):  # every block a little above the one before
        cache.view("k_zero")[table[3, j].item()] = 0.3 * j
    q = torch.rand(4, 4, 128, generator=g, device="cuda").half()
    out = cache.attend(_i32(lens), q, scale=1.0)
    _check_attention(cache, table, lens, q, out, 1.0)


def test_attention_rows_of_a_step():
    """With a step's plan the last new token of each sequence is attended and no other row is written."""
    g = torch.Generator("cuda").manual_seed(2)
    cache = _cache(num_seqs=6)
    _fill(cache, g)
    plan = cache.new_plan(64)
    lens, new = _i32([100, 5, 300, 127, 0, 640]), [3, 0, 1, 5, 0, -1]
    table, ring, queue = _state(cache, lens.tolist(), random.Random(8))
    cache.view("block_table").copy_(torch.from_numpy(table))
    cache.view("free_pages").copy_(torch.from_numpy(ring))
    cache.view("queue").copy_(torch.tensor(queue))
    cache.build_tables(plan, lens, _i32(new))
    q = torch.randn(12, 4, 128, generator=g, device="cuda").half()
    out = torch.full_like(q, 7.0)
    cache.attend(lens, q, plan=plan, out=out)
    rows = [2, None, 3, 8, None, None]
    _check_attention(cache, cache.view("block_table").cpu().numpy(), lens.tolist(), q, out, 128 ** -0.5, rows=rows)
    left = [r for r in range(12) if r not in rows]
    assert (out[left] == 7.0).all() and cache.read_status() == 0
    # rows outside q: skipped and reported
    few = q[:5].contiguous()
    out = torch.full_like(few, 7.0)
    cache.attend(lens, few, plan=plan, out=out)
    assert cache.read_status() == 11 and (out[[0, 1, 4]] == 7.0).all()
    _check_attention(cache, cache.view("block_table").cpu().numpy(), lens.tolist(), few, out, 128 ** -0.5,
                     rows=[2, None, 3, None, None, None])


def test_attention_bad_pages_and_lengths():
    """Pages outside the pool are left out, lengths the table cannot hold give zeros; both are reported."""
    g = torch.Generator("cuda").manual_seed(6)
    cache = _cache(num_seqs=5, max_blocks=6)
    _fill(cache, g)
    lens = [500, 700, -3, 5000, 260]
    table = _pages(cache, [500, 700, 0, 0, 260], random.Random(2))
    q = torch.randn(5, 2, 128, generator=g, device="cuda").half()
    bad = table.copy()
    bad[1, 1], bad[1, 3] = -1, cache.cfg.num_pages
    cache.view("block_table").copy_(torch.from_numpy(bad))
    out = cache.attend(_i32(lens), q)
    assert cache.read_status() == 11
    _check_attention(cache, table, [500, 0, 0, 0, 260], q, out, 128 ** -0.5, rows=[0, None, None, None, 4])
    assert not out[2].any() and not out[3].any()
    k, v, ka, va = _rows(cache, table, 1, 700)
    keep = torch.ones(700, dtype=torch.bool, device="cuda")
    keep[128:256] = keep[384:512] = False
    for h in range(2):
        want = ref.attend(q[1, h:h + 1].double(), k[h], v[h], 128 ** -0.5, keep)
        tol = ref.attend_bound(q[1, h:h + 1].double(), ka[h], va[h], 128 ** -0.5, keep, want)
        assert ((out[1, h:h + 1].double() - want).abs() <= tol).all()


def test_attention_nothing_to_do():
    cache = _cache()
    q = torch.randn(4, 2, 128, device="cuda").half()
    out = torch.full_like(q, 3.0)
    cache.attend(_i32([0, 0]), q, out=out)
    assert not out[:2].any() and (out[2:] == 3.0).all()
    empty = torch.zeros(0, dtype=torch.int32, device="cuda")
    cache.attend(empty, q, out=out)
    assert (out[2:] == 3.0).all()
    assert cache.attend(empty, q[:0]).shape == (0, 2, 128)
    assert cache.read_status() == 0


def test_attention_long_and_wide():
    """One long sequence split over every worker beside short ones; more heads than workers."""
    g = torch.Generator("cuda").manual_seed(4)
    cache = _cache(num_pages=300, num_seqs=3, max_blocks=300, num_kv_heads=1)
    _fill(cache, g)
    lens = [200 * 128 + 77, 1, 130]
    table = _pages(cache, lens, random.Random(3))
    q = torch.randn(3, 2, 128, generator=g, device="cuda").half()
    _check_attention(cache, table, lens, q, cache.attend(_i32(lens), q), 128 ** -0.5)
    cache = _cache(num_pages=300, num_seqs=90, max_blocks=3, num_kv_heads=64)
    _fill(cache, g)
    lens = [(37 * i) % 300 for i in range(90)]
    table = _pages(cache, lens, random.Random(3))
    q = torch.randn(90, 64, 128, generator=g, device="cuda").half()
    _check_attention(cache, table, lens[:12], q, cache.attend(_i32(lens), q), 128 ** -0.5)


@pytest.mark.parametrize("bits, G", [(2, 1), (4, 1), (2, 4), (4, 7)])
@pytest.mark.parametrize("H", [1, 3])
def test_attention_few_units(bits, G, H):
    """Few units of one row: heads in one block, in several and in many; among rows without tokens; beside a row of another length."""
    g = torch.Generator("cuda").manual_seed(H)
    blocks = 120 if H == 3 else 260
    cache = _cache(num_pages=blocks + 2, num_seqs=70, max_blocks=blocks, num_kv_heads=H, bits=bits)
    _fill(cache, g)
    for T in (1, 16, 17, 128, 129, 400, 1024, 1500, 2049, 4100, 9000, 15000) + ((20000, 33000) if H == 1 else ()):
        for lens in ([T], [0] * 5 + [T] + [0] * 64, [T, 40]):
            table = _pages(cache, lens, random.Random(T))
            q = torch.randn(len(lens), H * G, 128, generator=g, device="cuda").half()
            out = cache.attend(_i32(lens), q)
            _check_attention(cache, table, lens, q, out, 128 ** -0.5)
            assert torch.equal(out, cache.attend(_i32(lens), q)), (T, lens)
    assert cache.read_status() == 0


def test_sequences_that_share_pages():
    """The same page in two tables and twice in one (a shared prefix)."""
    g = torch.Generator("cuda").manual_seed(4)
    cache = _cache(num_seqs=3)
    _fill(cache, g)
    table = np.full((3, 16), -1, np.int32)
    table[0, :3], table[1, :3], table[2, :3] = [5, 6, 7], [5, 6, 9], [5, 5, 5]
    cache.view("block_table").copy_(torch.from_numpy(table))
    lens = [390, 400, 385]
    q = torch.randn(3, 4, 128, generator=g, device="cuda").half()
    _check_attention(cache, table, lens, q, cache.attend(_i32(lens), q), 128 ** -0.5)


# ---- steps ----------------------------------------------------------------------------------------
def _steps(cache, rng, n_steps, n, H, G, on_step, finish=True):
    """A batch that comes and goes through PagedKiviCache.step: prompts, single tokens, finished sequences."""
    R = cache.cfg.residual
    lens = torch.zeros(n, dtype=torch.int32, device="cuda")
    plan = cache.new_plan(6 * R)
    g = torch.Generator("cuda").manual_seed(rng.randrange(1000))
    held = [0] * n
    for _ in range(n_steps):
        new = []
        for i in range(n):
            if held[i] == 0:
                new.append(rng.choice([0, 1, 3, R - 1, R, R + 5]))
            elif finish and rng.random() < 0.1:
                new.append(-1)
            else:
                new.append(rng.choice([1, 1, 1, 0, 2, R // 2]))
            held[i] = 0 if new[-1] < 0 else held[i] + new[-1]
        tokens = sum(max(a, 0) for a in new)
        qkv = torch.randn(tokens, (G + 2) * H, 128, generator=g, device="cuda")
        on_step(plan, lens, new, qkv, held)
    return lens


@pytest.mark.parametrize("bits, R, G, H", [(2, 128, 1, 2), (4, 128, 4, 1), (2, 256, 3, 1)])
def test_steps(bits, R, G, H):
    """The cache holds the oracle's blocks of every sequence, and every output is attention over it."""
    n = 4
    cache = _cache(num_pages=60, num_seqs=n, max_blocks=14, num_kv_heads=H, bits=bits, residual=R)
    kv = [(np.zeros((0, H, 128), np.float16),) * 2 for _ in range(n)]

    def on_step(plan, lens, new, qkv, held):
        x = qkv.half()
        q, k, v = x[:, :G * H], x[:, G * H:(G + 1) * H], x[:, (G + 1) * H:]
        out = cache.step(plan, lens, _i32(new), q, k, v)
        assert lens.tolist() == held
        at, rows = 0, []
        kh, vh = k.cpu().numpy(), v.cpu().numpy()
        for i, a in enumerate(new):
            if a < 0:
                kv[i] = (np.zeros((0, H, 128), np.float16),) * 2
            kv[i] = tuple(np.concatenate([old, y[at:at + max(a, 0)]]) for old, y in zip(kv[i], (kh, vh)))
            at += max(a, 0)
            rows.append(at - 1 if a > 0 else None)
        _check_cache(cache, lens.tolist(), kv)
        _check_attention(cache, cache.view("block_table").cpu().numpy(), held, q, out, 128 ** -0.5, rows=rows)

    _steps(cache, random.Random(R + G), 12, n, H, G, on_step)
    assert cache.read_status() == 0


def test_steps_with_rotary():
    """step() with norms and rotation is the calls one by one, in bf16 and fp16."""
    rot = kivi.Rotary(rotary_dim=64, theta=10000.0)
    H, G, n = 2, 2, 3
    for dtype in (torch.bfloat16, torch.float16):
        a, b = (_cache(num_pages=60, num_seqs=n, max_blocks=14, num_kv_heads=H) for _ in range(2))
        lens_b = torch.zeros(n, dtype=torch.int32, device="cuda")
        plan_b = b.new_plan(6 * 128)
        w = (1 + 0.1 * torch.randn(2, 128, device="cuda")).to(dtype)

        def on_step(plan, lens, new, qkv, held):
            x = qkv.to(dtype)
            q, k, v = x[:, :G * H], x[:, G * H:(G + 1) * H], x[:, (G + 1) * H:]
            out = a.step(plan, lens, _i32(new), q, k, v, rotary=rot, q_weight=w[0], k_weight=w[1], window=200, sinks=4,
                         out=torch.zeros(q.shape, dtype=torch.float16, device="cuda"))
            b.build_tables(plan_b, lens_b, _i32(new))
            q2, k2, _ = rot.apply(q, k, positions=plan_b.positions[:len(q)], q_weight=w[0], k_weight=w[1])
            b.append(plan_b, k2, v.half().contiguous())
            out2 = b.attend(lens_b, q2, plan=plan_b, out=torch.zeros_like(q2), window=200, sinks=4)
            assert torch.equal(out, out2) and torch.equal(lens, lens_b)

        _steps(a, random.Random(5), 8, n, H, G, on_step)
        for name in ("block_table", "free_pages", "queue"):
            assert torch.equal(a.view(name), b.view(name))


def test_one_sequence_is_the_contiguous_cache():
    """A batch of equal lengths: the pages hold the contiguous cache's blocks bit for bit, outputs agree."""
    B, H, G = 2, 2, 2
    flat = kivi.KiviCache(B, H, 1024, num_q_heads=H * G)
    paged = _cache(num_seqs=B, num_kv_heads=H)
    g = torch.Generator("cuda").manual_seed(1)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    plan = paged.new_plan(2 * 300)
    for T in (253, 1, 1, 1, 1):
        k = torch.randn(B, H, T, 128, generator=g, device="cuda").half()
        v = torch.randn(B, H, T, 128, generator=g, device="cuda").half()
        q = torch.randn(B, H * G, 128, generator=g, device="cuda").half()
        if T > 1:
            flat.prefill(k, v)
            a = flat.attend(q)
        else:
            a = flat.step(k[:, :, 0].contiguous(), v[:, :, 0].contiguous(), q)
        paged.build_tables(plan, lens, _i32([T] * B))
        paged.append(plan, *(x.transpose(1, 2).reshape(B * T, H, 128) for x in (k, v)))
        b = paged.attend(lens, q)
        assert (a.double() - b.double()).abs().max() <= 2.0 ** -10  # two roundings to fp16 of outputs below 1 and 2^-12 of arithmetic
        for i in range(B):
            for j in range(flat.n_quant // 128):
                page = paged.view("block_table")[i, j].item()
                assert torch.equal(paged.view("k_codes")[page], flat.view("k_codes")[i, :, j * 128:(j + 1) * 128])
                assert torch.equal(paged.view("v_codes")[page], flat.view("v_codes")[i, :, j * 8:(j + 1) * 8])
                assert torch.equal(paged.view("k_zero")[page], flat.view("k_zero")[i, :, j])
                assert torch.equal(paged.view("v_scale")[page], flat.view("v_scale")[i, :, j * 4:(j + 1) * 4])


def test_graph_of_steps():
    """A captured step replayed over changing lengths, beside an eager cache that does the same."""
    H, G, n = 2, 4, 3
    rot = kivi.Rotary()
    a, b = (_cache(num_seqs=n, num_kv_heads=H, num_q_heads=H * G) for _ in range(2))
    lens_a, lens_b = _i32([0] * n), _i32([0] * n)
    plan_a, plan_b = a.new_plan(n * 120), b.new_plan(n * 120)
    ones = _i32([1] * n)
    g = torch.Generator("cuda").manual_seed(7)
    for cache, lens, plan in ((a, lens_a, plan_a), (b, lens_b, plan_b)):
        x = torch.randn(330, (G + 2) * H, 128, generator=torch.Generator("cuda").manual_seed(3), device="cuda").half()
        cache.step(plan, lens, _i32([120, 100, 110]), x[:, :G * H], x[:, G * H:(G + 1) * H], x[:, (G + 1) * H:], rotary=rot)
    x = torch.zeros(n, (G + 2) * H, 128, dtype=torch.float16, device="cuda")
    out = torch.zeros(n, H * G, 128, dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(plan_a, lens_a, ones, x[:, :G * H], x[:, G * H:(G + 1) * H], x[:, (G + 1) * H:], rotary=rot, out=out)
    for _ in range(40):  # every sequence crosses a block
        y = torch.randn(x.shape, generator=g, device="cuda").half()
        x.copy_(y)
        graph.replay()
        want = b.step(plan_b, lens_b, ones, y[:, :G * H], y[:, G * H:(G + 1) * H], y[:, (G + 1) * H:], rotary=rot)
        assert torch.equal(out, want) and torch.equal(lens_a, lens_b)
    assert lens_a.tolist() == [160, 140, 150] and a.read_status() == 0
    with pytest.raises(RuntimeError):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            a.attend(lens_a, torch.zeros(n, H, 128, dtype=torch.float16, device="cuda"))


def test_layers_share_tables():
    """Two layers of other heads and bits on one set of tables: one build_tables() a step, and each layer its own data."""
    n, g = 3, torch.Generator("cuda").manual_seed(5)
    first = _cache(num_seqs=n, num_kv_heads=2, bits=2)
    second = kivi.PagedKiviCache(num_pages=64, num_seqs=n, max_blocks=16, num_kv_heads=1, bits=4, group_k=128, group_v=64, tables=first)
    assert second.view("block_table").data_ptr() == first.view("block_table").data_ptr()
    lens, plan = _i32([0] * n), first.new_plan(900)
    kv = {c: [(np.zeros((0, c.cfg.num_kv_heads, 128), np.float16),) * 2 for _ in range(n)] for c in (first, second)}
    for new in ([300, 5, 127], [1, 130, 1], [1, 1, 1]):
        first.build_tables(plan, lens, _i32(new))
        for cache in (first, second):
            H, at = cache.cfg.num_kv_heads, 0
            k, v = (torch.randn(sum(new), H, 128, generator=g, device="cuda").half() for _ in range(2))
            cache.append(plan, k, v)
            q = torch.randn(sum(new), 4, 128, generator=g, device="cuda").half()
            out = cache.attend(lens, q, plan=plan)
            for i, a in enumerate(new):
                kv[cache][i] = tuple(np.concatenate([old, y[at:at + a].cpu().numpy()]) for old, y in zip(kv[cache][i], (k, v)))
                at += a
            _check_cache(cache, lens.tolist(), kv[cache])
            _check_attention(cache, cache.view("block_table").cpu().numpy(), lens.tolist(), q, out, 128 ** -0.5,
                             rows=(np.cumsum(new) - 1).tolist())
    with pytest.raises(ValueError):
        kivi.PagedKiviCache(num_pages=65, num_seqs=n, max_blocks=16, num_kv_heads=1, tables=first)


def test_append_reports_a_plan_of_more_runs_than_rows():
    cache = _cache(num_seqs=4, num_kv_heads=1)
    plan, lens = cache.new_plan(8), _i32([0] * 4)
    cache.build_tables(plan, lens, _i32([1] * 4))
    k = torch.randn(4, 1, 128, device="cuda").half()
    cache.append(plan, k, k)
    assert cache.read_status() == 0
    cache.append(plan, k[:2], k[:2])
    assert cache.read_status() == 11


def test_pool_past_32_bits():
    """Pages whose codes and residual rows lie past 2^32 bytes."""
    g = torch.Generator("cuda").manual_seed(8)
    H, pages = 16, 70000
    cache = _cache(num_pages=pages, num_seqs=5000, max_blocks=4, num_kv_heads=H)
    assert cache.buffers["k_codes"].numel() > 1 << 32 and cache.buffers["k_res"].numel() > 1 << 31
    for name in kivi.BUFFERS:
        cache.buffers[name].zero_()
    lens = torch.zeros(5000, dtype=torch.int32, device="cuda")
    new = torch.zeros(5000, dtype=torch.int32, device="cuda")
    plan = cache.new_plan(600)
    cache.view("queue").copy_(torch.tensor([pages - 4, pages]))
    new[4999], new[17] = 260, 300
    k, v = (torch.randn(560, H, 128, generator=g, device="cuda").half() for _ in range(2))
    cache.build_tables(plan, lens, new)
    cache.append(plan, k, v)
    assert cache.read_status() == 0
    assert sorted(cache.view("block_table")[[17, 4999], :2].flatten().tolist()) == list(range(pages - 4, pages))
    q = torch.randn(560, 2 * H, 128, generator=g, device="cuda").half()
    out = cache.attend(lens, q, plan=plan)
    for i, (T, row, src) in {17: (300, 299, 0), 4999: (260, 559, 300)}.items():
        page = cache.view("block_table")[i, 1].item()
        for h in (0, H - 1):
            want = _oracle_block(k[src + 128:src + 256, h].cpu().numpy(), v[src + 128:src + 256, h].cpu().numpy(), cache.cfg)
            for name, w in want.items():
                assert np.array_equal(_bits(cache.view(name)[page, h].cpu().numpy()), _bits(w)), name
        table = {i: cache.view("block_table")[i].cpu().numpy()}
        _check_attention(cache, _Rows(table), [0] * i + [T], q, out, 128 ** -0.5, rows=[None] * i + [row])


class _Rows:
    """Rows of a block table by index, as _rows reads them."""

    def __init__(self, rows):
        self.rows = rows

    def __getitem__(self, at):
        return self.rows[at[0]][at[1]]


def test_graph_with_copies_between():
    """Copies and fills between the calls of a captured step: each kernel sees what came before it."""
    H, n = 2, 3
    a, b = (_cache(num_seqs=n, num_kv_heads=H, num_q_heads=4) for _ in range(2))
    lens, plan = _i32([0] * n), a.new_plan(3 * n)
    lens_b, plan_b = _i32([0] * n), b.new_plan(3 * n)
    host = torch.randn(3 * n, 8, 128).half().pin_memory()
    x, out = (torch.zeros(r, h, 128, dtype=torch.float16, device="cuda") for r, h in ((3 * n, 8), (n, 4)))
    new, kept = _i32([3, 2, 1]), torch.zeros(n, dtype=torch.int32, device="cuda")
    q = torch.zeros(n, 4, 128, dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.build_tables(plan, lens, new)
        kept.copy_(lens)
        x.copy_(host, non_blocking=True)
        a.append(plan, x[:, 4:6], x[:, 6:8])
        x[:, 4:].zero_()
        q.copy_(x[:n, :4])
        out.fill_(9.0)
        a.attend(kept, q, out=out)
    for step in range(60):
        host.copy_(torch.randn(host.shape, generator=torch.Generator().manual_seed(step)).half())
        graph.replay()
        torch.cuda.synchronize()
        y = host.cuda()
        b.build_tables(plan_b, lens_b, new)
        b.append(plan_b, y[:, 4:6], y[:, 6:8])
        want = b.attend(lens_b, y[:n, :4].contiguous())
        assert torch.equal(out, want) and torch.equal(kept, lens_b), step
    assert a.read_status() == b.read_status() == 0 and lens.tolist() == [180, 120, 60]


def test_other_stream():
    cache = _cache(num_seqs=2)
    g = torch.Generator("cuda").manual_seed(1)
    _fill(cache, g)
    lens = _i32([500, 40])
    _pages(cache, lens.tolist(), random.Random(1))
    q = torch.randn(2, 4, 128, generator=g, device="cuda").half()
    want = cache.attend(lens, q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = cache.attend(lens, q, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    # a whole step there, of sources that have to be copied first
    rot = kivi.Rotary()
    a, b = _cache(num_seqs=2, num_q_heads=4), _cache(num_seqs=2, num_q_heads=4)
    x = torch.randn(300, 8, 128, generator=g, device="cuda").bfloat16()
    args = lambda c: (c.new_plan(300), _i32([0, 0]), _i32([170, 130]), x[:, :4], x[:, 4:6], x[:, 6:8])
    torch.cuda.synchronize()
    one = a.step(*args(a), rotary=rot, out=torch.zeros(300, 4, 128, dtype=torch.float16, device="cuda"))
    more = args(b)
    out = torch.zeros(300, 4, 128, dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    two = b.step(*more, rotary=rot, out=out, stream=side)
    side.synchronize()
    assert torch.equal(one, two) and a.read_status() == b.read_status() == 0


def test_torch_layer_refusals():
    cache = _cache(num_seqs=2)
    plan = cache.new_plan(16)
    lens, q = _i32([3, 4]), torch.zeros(2, 2, 128, dtype=torch.float16, device="cuda")
    for bad in (lambda: cache.attend(lens.long(), q), lambda: cache.attend(lens, q.float()), lambda: cache.attend(lens, q[:1]),
                lambda: cache.attend(lens, q.transpose(0, 1)), lambda: cache.attend(lens.cpu(), q),
                lambda: cache.attend(lens, q, out=q[:, :1]), lambda: cache.attend(lens, q, window=1 << 31),
                lambda: cache.build_tables(plan, lens, lens[:1]), lambda: cache.build_tables(plan, lens, lens, lens_out=lens.long()),
                lambda: cache.append(plan, q, q[:, :1]), lambda: cache.append(plan, q, q.float()),
                lambda: cache.step(plan, lens, lens, q.repeat(9, 1, 1), q, q), lambda: cache.new_plan(0)):
        with pytest.raises(ValueError):
            bad()
    other = _cache(num_seqs=3).new_plan(16)  # a plan of another geometry
    for bad in (lambda: cache.build_tables(other, lens, lens), lambda: cache.append(other, q, q), lambda: cache.attend(lens, q, plan=other),
                lambda: cache.attend(lens, q, plan=_cache(num_seqs=2, residual=256).new_plan(16))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(kivi.KiviError):
        cache.attend(lens, torch.zeros(2, 3, 128, dtype=torch.float16, device="cuda"))
    with pytest.raises(kivi.KiviError):
        _cache(residual=1024)
