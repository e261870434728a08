"""The serving operators of the low-bit KV cache as measured work: their cases, inputs, plain forms and 64-bit definitions.

Operators (``op`` of a case):
  tables   block tables and the slot map of a step, built from request lengths (kivi_paged_build_tables)
  rotary   norms of queries and keys per head with the position rotation in the same pass (kivi_rotary)
  append   new tokens written into the paged cache: fp16 residual rows, codes of completed blocks (kivi_paged_append)
  paged    attention of one new token per request over the paged cache (kivi_paged_decode_attention)
  window   attention with a sliding window and sinks over the contiguous cache (kivi_decode_attention_window)

The cache's layout is the library's: pages (or blocks) of R tokens, P = 32 / bits codes per 32-bit word, K codes
[..][R][128 / P] with one (s, z) per block and group_k channels, V codes [..][R / P][128] with one (s, z) per group_v tokens,
the newest ((T - 1) mod R) + 1 tokens of a sequence in fp16 residual rows.
"""
import math

import numpy as np
import torch

own = False

D = 128
DEV = "cuda"


# ---- the cases ----------------------------------------------------------------------------------
def listed():
    base = dict(bits=2, gk=32, gv=32, R=128)
    return [
        # a step of 64 running requests, one new token each: what precedes every decode step (latency)
        dict(base, name="tables_decode_b64", op="tables", n=64, cached=8192, new=1, done=2),
        # a scheduling step that admits prompts of many lengths among 1000 slots
        dict(base, name="tables_prompts_b1000", op="tables", n=1000, cached=700, new=500, done=37),
        # one decode step of 8 sequences in fp16: rotation only, half layout (latency)
        dict(name="rotary_decode_b8", op="rotary", tokens=8, hq=32, hk=32, rd=128, layout="half", scaling="none", norm=False,
             dtype="float16", start=4095),
        # the prompts of a grouped-query layer in bf16, normed, a long context with scaled frequencies
        dict(name="rotary_prompt_32768", op="rotary", tokens=32768, hq=32, hk=8, rd=128, layout="half", scaling="bands", norm=True,
             dtype="bfloat16", start=98304),
        # a decode step of the large batch: 64 sequences x 32 heads, one new token each, some completing a block
        dict(base, name="append_decode_b64_h32", op="append", n=64, H=32, cached=8192, new=1),
        # the streaming prefill: 4 prompts of up to 32768 tokens, 32 heads
        dict(base, name="append_prompts_b4_h32_t32768", op="append", n=4, H=32, cached=0, new=32768),
        # one short sequence, 4 heads, 1024 tokens (latency)
        dict(base, name="paged_tiny_b1_h4_t1024", op="paged", n=1, H=4, gqa=1, T=1024, window=0, sinks=0),
        # the large batch: 64 sequences of up to 8192 tokens
        dict(base, name="paged_large_b64_h32_t8192", op="paged", n=64, H=32, gqa=1, T=8192, window=0, sinks=0),
        # grouped queries: 32 query heads over 8 KV heads, up to 32768 tokens
        dict(base, name="paged_gqa4_b16_h8_t32768", op="paged", n=16, H=8, gqa=4, T=32768, window=0, sinks=0),
        # the streaming workload's 4-bit form, odd lengths
        dict(base, name="paged_4bit_b4_h32_t32001", op="paged", n=4, H=32, gqa=1, T=32001, bits=4, gk=128, gv=128, window=0, sinks=0),
        # 8 sequences of a 32-head layer with a short window and 4 sinks
        dict(base, name="window1024_b8_h32_t4096", op="window", n=8, H=32, gqa=1, T=4096, window=1024, sinks=4),
        # grouped queries over a long 4-bit cache with a long window
        dict(base, name="window8000_b16_h8_t32700", op="window", n=16, H=8, gqa=4, T=32700, bits=4, window=8000, sinks=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rotary", "append", "paged", "paged", "window"])
    bits, R = rng.choice([2, 4]), rng.choice([128, 128, 256])
    base = dict(op=op, bits=bits, gk=rng.choice([32, 64, 128]), gv=rng.choice([32, 64, 128]), R=R)
    if op == "tables":
        n = _log(rng, 1, 1000)
        return dict(base, n=n, cached=_log(rng, 1, 8192), new=_log(rng, 1, max(1, 500000 // n)) if n > 16 else _log(rng, 1, 8192),
                    done=rng.randint(0, n // 4))
    if op == "rotary":
        hk = rng.choice([1, 2, 4, 8, 32])
        hq = hk * (1 if hk == 32 else rng.choice([1, 2, 4, 7]))
        return dict(op=op, tokens=_log(rng, 1, 40 * 32768 // (hq + hk) // 2), hq=hq, hk=hk, rd=16 * rng.randint(1, 8),
                    layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "base", "bands", "ramp"]),
                    norm=rng.random() < 0.5, dtype=rng.choice(["float16", "bfloat16"]), start=_log(rng, 1, 1000000))
    H = rng.choice([1, 2, 3, 4, 8, 32])
    if op == "append":
        if rng.random() < 0.4:
            return dict(base, n=_log(rng, 1, 64), H=H, cached=_log(rng, 1, 8192), new=1)
        n = _log(rng, 1, 16)
        return dict(base, n=n, H=H, cached=0, new=_log(rng, 1, min(32768, 4 * 32 * 32768 // (n * H) // 2)))
    n = _log(rng, 1, 64)
    gqa = rng.randint(1, 8)
    T = _log(rng, 1, min(32768, 64 * 32 * 8192 // (n * H) // 2))
    window = rng.choice([0, _log(rng, 1, T)]) if op == "paged" else _log(rng, 1, T)
    if op == "window":
        base["R"] = rng.choice([128, 256, 512, 1024])
    return dict(base, n=n, H=H, gqa=gqa, T=T, window=window, sinks=rng.choice([0, 1, 4, 5, 130]) if window else 0)


# ---- lengths, the same for every seed -----------------------------------------------------------
def _spread(n, top, salt):
    """n lengths in (top / 2, top], the first `top` itself."""
    span = max(1, top - top // 2)
    return [top - (i * 40503 * (salt + 1)) % span for i in range(n)]


def _lens(case):
    return [case["T"]] * case["n"] if case["op"] == "window" else _spread(case["n"], case["T"], 1)


def _append_lens(case):
    n, R = case["n"], case["R"]
    if case["new"] == 1:  # a decode step: every fourth sequence completes a block with this token
        old = _spread(n, max(1, case["cached"]), 2)
        old = [l // R * R + R - 1 if i % 4 == 3 else l for i, l in enumerate(old)]
        return old, [1] * n
    return [0] * n, _spread(n, case["new"], 3)


def _tables_lens(case):
    n = case["n"]
    old = _spread(n, case["cached"], 4)
    new = [1] * n if case["new"] == 1 else _spread(n, case["new"], 5)
    for i in range(case["done"]):  # finished requests return their pages
        new[(i * 31) % n] = -1
    return old, new


def _visible(case, T):
    if not case["window"]:
        return T
    start = max(0, T - case["window"])
    return T if case["sinks"] >= start else case["sinks"] + T - start


# ---- shared by the plain forms and the inputs ---------------------------------------------------
def _half(v):
    """fp16 of float64 values >= 0 in one rounding: float32 rounded to odd first."""
    f = v.float()
    f = torch.where(f.double() > v, torch.nextafter(f, torch.zeros_like(f)), f)
    return torch.where(f.double() == v, f, (f.view(torch.int32) | 1).view(torch.float32)).half()


def _codes(x, lo, hi, bits):
    """Codes and the stored (s, z) of x (float64) with group extremes lo and hi, broadcast against it."""
    s, z = _half((hi - lo) / (2 ** bits - 1)), lo + 0.0
    sd = s.double()
    c = torch.where(sd > 0, torch.round((x - z) / torch.where(sd > 0, sd, 1.0)), 0.0).clamp_(0, 2 ** bits - 1)
    return c.int(), s, z.half()


def _pack(c, bits):
    """[..][P] codes -> one int32 word."""
    w = c.long() << (torch.arange(32 // bits, device=c.device) * bits)
    w = w.sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).int()


def _quantise(k, v, bits, gk, gv):
    """Blocks k, v fp16 [N][H][R][128] -> the library's six arrays of those blocks."""
    N, H, R, _ = k.shape
    P = 32 // bits
    x = k.double().view(N, H, R, D // gk, gk)
    kc, ks, kz = _codes(x, x.amin((2, 4), keepdim=True), x.amax((2, 4), keepdim=True), bits)
    kw = _pack(kc.view(N, H, R, D // P, P), bits)
    x = v.double().view(N, H, R // gv, gv, D)
    vc, vs, vz = _codes(x, x.amin((3, 4), keepdim=True), x.amax((3, 4), keepdim=True), bits)
    vw = _pack(vc.view(N, H, R // P, P, D).transpose(3, 4), bits)
    return kw, vw, ks.view(N, H, -1), kz.view(N, H, -1), vs.view(N, H, -1), vz.view(N, H, -1)


NAMES = ("k_codes", "v_codes", "k_scale", "k_zero", "v_scale", "v_zero")


def _pool(g, case, pages, channels):
    """Quantised pages of keys with outlier channels and plain values, as the cache holds them."""
    H, R, bits, P = case["H"], case["R"], case["bits"], 32 // case["bits"]
    out = [torch.zeros(pages, H, R, D // P, dtype=torch.int32, device=DEV), torch.zeros(pages, H, R // P, D, dtype=torch.int32, device=DEV)]
    out += [torch.zeros(pages, H, D // case["gk"], dtype=torch.float16, device=DEV) for _ in range(2)]
    out += [torch.zeros(pages, H, R // case["gv"], dtype=torch.float16, device=DEV) for _ in range(2)]
    step = max(1, (1 << 26) // (H * R * D))
    for p in range(0, pages, step):
        m = min(step, pages - p)
        k = torch.randn(m, H, R, D, generator=g, device=DEV)
        k = torch.where(channels[None, :, None], 10 * k, k).half()
        v = torch.randn(m, H, R, D, generator=g, device=DEV).half()
        for o, a in zip(out, _quantise(k, v, bits, case["gk"], case["gv"])):
            o[p:p + m] = a
    return dict(zip(NAMES, out))


def _channels(g, H):
    """Four outlier channels of each KV head."""
    at = torch.rand(H, D, generator=g, device=DEV).argsort(1)[:, :4]
    return torch.zeros(H, D, dtype=torch.bool, device=DEV).scatter_(1, at, True)


def _frequencies(case):
    """Radians a position for each rotated pair, and the factor of cos and sin (float64)."""
    rd, theta, factor, orig = case["rd"], 500000.0, 8.0, 8192
    if case["scaling"] == "base":
        theta *= factor ** (rd / (rd - 2))
    f = [theta ** (-2.0 * i / rd) for i in range(rd // 2)]
    m = 1.0
    if case["scaling"] == "linear":
        f = [x / factor for x in f]
    elif case["scaling"] == "bands":
        low, high = 1.0, 4.0
        t = [min(1.0, max(0.0, (orig * x / (2 * math.pi) - low) / (high - low))) for x in f]
        f = [x * (a + (1 - a) / factor) for x, a in zip(f, t)]
    elif case["scaling"] == "ramp":
        at = [rd * math.log(orig / (r * 2 * math.pi)) / (2 * math.log(theta)) for r in (32.0, 1.0)]
        low, high = max(0, math.floor(at[0])), min(rd - 1, math.ceil(at[1]))
        t = [min(1.0, max(0.0, (i - low) / max(high - low, 1e-3))) for i in range(rd // 2)]
        f = [x * (1 - a + a / factor) for x, a in zip(f, t)]
        m = 0.1 * math.log(factor) + 1.0
    return f, m


# ---- inputs ---------------------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    s = dict(case=case)
    op = case["op"]
    if op == "rotary":
        return _prepare_rotary(case, g, s)
    R, n = case["R"], case["n"]
    if op == "tables":
        old, new = _tables_lens(case)
        H = 1
    elif op == "append":
        old, new = _append_lens(case)
        H = case["H"]
    else:
        old, new = _lens(case), [0] * n
        H = case["H"]
    if op == "window":
        return _prepare_window(case, g, s)
    blocks = [(l + max(a, 0)) // R for l, a in zip(old, new)]
    held = [l // R for l in old]
    pages, width = sum(blocks) + sum(h for h, a in zip(held, new) if a < 0) + 3, max(blocks + held) + 1
    ids = torch.randperm(pages, generator=g, device=DEV).int()
    at = torch.arange(width, device=DEV)[None]
    held_t = torch.tensor(held, device=DEV)
    first = torch.cumsum(held_t, 0) - held_t
    table = torch.where(at < held_t[:, None], ids[(first[:, None] + at).clamp(max=pages - 1)], -1)
    s.update(lens=torch.tensor(old, dtype=torch.int32, device=DEV), new=torch.tensor(new, dtype=torch.int32, device=DEV),
             block_table=table.contiguous(), free_pages=torch.roll(ids, -sum(held)).contiguous(),
             queue=torch.tensor([0, pages - sum(held)], dtype=torch.int64, device=DEV))
    tokens = sum(max(a, 0) for a in new)
    most_runs = 2 * n + (tokens + 5) // R
    s.update(lens_out=torch.zeros(n, dtype=torch.int32, device=DEV), queue_out=torch.zeros(2, dtype=torch.int64, device=DEV),
             cu_tokens=torch.zeros(n + 1, dtype=torch.int32, device=DEV), positions=torch.full((tokens + 5,), -7, dtype=torch.int32, device=DEV),
             runs=torch.full((most_runs, 8), -7, dtype=torch.int32, device=DEV), counts=torch.zeros(2, dtype=torch.int32, device=DEV))
    chan = _channels(g, H)
    if op == "append":
        P = 32 // case["bits"]
        for name, shape, dt in (("k_codes", (R, D // P), torch.int32), ("v_codes", (R // P, D), torch.int32),
                                ("k_scale", (D // case["gk"],), torch.float16), ("k_zero", (D // case["gk"],), torch.float16),
                                ("v_scale", (R // case["gv"],), torch.float16), ("v_zero", (R // case["gv"],), torch.float16)):
            s[name] = torch.zeros(pages, H, *shape, dtype=dt, device=DEV)
        k = torch.empty(tokens, H, D, dtype=torch.float16, device=DEV).normal_(generator=g)
        s["k"] = k.mul_(torch.where(chan, 10.0, 1.0).half()[None])
        s["v"] = torch.empty(tokens, H, D, dtype=torch.float16, device=DEV).normal_(generator=g)
        _plain_tables(s)  # the plan that the step's program has built before it appends
    elif op == "paged":
        s.update(_pool(g, case, pages, chan))
        s["q"] = torch.randn(n, H * case["gqa"], D, generator=g, device=DEV).half()
    if op != "tables":
        k = torch.randn(n, H, R, D, generator=g, device=DEV)
        s["k_res"] = torch.where(chan[None, :, None], 10 * k, k).half()
        s["v_res"] = torch.randn(n, H, R, D, generator=g, device=DEV).half()
    if own:
        from bit_asymmetric_kv_02_b200 import kivi
        cache = kivi.PagedKiviCache(num_pages=pages, num_seqs=n, max_blocks=width, num_kv_heads=H, bits=case["bits"], group_k=case["gk"],
                                    group_v=case["gv"], residual=R, num_q_heads=H * case.get("gqa", 1))
        for name in ("block_table", "free_pages", "queue") + (() if op == "tables" else NAMES + ("k_res", "v_res")):
            s[name] = cache.view(name).copy_(s[name])
        plan = cache.new_plan(max_tokens=tokens + 5)
        for name in ("cu_tokens", "positions", "runs", "counts"):
            s[name] = getattr(plan, name).copy_(s[name])
        s.update(cache=cache, plan=plan)
    return s


def _prepare_rotary(case, g, s):
    dt = getattr(torch, case["dtype"])
    N, hq, hk = case["tokens"], case["hq"], case["hk"]
    # one projection's output holds queries, keys and values side by side, as models keep them
    s["qkv"] = torch.randn(N, hq + 2 * hk, D, generator=g, device=DEV).to(dt)
    s["positions"] = (case["start"] + torch.arange(N, device=DEV)).int()
    for name in ("q_weight", "k_weight"):
        s[name] = (1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(dt) if case["norm"] else None
    if own:
        from bit_asymmetric_kv_02_b200 import kivi
        s["rotary"] = kivi.Rotary(rotary_dim=case["rd"], theta=500000.0, interleaved=case["layout"] == "interleaved", scaling=case["scaling"],
                                  factor=8.0, original_positions=8192)
    return s


def _prepare_window(case, g, s):
    n, H, R, T = case["n"], case["H"], case["R"], case["T"]
    nq = (T - 1) // R * R
    cap = nq + R
    chan = _channels(g, H)
    blocks = _pool(g, case, n * (cap // R), chan)
    P = 32 // case["bits"]
    for name in NAMES:  # [B * C / R][H][..] -> [B][H][C ..][..]
        x = blocks[name].view(n, cap // R, *blocks[name].shape[1:]).transpose(1, 2)
        tail = {"k_codes": (cap, D // P), "v_codes": (cap // P, D), "k_scale": (cap // R, D // case["gk"]),
                "k_zero": (cap // R, D // case["gk"])}.get(name, (cap // case["gv"],))
        s[name] = x.reshape(n, H, *tail)
    k = torch.randn(n, H, R, D, generator=g, device=DEV)
    s["k_res"] = torch.where(chan[None, :, None], 10 * k, k).half()
    s["v_res"] = torch.randn(n, H, R, D, generator=g, device=DEV).half()
    s["q"] = torch.randn(n, H * case["gqa"], D, generator=g, device=DEV).half()
    if own:
        from bit_asymmetric_kv_02_b200 import kivi
        cache = kivi.KiviCache(n, H, cap, bits=case["bits"], group_k=case["gk"], group_v=case["gv"], residual=R)
        for name in NAMES + ("k_res", "v_res"):
            s[name] = cache.view(name).copy_(s[name])
        cache.c.n_quant, cache.c.n_res = nq, T - nq
        s["cache"] = cache
    return s


# ---- one pass -------------------------------------------------------------------------------------
def run(s):
    case = s["case"]
    return {"tables": _run_tables, "rotary": _run_rotary, "append": _run_append, "paged": _run_paged, "window": _run_window}[case["op"]](s, case)


def _run_tables(s, case):
    if own:
        s["cache"].build_tables(s["plan"], s["lens"], s["new"], lens_out=s["lens_out"], queue_out=s["queue_out"])
    else:
        _plain_tables(s)
    return [s[x] for x in ("block_table", "free_pages", "lens_out", "queue_out", "cu_tokens", "positions", "runs", "counts")]


def _plain_tables(s):
    """The step's block table, page queue, positions and runs, in whole numbers."""
    R = s["case"]["R"]
    table, ring = s["block_table"], s["free_pages"]
    L, new, queue = s["lens"].long(), s["new"].long(), s["queue"]
    n, width, pages, dev = len(L), table.shape[1], len(ring), L.device
    cnt = new.clamp(min=0)
    cu = torch.cat([cnt.new_zeros(1), cnt.cumsum(0)])
    have, end = L // R, L + cnt
    wide = end // R > width
    need = torch.where(wide | (new < 0), 0, end // R - have)
    upto = need.cumsum(0)
    ok = (new >= 0) & ~wide & ((need == 0) | (upto <= queue[1] - queue[0]))
    back = torch.where(new < 0, have, 0)
    back_to = back.cumsum(0) - back
    at = torch.arange(width, device=dev)[None]
    # finished requests: their pages go behind the queue's tail
    gone = at < back[:, None]
    slot = (queue[1] + back_to[:, None] + at) % pages
    taken = (at >= have[:, None]) & (at < (have + need)[:, None]) & ok[:, None]
    page = ring[(queue[0] + (upto - need)[:, None] + at - have[:, None]) % pages]
    ring[slot[gone]] = table[:n][gone]
    table[:n] = torch.where(taken, page, table[:n])
    used = torch.where(ok, need, 0).sum()
    s["queue_out"].copy_(torch.stack([queue[0] + used, queue[1] + back.sum()]))
    s["lens_out"].copy_(torch.where(new < 0, 0, torch.where(ok, end, L)))
    s["cu_tokens"].copy_(cu)
    total = int(cu[-1])
    row = torch.repeat_interleave(torch.arange(n, device=dev), cnt)
    s["positions"][:total] = torch.where(ok[row], L[row] + torch.arange(total, device=dev) - cu[row], -1).int()
    touched = torch.where(ok & (cnt > 0), (end - 1) // R - have + 1, 0)
    r = torch.repeat_interleave(torch.arange(n, device=dev), touched)
    k = torch.arange(len(r), device=dev) - (touched.cumsum(0) - touched)[r]
    b = have[r] + k
    lo, hi = torch.maximum(L[r], b * R) - b * R, torch.minimum(end[r], (b + 1) * R) - b * R
    last = k == touched[r] - 1
    chained = (L % R > 0) & (touched > 1)  # the first run still reads residual rows that the last one replaces
    chain = torch.where(chained[r] & (k == 0), touched[r] - 1, 0)
    flags = last.long() + 2 * (last & chained[r]).long()
    page = torch.where(hi == R, table[r, b.clamp(max=width - 1)].long(), -1)
    src = cu[r] + b * R + lo - L[r]
    s["runs"][:len(r)] = torch.stack([r, page, src, lo, hi, flags, chain, torch.zeros_like(r)], 1).int()
    s["counts"].copy_(torch.tensor([len(r), total], device=dev))


def _run_rotary(s, case):
    hq, hk = case["hq"], case["hk"]
    q, k = s["qkv"][:, :hq], s["qkv"][:, hq:hq + hk]
    if own:
        return s["rotary"].apply(q, k, positions=s["positions"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6)[:2]
    f, m = _frequencies(case)
    a = s["positions"].double()[:, None] * torch.tensor(f, dtype=torch.float64, device=q.device)
    c, sn = (m * a.cos()).float()[:, None], (m * a.sin()).float()[:, None]
    return _plain_rotate(q, s["q_weight"], c, sn, case), _plain_rotate(k, s["k_weight"], c, sn, case)


def _plain_rotate(x, w, c, sn, case):
    x, rd = x.float(), case["rd"]
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
    if case["layout"] == "half":
        a, b = x[..., :rd // 2], x[..., rd // 2:rd]
        y = torch.cat([a * c - b * sn, a * sn + b * c], -1)
    else:
        a, b = x[..., :rd:2], x[..., 1:rd:2]
        y = torch.stack([a * c - b * sn, a * sn + b * c], -1).flatten(-2)
    return torch.cat([y, x[..., rd:]], -1).half()


def _run_append(s, case):
    if own:
        s["cache"].append(s["plan"], s["k"], s["v"])
    else:
        _plain_append(s, case)
    return [s[x] for x in NAMES + ("k_res", "v_res")]


def _plain_append(s, case):
    R = case["R"]
    runs = s["runs"][:int(s["counts"][0])].long()
    row = torch.arange(R, device=runs.device)[None]
    full = runs[runs[:, 1] >= 0]
    src = (full[:, 2:3] + row - full[:, 3:4]).clamp(0, len(s["k"]) - 1)
    fresh = (row >= full[:, 3:4])[:, :, None, None]
    k = torch.where(fresh, s["k"][src], s["k_res"][full[:, 0]].transpose(1, 2)).transpose(1, 2)
    v = torch.where(fresh, s["v"][src], s["v_res"][full[:, 0]].transpose(1, 2)).transpose(1, 2)
    if len(full):
        for name, a in zip(NAMES, _quantise(k.contiguous(), v.contiguous(), case["bits"], case["gk"], case["gv"])):
            s[name][full[:, 1]] = a
    last = runs[(runs[:, 5] & 1) == 1]
    r, t = torch.nonzero((row >= last[:, 3:4]) & (row < last[:, 4:5]), as_tuple=True)
    for res, x in (("k_res", "k"), ("v_res", "v")):
        s[res][last[r, 0], :, t] = s[x][last[r, 2] + t - last[r, 3]]


def _unpack(w, bits):
    return (w[..., None] >> (torch.arange(32 // bits, dtype=torch.int32, device=w.device) * bits)) & (2 ** bits - 1)


def _dequantise(kc, vc, ks, kz, vs, vz, case):
    """Blocks as fp32: [..][R][128] of K and of V."""
    R, bits = case["R"], case["bits"]
    lead = ks.shape[:-1]
    k = _unpack(kc, bits).view(*lead, R, D // case["gk"], case["gk"])
    k = (k * ks.float()[..., None, :, None] + kz.float()[..., None, :, None]).view(*lead, R, D)
    v = _unpack(vc, bits).transpose(-1, -2).reshape(*lead, R // case["gv"], case["gv"], D)
    v = (v * vs.float()[..., None, None] + vz.float()[..., None, None]).view(*lead, R, D)
    return k, v


def _plain_attend(q, k, v, k_res, v_res, lens, case):
    """q [n][H * gqa][128]; k, v fp32 [n][blocks][H][R][128] of the quantised blocks; residual rows [n][H][R][128]."""
    n, nb, H, R, _ = k.shape
    G = case["gqa"]
    q = q.float().view(n, 1, H, G, D).transpose(3, 4)
    lens = lens.long()[:, None]
    nq = (lens - 1).clamp(min=0) // R * R
    t = torch.arange(nb * R + R, device=q.device)[None]
    pos = torch.where(t < nb * R, t, nq + t - nb * R)
    seen = (pos < lens) & torch.where(t < nb * R, t < nq, True)
    if case["window"]:
        seen &= (pos < case["sinks"]) | (pos >= lens - case["window"])
    logits = torch.cat([k @ q, (k_res.float()[:, None] @ q)], 1) / math.sqrt(D)  # [n][nb + 1][H][R][G]
    seen = seen.view(n, nb + 1, 1, R, 1)
    logits = torch.where(seen, logits, -math.inf)
    e = torch.exp(logits - logits.amax((1, 3), keepdim=True))
    p = (e / e.sum((1, 3), keepdim=True)).transpose(3, 4)
    out = (p[:, :nb] @ v).sum(1) + p[:, nb] @ v_res.float()
    return out.view(n, H * G, D).half()


def _run_paged(s, case):
    if own:
        return s["cache"].attend(s["lens"], s["q"], window=case["window"], sinks=case["sinks"])
    nb = max(1, (case["T"] - 1) // case["R"])
    at = s["block_table"][:, :nb].long().clamp(min=0)
    k, v = _dequantise(*(s[x][at] for x in NAMES), case)
    return _plain_attend(s["q"], k, v, s["k_res"], s["v_res"], s["lens"], case)


def _run_window(s, case):
    if own:
        return s["cache"].attend_window(s["q"], case["window"], sinks=case["sinks"])
    n, H, R = case["n"], case["H"], case["R"]
    nb = s["k_codes"].shape[2] // R
    P = 32 // case["bits"]
    blocks = [s["k_codes"].view(n, H, nb, R, D // P), s["v_codes"].view(n, H, nb, R // P, D), s["k_scale"], s["k_zero"],
              s["v_scale"].view(n, H, nb, -1), s["v_zero"].view(n, H, nb, -1)]
    k, v = _dequantise(*(x.transpose(1, 2).contiguous() for x in blocks), case)
    lens = torch.full((n,), case["T"], device=k.device)
    return _plain_attend(s["q"], k, v, s["k_res"], s["v_res"], lens, case)


# ---- what a pass cannot do without ----------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "rotary":
        e = case["tokens"] * (case["hq"] + case["hk"]) * D
        return {"bytes": 4 * e + 4 * case["tokens"] + (4 * D if case["norm"] else 0), "flops": e * (3 + (4 if case["norm"] else 0))}
    R = case["R"]
    if op == "tables":
        old, new = _tables_lens(case)
        tokens = sum(max(a, 0) for a in new)
        blocks = sum((l + a) // R - l // R if a >= 0 else 2 * (l // R) for l, a in zip(old, new))
        runs = sum((l + a - 1) // R - l // R + 1 for l, a in zip(old, new) if a > 0)
        return {"bytes": 16 * case["n"] + 4 * tokens + 8 * blocks + 32 * runs + 44, "flops": 0}
    H, bits = case["H"], case["bits"]
    page = 2 * R * D * bits // 8 + 4 * (D // case["gk"]) + 4 * (R // case["gv"])  # codes and (s, z) of one block, K and V
    if op == "append":
        old, new = _append_lens(case)
        total = 0
        for l, a in zip(old, new):
            total += 4 * D * a + ((l + a) // R - l // R) * page + 4 * D * min(a, (l + a - 1) % R + 1)
            total += 4 * D * (l % R) if (l + a) // R > l // R else 0  # residual rows that join a completed block
        return {"bytes": H * total, "flops": 0}
    total = flops = 0
    for T in _lens(case):
        nq = (T - 1) // R * R
        start = max(0, T - case["window"]) if case["window"] else 0
        sinks = min(case["sinks"], start)
        first = max(start - nq, 0)
        res = (T - nq - first) + max(0, min(sinks, T) - nq)
        total += (max(0, nq - start) + min(sinks, nq)) / R * page + 4 * D * res + 4 * D * case["gqa"]
        flops += 4 * D * case["gqa"] * _visible(case, T)
    return {"bytes": H * total, "flops": H * flops}


# ---- the definitions in 64 bits ---------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "tables":
        return _exact_tables(s, case)
    if op == "rotary":
        return _exact_rotary(s, case)
    if op == "append":
        return _exact_append(s, case)
    return _exact_attention(s, case)


def _exact_tables(s, case):
    """Request by request."""
    R = case["R"]
    table, ring = s["block_table"].cpu().numpy().copy(), s["free_pages"].cpu().numpy().copy()
    L, new, (head, tail) = s["lens"].tolist(), s["new"].tolist(), s["queue"].tolist()
    positions, runs = s["positions"].cpu().numpy().copy(), s["runs"].cpu().numpy().copy()
    pages, width = len(ring), table.shape[1]
    out, cu, nr, avail, used, asked, freed = [], [0], 0, tail - head, 0, 0, []
    for i, (l, a) in enumerate(zip(L, new)):
        if a < 0:
            freed += table[i, :l // R].tolist()
            out.append(0)
            cu.append(cu[-1])
            continue
        need = (l + a) // R - l // R
        bad = (l + a) // R > width
        asked += 0 if bad else need
        bad = bad or (need > 0 and asked > avail)
        positions[cu[-1]:cu[-1] + a] = -1 if bad else np.arange(l, l + a)
        if not bad:
            for j in range(l // R, l // R + need):
                table[i, j] = ring[(head + used) % pages]
                used += 1
            blocks = list(range(l // R, (l + a - 1) // R + 1)) if a else []
            for j in blocks:
                lo, hi = max(l - j * R, 0), min(l + a - j * R, R)
                last, chained = j == blocks[-1], l % R > 0 and len(blocks) > 1
                runs[nr] = [i, table[i, j] if hi == R else -1, cu[-1] + max(j * R - l, 0), lo, hi, last + 2 * (last and chained),
                            len(blocks) - 1 if chained and j == blocks[0] else 0, 0]
                nr += 1
        out.append(l if bad else l + a)
        cu.append(cu[-1] + a)
    for j, p in enumerate(freed):
        ring[(tail + j) % pages] = p
    return [table, ring, np.array(out, np.int32), np.array([head + used, tail + len(freed)]), np.array(cu, np.int32), positions, runs,
            np.array([nr, cu[-1]], np.int32)]


def _exact_rotary(s, case):
    """Each pair as a complex number times m exp(i pos f), a part of the tokens at a time."""
    f, m = _frequencies(case)
    f = torch.tensor(f, dtype=torch.float64, device=DEV)
    rd, out = case["rd"], []
    for x, w in ((s["qkv"][:, :case["hq"]], s["q_weight"]), (s["qkv"][:, case["hq"]:case["hq"] + case["hk"]], s["k_weight"])):
        parts = []
        for x, pos in zip(x.split(2048), s["positions"].split(2048)):
            x = x.double()
            if w is not None:
                x = x / ((x ** 2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
            y = x.clone()
            turn = torch.polar(torch.full_like(f, m).expand(len(pos), -1).contiguous(), pos.double()[:, None] * f)[:, None]
            i = torch.arange(rd // 2, device=DEV)
            a, b = (i, i + rd // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
            z = torch.complex(x[..., a], x[..., b]) * turn
            y[..., a], y[..., b] = z.real, z.imag
            parts.append(y)
        out.append(torch.cat(parts))
    return tuple(out)


def _exact_append(s, case):
    """Sequence by sequence, block by block from the tokens in order."""
    R, H, bits, gk, gv = case["R"], case["H"], case["bits"], case["gk"], case["gv"]
    P, top = 32 // bits, 2 ** bits - 1
    old, new = _append_lens(case)
    at = 0
    shift = torch.arange(P, device=DEV) * bits

    def coded(x, dims):
        lo, hi = x.amin(dims, keepdim=True), x.amax(dims, keepdim=True)
        sc = torch.from_numpy(((hi - lo) / top).cpu().numpy().astype(np.float16)).to(DEV)  # numpy rounds float64 to fp16 once
        d = sc.double()
        c = torch.where(d == 0, torch.zeros_like(x), ((x - lo) / d).nan_to_num(0, 0, 0).round().clamp(0, top))
        return c.long(), sc, (lo + 0.0).half()

    def words(c):
        w = (c << shift).sum(-1)
        return (w - ((w >> 31) << 32)).int()

    for i, (l, a) in enumerate(zip(old, new)):
        kr, vr = s["k_res"][i].clone(), s["v_res"][i].clone()
        begin = l // R * R
        k = torch.cat([kr[:, :l - begin], s["k"][at:at + a].transpose(0, 1)], 1)
        v = torch.cat([vr[:, :l - begin], s["v"][at:at + a].transpose(0, 1)], 1)
        at += a
        done = (l + a) // R - l // R
        pages = s["block_table"][i, l // R:l // R + done].long()
        for b in range(0, done, 32):
            m = min(32, done - b)
            x = k[:, b * R:(b + m) * R].double().view(H, m, R, D // gk, gk).transpose(0, 1)
            c, sc, z = coded(x, (2, 4))
            s["k_codes"][pages[b:b + m]] = words(c.reshape(m, H, R, D // P, P))
            s["k_scale"][pages[b:b + m]], s["k_zero"][pages[b:b + m]] = sc.reshape(m, H, -1), z.reshape(m, H, -1)
            x = v[:, b * R:(b + m) * R].double().view(H, m, R // gv, gv, D).transpose(0, 1)
            c, sc, z = coded(x, (3, 4))
            s["v_codes"][pages[b:b + m]] = words(c.reshape(m, H, R // P, P, D).transpose(3, 4))
            s["v_scale"][pages[b:b + m]], s["v_zero"][pages[b:b + m]] = sc.reshape(m, H, -1), z.reshape(m, H, -1)
        keep = (l + a - 1) // R * R - begin  # the newest tokens stay in residual rows
        s["k_res"][i, :, :k.shape[1] - keep], s["v_res"][i, :, :k.shape[1] - keep] = k[:, keep:], v[:, keep:]
    return [s[x].double() if s[x].dtype == torch.float16 else s[x] for x in NAMES + ("k_res", "v_res")]


def _exact_attention(s, case):
    """Sequence by sequence: the visible tokens in order, their weights, the weighted sum."""
    n, H, R, G, bits, gk, gv = (case[x] for x in ("n", "H", "R", "gqa", "bits", "gk", "gv"))
    P = 32 // bits
    out = torch.zeros(n, H * G, D, dtype=torch.float64, device=DEV)
    shift = torch.arange(P, device=DEV, dtype=torch.int64) * bits
    for i, T in enumerate(_lens(case)):
        nb = (T - 1) // R
        if case["op"] == "paged":
            at = s["block_table"][i, :nb].long()
            kc, vc, ks, kz, vs, vz = (s[x][at].transpose(0, 1) for x in NAMES)  # [H][nb][..]
        else:
            kc, vc, ks, kz, vs, vz = (s[x][i].reshape(H, s["k_codes"].shape[2] // R, -1)[:, :nb] for x in NAMES)
        k = ((kc.reshape(H, nb, R, D // P, 1).long() >> shift) % 2 ** bits).double().reshape(H, nb, R, D // gk, gk)
        k = k * ks.double().reshape(H, nb, 1, D // gk, 1) + kz.double().reshape(H, nb, 1, D // gk, 1)
        v = ((vc.reshape(H, nb, R // P, 1, D).long() >> shift[:, None]) % 2 ** bits).double().reshape(H, nb, R // gv, gv, D)
        v = v * vs.double().reshape(H, nb, R // gv, 1, 1) + vz.double().reshape(H, nb, R // gv, 1, 1)
        k = torch.cat([k.reshape(H, nb * R, D), s["k_res"][i, :, :T - nb * R].double()], 1)
        v = torch.cat([v.reshape(H, nb * R, D), s["v_res"][i, :, :T - nb * R].double()], 1)
        keep = torch.arange(T, device=DEV)
        if case["window"]:
            keep = keep[(keep < case["sinks"]) | (keep >= T - case["window"])]
        w = torch.softmax(s["q"][i].double().view(H, G, D) @ k[:, keep].transpose(1, 2) / math.sqrt(D), -1)
        out[i] = (w @ v[:, keep]).reshape(H * G, D)
    return out
