"""Plain implementations of the paged-cache operators, for tests: Python and float64, no library code."""
from __future__ import annotations

import math

import numpy as np

D = 128


def build_tables(table, ring, queue, lens, new, R, max_tokens):
    """What kivi_paged_build_tables does, row by row.  table [n][width] and ring are changed in place; returns
    (lens, queue, cu, positions, runs, failed)."""
    head, tail = queue
    pages, width, n = len(ring), table.shape[1], len(lens)
    if sum(max(a, 0) for a in new) > max_tokens:
        return list(lens), (head, tail), [0] * (n + 1), [], [], True
    out, cu, positions, runs, used, asked, freed, failed = [], [0], [], [], 0, 0, [], False
    for i, (length, a) in enumerate(zip(lens, new)):
        end = length + max(a, 0)
        bad = length < 0 or length // R > width or end // R > width
        need = 0 if bad else end // R - length // R
        asked += need
        bad = bad or (need > 0 and asked > tail - head)
        cu.append(cu[-1] + max(a, 0))
        positions += [-1 if bad else length + j for j in range(max(a, 0))]
        if bad:
            failed = True
            out.append(length)
            continue
        if a < 0:
            freed += table[i, :length // R].tolist()
            out.append(0)
            continue
        for j in range(length // R, length // R + need):
            table[i, j] = ring[(head + used) % pages]
            used += 1
        out.append(end)
        blocks = list(range(length // R, (end - 1) // R + 1)) if a else []
        chained = length % R > 0 and len(blocks) > 1
        for j in blocks:
            lo, hi, last = max(length - j * R, 0), min(end - j * R, R), j == blocks[-1]
            runs.append([i, table[i, j] if hi == R else -1, cu[i] + max(j * R - length, 0), lo, hi,
                         int(last) + 2 * int(last and chained), len(blocks) - 1 if chained and j == blocks[0] else 0, 0])
    for k, p in enumerate(freed):
        ring[(tail + k) % pages] = p
    return out, (head + used, tail + len(freed)), cu, positions, runs, failed


def dequantised(kc, vc, ks, kz, vs, vz, bits):
    """float64 K and V rows of blocks: kc [..][R][128 / P], vc [..][R / P][128] int32 words, scales [..][groups]."""
    import torch
    P = 32 // bits
    R = kc.shape[-2]
    lead = kc.shape[:-2]
    sh = torch.arange(P, device=kc.device, dtype=torch.int64) * bits
    k = ((kc.long()[..., None] >> sh) & (2 ** bits - 1)).double().reshape(*lead, R, D)
    v = ((vc.long()[..., None] >> sh) & (2 ** bits - 1)).double().transpose(-1, -2).reshape(*lead, R, D)
    gk, gv = D // ks.shape[-1], R // vs.shape[-1]
    ks, kz = (x.double().repeat_interleave(gk, -1)[..., None, :] for x in (ks, kz))
    vs, vz = (x.double().repeat_interleave(gv, -1)[..., :, None] for x in (vs, vz))
    # the size of the terms a logit and an output are summed from
    return k * ks + kz, v * vs + vz, k * ks.abs() + kz.abs(), v * vs.abs() + vz.abs()


def visible(T, window, sinks):
    t = np.arange(T)
    return (t < sinks) | (t >= T - window) if window else np.ones(T, bool)


def attend(q, k, v, scale, keep):
    """q [G][128], k, v [T][128] float64: softmax over the kept tokens; zeros when none is kept."""
    import torch
    k, v = k[keep], v[keep]
    if len(k) == 0:
        return torch.zeros_like(q)
    return torch.softmax(q @ k.T * scale, -1) @ v


def attend_bound(q, kabs, vabs, scale, keep, want):
    """Largest error of an output [G][128] whose logits and weights are formed in 32 bits and rounded to fp16 once.

    A logit is a sum of products of size q_c |k_c| with fewer than 2^4 roundings of 2^-24 relative to the sum of the
    sizes A (operands of 22 bits or more, the k-chunk sums, scale and constant): below 2^-20 A.  A weight's relative
    error is that of exp, delta = 2 * 2^-20 A + 2^-20 (exp2 and the 22-bit weight operand), and the output moves by at
    most 2 delta times the largest value size.  Sums of weights add 2^-20 more.  Half a step of fp16 comes on top."""
    import torch
    kabs, vabs = kabs[keep], vabs[keep]
    if len(kabs) == 0:
        return torch.full_like(want, 2.0 ** -25)
    A = (q.abs() @ kabs.T * abs(scale)).max()
    step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0 ** -14))) - 11)
    return step + (2 * A + 4) * 2.0 ** -19 * vabs.max()


def rotate(x, weight, eps, positions, rd, interleaved, freqs, m):
    """x [tokens][heads][128] float64; freqs: radians a position of each pair."""
    import torch
    if weight is not None:
        x = x / ((x * x).mean(-1, keepdim=True) + eps).sqrt() * weight
    ang = positions.double()[:, None] * freqs
    c, s = (m * ang.cos())[:, None], (m * ang.sin())[:, None]
    y = x.clone()
    i = torch.arange(rd // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rd // 2)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y


def frequencies(rd, theta=10000.0, scaling="none", factor=1.0, low=1.0, high=4.0, original=8192):
    """(radians a position of each pair, factor of cos and sin), from the definitions in include/kivi.h."""
    if scaling == "base" and rd > 2:
        theta = theta * factor ** (rd / (rd - 2))
    f = [theta ** (-2 * i / rd) for i in range(rd // 2)]
    m = 1.0
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "bands":
        keep = [min(1, max(0, (original * x / (2 * math.pi) - low) / (high - low))) for x in f]
        f = [x * (w + (1 - w) / factor) for x, w in zip(f, keep)]
    if scaling == "ramp":
        def pair(turns):  # the (real) pair index that makes so many turns over the original context
            return rd * math.log(original / (2 * math.pi * turns)) / (2 * math.log(theta))
        a, b = max(0, math.floor(pair(high))), min(rd - 1, math.ceil(pair(low)))
        keep = [1 - min(1, max(0, (i - a) / max(b - a, 1e-3))) for i in range(rd // 2)]
        f = [x * (w + (1 - w) / factor) for x, w in zip(f, keep)]
        m = 0.1 * math.log(factor) + 1
    return f, m
