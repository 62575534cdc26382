"""Float64 references of rotary positions and of the packed-batch operators, written from their
definitions; nothing here uses the library."""
from __future__ import annotations

import math

import torch

from tests import paged_ref as R

E4M3 = torch.float8_e4m3fn


def frequencies(rot, base=10000.0, scaling=None, factor=1.0, original=0.0, fast=32.0, slow=1.0):
    """(radians per position of each pair, factor of the turned channels)."""
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    m = 1.0
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "parts":
        m = 0.1 * math.log(factor) + 1
        g = [min(1.0, max(0.0, (original * x / (2 * math.pi) - slow) / (fast - slow))) for x in f]
        f = [x * (k + (1 - k) / factor) for x, k in zip(f, g)]
    return torch.tensor(f, dtype=torch.float64), m


def turn(x, pos, freq, m, neighbours, inverse=False, short=True):
    """(y, tolerance before y is rounded): x [..., N, d] float64 turned by pos [..., N].

    Short (bf16 is written): an angle is off by 2^-24 of half a turn (its fp32 rounding; the 64-bit
    product's upper half adds 2^-32 of a turn) and once more where it becomes radians, the sine and
    cosine by 2^-21.19 (the bound of CUDA's __cosf between -pi and pi), the scale and the two
    products and their sum by 2^-24 each: with |c|, |s| <= m, that is
    (2 pi + 2^2.81 + 3) 2^-24 (|a| + |b|) m at most, below 16.4 * 2^-24.  Else the angle has its 32
    bits (2^-29.3 radians), sine and cosine are off by 2 ulp, 4 * 2^-24, at most, and by 2^-24 where
    the last eight bits are added: 4 + 1 + 3 and a little, 8.1 * 2^-24.  The frequencies of both
    sides carry 2^-51 of a far angle.
    """
    r = 2 * freq.numel()
    angle = pos.double()[..., None] * freq.to(x.device)
    if inverse:
        angle = -angle
    c, s = torch.cos(angle) * m, torch.sin(angle) * m
    y, tol = x.clone(), torch.zeros_like(x)
    ia, ib = (slice(0, r, 2), slice(1, r, 2)) if neighbours else (slice(0, r // 2),
                                                                   slice(r // 2, r))
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    t = (a.abs() + b.abs()) * m * ((16.4 if short else 8.1) * 2.0 ** -24 + angle.abs() * 2.0 ** -51)
    tol[..., ia], tol[..., ib] = t, t
    return y, tol


def rounded(y, tol, dtype):
    """The tolerance of y rounded to dtype: half a step of the largest value it may have."""
    if dtype == E4M3:  # 2^-4 of the value, at least half of the smallest step
        return tol + ((y.abs() + tol) * 2.0 ** -4).clamp_min(2.0 ** -10)
    eps = torch.finfo(dtype).eps / 2
    return tol + (y.abs() + tol) * eps + 1e-37


def step(new, lens, held, table, free, count, page, max_pages, N):
    """The step on lists; None where it does not fit, else the new state and outputs."""
    lens, held, free = list(lens), list(held), list(free)
    table = [list(t) for t in table]
    after = [0 if n == -1 else x + n for n, x in zip(new, lens)]
    for n, x, a, h in zip(new, lens, after, held):
        if n < -1 or x < 0 or a > max_pages * page or not -(-x // page) <= h <= max_pages:
            return None
    need = [-(-a // page) for a in after]
    given = [(b, k) for b in range(len(new)) for k in range(need[b], held[b])]
    taken = [(b, k) for b in range(len(new)) for k in range(held[b], need[b])]
    if count < 0 or count + len(given) > len(free) or len(taken) > count + len(given) or \
            sum(max(0, n) for n in new) > N:
        return None
    for b, k in given:
        free[count] = table[b][k]
        count += 1
    for b, k in taken:
        count -= 1
        table[b][k] = free[count]
    q_start, positions, slots = [0], [], []
    for b, n in enumerate(new):
        for t in range(after[b] - max(0, n), after[b]):
            positions.append(t)
            slots.append(table[b][t // page] * page + t % page)
        q_start.append(len(positions))
    left = [-1] * (N - len(positions))
    return dict(kv_len=after, held=need, page_table=table, free_pages=free, free_count=[count],
                q_start=q_start, positions=positions + left, slots=slots + left)


def attend(c, q_start, q1, q2, lam, *, causal=True, headnorm=1, norm_w=None, eps=1e-5,
           lambda_init=0.0):
    """(out [T, H, 2d], tolerance) in float64; rows of no sequence are left at zero.

    The tolerance is paged_ref.attend's with probabilities in the second product as one bf16
    number (bf16 has 8 significant bits, so a step is 2^-7 of the binade's least value and half of
    one at most 2^-8 of a value, torch.finfo(torch.bfloat16).eps / 2).

    The sum of a row's first tile is of the rounded numbers p (1 + e), |e| <= E = 2^-8, that of the
    others of the unrounded ones.  With F the first tile's keys and S = sum_F p e <= E,
        o' - o = (sum_all p v (1 + e)) / (1 + S) - o = (sum_all p e v - S o) / (1 + S),
    at most (E sum p |v| + E |o|) / (1 - E) for each map: the maps' own |o| beside sum p |v|, and a
    factor of 1 / (1 - 2^-8) that the last line's 1.01 holds.
    """
    T, H, d = q1.shape
    G = H // c.kv
    out = torch.zeros(T, H, 2 * d, dtype=torch.float64, device=q1.device)
    tol = torch.zeros_like(out)
    for b in range(c.B):
        n, s, e = c.lens[b], q_start[b], q_start[b + 1]
        first = n - (e - s)
        for h in range(H):
            k1, k2, v = (R.f64(c.rows(t, b))[h // G] for t in ("k1", "k2", "v"))
            pos = torch.arange(first, n, device=q1.device)
            rows = (pos >= 0).nonzero().flatten()
            if not len(rows):
                continue
            j = torch.arange(n, device=q1.device)
            see = j[None] <= (pos[rows, None] if causal else n - 1)
            maps, dx = [], torch.zeros(len(rows), dtype=torch.float64, device=q1.device)
            for q, k in ((q1, k1), (q2, k2)):
                qr = R.f64(q[s:e, h])[rows]
                x = torch.where(see, qr @ k.T / math.sqrt(d), -math.inf)
                maps.append(torch.softmax(x, -1))
                size = torch.where(see & torch.isfinite(x), qr.abs() @ k.abs().T, 0.0).nan_to_num(0)
                dx = torch.maximum(dx, size.amax(-1) / math.sqrt(d) * 1.4427 * (d / 16 + 2)
                                   * 2.0 ** -22 + 2.0 ** -22)
            lh = float(lam[h])
            w = maps[0] - lh * maps[1]
            vs = torch.where(torch.isfinite(v), v, 0.0)
            o = w @ vs
            both = maps[0] + abs(lh) * maps[1]
            own = (maps[0] @ vs).abs() + abs(lh) * (maps[1] @ vs).abs()
            rel = 2 * (math.log(2) * dx + 2.0 ** -22) + 2 * (n / 16 + 8) * 2.0 ** -23
            a = (both @ vs.abs()) * (rel[:, None] + 2.0 ** -8 + 2.0 ** -16) + own * 2.0 ** -8
            bad = (see[:, :, None] & ~torch.isfinite(v)[None]).any(1) if not \
                torch.isfinite(v).all() else torch.zeros_like(o, dtype=torch.bool)
            o = torch.where(bad, math.nan, o)
            y, at = o, a
            if headnorm:
                if headnorm == 2:
                    o = o - o.mean(-1, keepdim=True)
                    a = a + a.mean(-1, keepdim=True)
                rms = torch.sqrt((o * o).mean(-1, keepdim=True) + eps)
                gain = (R.f64(norm_w[h]) if norm_w is not None else torch.ones(
                    2 * d, dtype=torch.float64, device=q1.device)) * (1 - lambda_init)
                y = o / rms * gain
                # of each value its own, and of the root mean square's change the quadratic mean
                at = gain.abs() * (a + o.abs() / rms * (a * a).mean(-1, keepdim=True).sqrt()) / rms
            out[s + rows, h] = y
            tol[s + rows, h] = at * 1.01 + y.abs() * (2.0 ** -8 + 12 * 2.0 ** -24) + 1e-30
    return out, tol
