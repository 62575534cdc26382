"""Float64 references of the paged-cache operators and the caches their tests use.

Written from the operators' definitions, position by position; nothing here uses the library.
"""
from __future__ import annotations

import math

import torch

E4M3 = torch.float8_e4m3fn


def f64(t):
    return t.float().double()


class Cache:
    """Pools with every place filled (`fill` where no token of a sequence sits), a shuffled page
    table whose unused entries are -1, and the B sequences' true rows."""

    def __init__(self, seed, *, lens, kv, d, page, dtype=torch.bfloat16, layout="head",
                 weights=False, fill=float("nan"), spare=2, device="cuda", extra_pages=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.kv, self.d, self.page, self.dtype = list(lens), kv, d, page, dtype
        B = len(lens)
        self.B = B
        self.max_pages = max(1, max(-(-n // page) for n in lens)) + extra_pages
        P = sum(-(-n // page) for n in lens) + spare
        ids = torch.randperm(P, generator=g).tolist()
        table = torch.full((B, self.max_pages), -1, dtype=torch.int32)
        for b, n in enumerate(lens):
            for k in range(-(-n // page)):
                table[b, k] = ids.pop()

        def pool(width, dt):
            x = torch.full((P, kv, page, width), fill)
            for b, n in enumerate(lens):
                for k in range(-(-n // page)):
                    m = min(page, n - k * page)
                    x[table[b, k].item(), :, :m] = torch.randn(kv, m, width, generator=g)
            x = x.to(device).to(dt)
            if layout == "token":
                x = x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
            return x

        self.k1, self.k2 = pool(d, dtype), pool(d, dtype)
        self.v = pool(2 * d, torch.bfloat16)
        self.weights = None
        if weights:
            self.weights = torch.rand(P, kv, page, generator=g).to(device) * 0.25
        self.table = table.to(device)
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device=device)

    def ops_cache(self):
        from differential_attention_attn_gb300 import ops
        return ops.PagedCache(self.k1, self.k2, self.v, self.table, self.kv_len,
                              weights=self.weights)

    def rows(self, name, b, n=None):
        """Positions 0 .. n - 1 of sequence b: [kv, n, width] (or [kv, n] weights), as stored."""
        n = self.lens[b] if n is None else n
        t = getattr(self, name)
        at = torch.arange(n, device=t.device)
        pages = self.table[b].long()[at // self.page]
        raw = t.view(torch.uint8) if t.dtype == E4M3 else t
        x = raw[pages, :, at % self.page].transpose(0, 1)
        return x.view(E4M3) if t.dtype == E4M3 else x


def queries(seed, B, H, N, d, dtype=torch.bfloat16, scale=1.5, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    q = [(torch.randn(B, H, N, d, generator=g) * scale).to(dtype).to(device) for _ in range(2)]
    lam = (torch.rand(H, generator=g) * 0.8 + 0.1).to(device)
    w = (1.0 + 0.1 * torch.randn(H, 2 * d, generator=g)).to(device)
    return q[0], q[1], lam, w


def attend(c, q1, q2, lam, *, causal=True, headnorm=1, norm_w=None, eps=1e-5, lambda_init=0.0):
    """(out, out tolerance, per-sequence added weights [kv, n], their tolerance), float64.

    The tolerance of one output value, from the number formats used: logits are fp32 sums of d
    exact products taken 16 at a time (at most 2^-22 of sum |q k| a step, one for the scale and
    2^-22 for the exponential, so dx in units of log2); probabilities enter the second product as
    two bf16 numbers (2^-17 of each); that product and the running sums add n / 16 + 8 fp32 steps
    of 2^-23.  A row of o is then off by at most
        a = (1 + |lambda|) max|v| (2 (ln2 dx + 2^-22) + 2^-16 + 2 (n / 16 + 8) 2^-23),
    the norm scales it by r g (1 + max|o| / rms) with 8 fp32 roundings of its own, and the result
    is rounded to bf16 (2^-8 of its value).
    """
    B, H, N, d = q1.shape
    G = H // c.kv
    out = torch.zeros(B, H, N, 2 * d, dtype=torch.float64, device=q1.device)
    tol = torch.zeros_like(out)
    added, added_tol = [], []
    for b in range(B):
        n = c.lens[b]
        k1, k2, v = (f64(c.rows(t, b)) for t in ("k1", "k2", "v"))
        add = torch.zeros(c.kv, n, dtype=torch.float64, device=q1.device)
        add_tol = torch.zeros_like(add)
        for h in range(H):
            for i in range(N):
                pos = n - N + i
                if pos < 0:
                    continue
                seen = pos + 1 if causal else n
                maps, dx = [], 0.0
                for q, k in ((q1, k1), (q2, k2)):
                    qr, kr = f64(q[b, h, i]), k[h // G, :seen]
                    x = kr @ qr / math.sqrt(d)
                    maps.append(torch.softmax(x, 0))
                    some = kr[torch.isfinite(x)]
                    if len(some):
                        s = float((some.abs() @ qr.abs()).max()) / math.sqrt(d) * 1.4427
                        dx = max(dx, s * (d / 16 + 2) * 2.0 ** -22 + 2.0 ** -22)
                lh = float(lam[h])
                w = maps[0] - lh * maps[1]
                o = w @ v[h // G, :seen]
                rel = 2 * (math.log(2) * dx + 2.0 ** -22) + 2 * (n / 16 + 8) * 2.0 ** -23
                vmax = float(v[h // G, :seen].abs().max())
                a = (1 + abs(lh)) * vmax * (rel + 2.0 ** -16)
                add[h // G, :seen] += w.abs()
                add_tol[h // G, :seen] += (maps[0] + abs(lh) * maps[1]) * rel
                y, at = o, a
                if headnorm:
                    if headnorm == 2:
                        o = o - o.mean()
                        a = 2 * a
                    rms = float(torch.sqrt((o * o).mean() + eps))
                    gain = (f64(norm_w[h]) if norm_w is not None else 1.0) * (1 - lambda_init)
                    y = o / rms * gain if rms else o * float("nan")
                    g = float(gain.abs().max()) if norm_w is not None else abs(1 - lambda_init)
                    at = a * g / rms * (1 + float(o.abs().max()) / rms) if rms else 0.0
                out[b, h, i] = y
                tol[b, h, i] = at + y.abs() * (2.0 ** -8 + 8 * 2.0 ** -24) + 1e-30
        added.append(add)
        added_tol.append(add_tol)
    return out, tol, added, added_tol


def check(got, ref, tol, what):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    fine = torch.isfinite(ref)
    over = ((got - ref).abs() - tol)[fine]
    if over.numel():
        worst = int(over.argmax())
        assert float(over.max()) <= 0, (
            f"{what}: off by {float((got - ref).abs()[fine][worst]):.4g}, "
            f"tolerance {float(tol[fine][worst]):.4g}, value {float(ref[fine][worst]):.4g}")


def to_e4m3(x):
    """Nearest e4m3 value of float64 x: ties to even, saturating at 448, NaN stays."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6).clamp_max(448.0))) - 3)
    y = torch.round(x / step) * step
    return torch.where(torch.isnan(x), x, y.clamp(-448.0, 448.0))


def evict(c, b, keep, recent):
    """Kept positions of sequence b per head, ascending ([kv] lists), or None when it stays."""
    n = c.lens[b]
    if n <= keep:
        return None
    got = []
    for row in c.rows("weights", b).double().cpu():
        w = [math.inf if math.isnan(x) else x for x in row.tolist()]
        old = n - recent
        order = sorted(range(old), key=lambda j: (-w[j], j))[: keep - recent]
        got.append(sorted(order) + list(range(old, n)))
    return got
