"""The paged key/value-cache operators of the differential-attention head, as a serving program
calls them: what is timed, on which sizes, and each operator's plain form.

A cache holds k1, k2 [pages, kv_heads, page, d] and v [pages, kv_heads, page, 2d] (or the same
shapes as views of [pages, page, kv_heads, width] storage), a page table [B, max_pages], the
sequences' lengths kv_len [B] with their newest tokens counted, and one float32 weight per key
and key/value head.  Token i of the N newest of a sequence sits at position kv_len - N + i; a
negative position is padding.

  append  writes the N newest tokens' k1, k2, v at their positions (k1 and k2 rounded to e4m3
          where the cache holds that) and sets their weights to zero.
  attend  out = norm((map1 - lambda map2) V) w (1 - lambda_init) of the N newest tokens over
          their sequence; with `weights` it also adds sum |map1 - lambda map2|, over the query
          heads that share a key/value head and the N tokens, to each key's weight.
  evict   keeps, per sequence and key/value head, the last `recent` keys and of the others those
          of the largest weights (ties: the lowest index), `keep` in all, moved to the front in
          their order; rows behind the new length stay as they were.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
EPS = 1e-5
LAMBDA_INIT = 0.8 - 0.6 * math.exp(-0.3 * 23.0)  # layer 24


def _attend(name, B, H, kv, N, d, page, lo, hi, kind="bf16", layout="head", norm=1, causal=True,
            weights=False):
    return dict(op="attend", B=B, H=H, kv=kv, N=N, d=d, page=page, min_len=lo, max_len=hi,
                kind=kind, layout=layout, norm=norm, causal=causal, weights=weights,
                **({"name": name} if name else {}))


def _append(name, B, kv, N, d, page, lo, hi, kind="bf16", layout="head"):
    return dict(op="append", B=B, kv=kv, N=N, d=d, page=page, min_len=lo, max_len=hi, kind=kind,
                layout=layout, **({"name": name} if name else {}))


def _evict(name, B, kv, d, page, lo, hi, keep, recent, kind="bf16", layout="head"):
    return dict(op="evict", B=B, kv=kv, d=d, page=page, min_len=lo, max_len=hi, keep=keep,
                recent=recent, kind=kind, layout=layout, **({"name": name} if name else {}))


def listed():
    return [
        # one user's first tokens of an answer: latency alone
        _attend("attend_one_short", 1, 16, 16, 1, 64, 16, 200, 200),
        # one long conversation, the decoding workload of this repository's benchmark, in pages
        _attend("attend_one_16k", 1, 32, 32, 1, 64, 64, 16384, 16384),
        # a server's running batch: sequences of all ages, four query heads to a key/value head
        _attend("attend_batch_ragged", 24, 32, 8, 1, 64, 16, 100, 9001, norm=2),
        # the wide head with shared key/value heads
        _attend("attend_wide_shared", 8, 16, 4, 1, 128, 32, 2000, 5003),
        # an e4m3 key cache, every head its own keys
        _attend("attend_e4m3", 16, 16, 16, 1, 64, 64, 1000, 4097, kind="e4m3"),
        # four drafted tokens and the one before them, weights kept for eviction
        _attend("attend_draft_weights", 4, 16, 4, 5, 64, 16, 300, 3001, layout="token",
                weights=True),
        # long documents in a batch, weights kept for eviction
        _attend("attend_long_weights", 8, 32, 8, 1, 64, 64, 32768, 32768, weights=True),
        # every decoding step's new token
        _append("append_token", 64, 16, 1, 64, 16, 17, 2000, layout="token"),
        # the prompts of this repository's 4K workload
        _append("append_prompts_4k", 2, 16, 4096, 64, 64, 4096, 4096),
        # prompts of different lengths, padded at the front, keys to e4m3
        _append("append_padded_e4m3", 4, 8, 2049, 128, 32, 513, 2049, kind="e4m3"),
        # a budget of 1024 keys, passed by a page or two
        _evict("evict_step", 4, 16, 64, 32, 1025, 1088, 1024, 64, kind="e4m3"),
        # a batch of long sequences cut to half
        _evict("evict_half_8k", 16, 8, 64, 64, 8000, 8192, 4096, 256),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "evict"])
    d = rng.choice([64, 64, 128])
    kind = rng.choice(["bf16", "bf16", "e4m3"])
    layout = rng.choice(["head", "token"])
    page = 16 * rng.choice([1, 2, 3, 4, 8])
    kv = rng.choice([1, 2, 4, 5, 8, 16])
    B = _log(rng, 1, 64)
    most = (512 << 20) // (B * kv * 8 * d)  # keys that one sequence may have: 512 MB of bf16 rows
    hi = _log(rng, 16, min(32768, most))
    lo = max(1, int(hi * rng.uniform(0.05, 1.0)))
    if op == "attend":
        G = rng.choice([1, 1, 2, 4, 7, 8])
        N = rng.choice([1, 1, 1, 2, 5, 8])
        return _attend("", B, kv * G, kv, N, d, page, lo, hi, kind, layout, rng.choice([0, 1, 2]),
                       rng.random() < 0.8, rng.random() < 0.4)
    if op == "append":
        return _append("", B, kv, 1 if rng.random() < 0.3 else _log(rng, 1, hi), d, page, lo, hi,
                       kind, layout)
    keep = max(1, int(hi * rng.uniform(0.25, 0.95)))
    return _evict("", B, kv, d, page, lo, hi, keep, int(keep * rng.uniform(0.0, 0.6)), kind,
                  layout)


def _lengths(case):
    """The sequences' lengths: spread evenly from min_len to max_len, the longest among them."""
    B, lo, hi = case["B"], case["min_len"], case["max_len"]
    return [hi - (hi - lo) * i // max(1, B - 1) for i in range(B)]


def _row_bytes(case):
    d = case["d"]
    return 2 * d * (1 if case["kind"] == "e4m3" else 2) + 4 * d


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, kv, d, page = case["B"], case["kv"], case["d"], case["page"]
    max_pages = -(-case["max_len"] // page)
    P = B * max_pages + 3
    qk = E4M3 if case["kind"] == "e4m3" else torch.bfloat16

    def randn(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    def pool(width, dtype):
        if case["layout"] == "token":
            return randn(P, page, kv, width, dtype=dtype).permute(0, 2, 1, 3)
        return randn(P, kv, page, width, dtype=dtype)

    order = torch.randperm(B, generator=g, device="cuda")
    s = dict(case=case, k1=pool(d, qk), k2=pool(d, qk), v=pool(2 * d, torch.bfloat16),
             table=torch.randperm(P, generator=g, device="cuda")[: B * max_pages]
             .reshape(B, max_pages).to(torch.int32),
             kv_len=torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")[order])
    # weights as earlier decoding steps leave them, a few keys with most: for attend a step or
    # two (of the size of what the call adds), for the others many
    s["weights"] = torch.rand(P, kv, page, generator=g, device="cuda").pow_(6)
    s["weights"].mul_(1.0 / case["max_len"] if case["op"] == "attend" else 20.0)
    if case["op"] == "attend":
        H, N = case["H"], case["N"]
        # logits of standard deviation 2: maps with a few strong keys over many weak ones
        s.update(q1=randn(B, H, N, d, scale=2.0, dtype=qk),
                 q2=randn(B, H, N, d, scale=2.0, dtype=qk),
                 lam=torch.rand(H, generator=g, device="cuda") * 0.3 + 0.6,
                 norm_w=1.0 + 0.02 * torch.randn(H, 2 * d, generator=g, device="cuda"))
    elif case["op"] == "append":
        N = case["N"]
        s.update(k1_new=randn(B, kv, N, d), k2_new=randn(B, kv, N, d), v_new=randn(B, kv, N, 2 * d))
    else:
        s["full_len"] = s["kv_len"].clone()
    if own:
        from differential_attention_attn_gb300 import ops
        s["cache"] = cache = ops.PagedCache(s["k1"], s["k2"], s["v"], s["table"], s["kv_len"],
                                            weights=s["weights"])
        need = 0
        if case["op"] == "attend":
            need = ops.paged_fwd_plan(cache, case["H"], case["N"], accumulate=case["weights"])
        elif case["op"] == "evict":
            need = ops.paged_evict_plan(cache, keep=case["keep"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


def run(s):
    case = s["case"]
    if own:
        from differential_attention_attn_gb300 import ops
        if case["op"] == "attend":
            out = ops.paged_fwd(s["cache"], s["q1"], s["q2"], s["lam"], causal=case["causal"],
                                headnorm=case["norm"], norm_w=s["norm_w"], eps=EPS,
                                lambda_init=LAMBDA_INIT, accumulate=case["weights"],
                                workspace=s["workspace"])
            return {"out": out, "weights": s["weights"]} if case["weights"] else {"out": out}
        if case["op"] == "append":
            ops.paged_append(s["cache"], s["k1_new"], s["k2_new"], s["v_new"])
        else:
            s["kv_len"].copy_(s["full_len"])  # the sequences have grown past the budget again
            ops.paged_evict(s["cache"], keep=case["keep"], recent=case["recent"],
                            workspace=s["workspace"])
    elif case["op"] == "attend":
        return _plain_attend(s)
    elif case["op"] == "append":
        _plain_append(s)
    else:
        s["kv_len"].copy_(s["full_len"])
        _plain_evict(s)
    got = {"k1": s["k1"], "k2": s["k2"], "v": s["v"], "weights": s["weights"]}
    return {**got, "kv_len": s["kv_len"]} if case["op"] == "evict" else got


# ---- plain forms ---------------------------------------------------------------------------

def _bits(t):
    return t.view(torch.uint8) if t.dtype == E4M3 else t


def _gather(pool, table):
    """[B, kv, max_pages * page, width] of a pool, in its own type."""
    x = _bits(pool)[table.long()].transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, *x.shape[4:]).view(pool.dtype)


def _plain_attend(s):
    case, table, kv_len = s["case"], s["table"], s["kv_len"].long()
    B, H, N, d, kv = case["B"], case["H"], case["N"], case["d"], case["kv"]
    G = H // kv
    v = _gather(s["v"], table).float()
    L = v.shape[2]
    j = torch.arange(L, device="cuda")
    pos = kv_len[:, None] - N + torch.arange(N, device="cuda")
    last = pos if case["causal"] else (kv_len[:, None] - 1).expand(B, N)
    see = (j <= last[..., None]) & (pos >= 0)[..., None]
    see = see[:, None, None]  # [B, 1, 1, N, L]

    def softmax(q, k):
        q = q.float().reshape(B, kv, G * N, d)
        x = (q @ _gather(k, table).float().transpose(2, 3) * d ** -0.5).reshape(B, kv, G, N, L)
        x = torch.where(see, x, -math.inf)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
        l = p.sum(-1, keepdim=True)
        return p / torch.where(l == 0, 1.0, l)

    lam = s["lam"].reshape(1, kv, G, 1, 1)
    w = softmax(s["q1"], s["k1"]) - lam * softmax(s["q2"], s["k2"])
    o = (w.reshape(B, kv, G * N, L) @ v).reshape(B, H, N, 2 * d)
    if case["norm"]:
        if case["norm"] == 2:
            o = o - o.mean(-1, keepdim=True)
        o = o / torch.sqrt(o.square().mean(-1, keepdim=True) + EPS)
        o = o * s["norm_w"][None, :, None] * (1.0 - LAMBDA_INIT)
    out = {"out": o.to(torch.bfloat16)}
    if case["weights"]:
        page = case["page"]
        add = w.abs().sum((2, 3)).reshape(B, kv, L // page, page).transpose(1, 2)
        s["weights"][table.long()] = s["weights"][table.long()] + add
        out["weights"] = s["weights"]
    return out


def _plain_append(s):
    case, page = s["case"], s["case"]["page"]
    N = case["N"]
    pos = s["kv_len"].long()[:, None] - N + torch.arange(N, device="cuda")  # [B, N]
    b, i = torch.nonzero(pos >= 0, as_tuple=True)
    pos = pos[b, i]
    where, slot = s["table"].long()[b, pos // page], pos % page
    for name in ("k1", "k2", "v"):  # three tensors
        pool, rows = s[name], s[name + "_new"][b, :, i]
        if pool.dtype == E4M3:
            rows = rows.float().clamp(-448.0, 448.0).to(E4M3)
        _bits(pool)[where, :, slot] = _bits(rows)
    s["weights"][where, :, slot] = 0.0


def _plain_evict(s):
    case, table, page = s["case"], s["table"].long(), s["case"]["page"]
    keep, recent, kv = case["keep"], case["recent"], case["kv"]
    kv_len = s["kv_len"].long()
    w = _gather(s["weights"], table)  # [B, kv, L]
    j = torch.arange(w.shape[2], device="cuda")
    n = kv_len[:, None, None]
    rank = torch.where(j >= n, -math.inf, torch.where(j >= n - recent, math.inf, w))
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    src = torch.sort(order[..., :keep], dim=-1).values  # [B, kv, kept]
    b = torch.arange(src.shape[0], device="cuda")[:, None, None]
    h = torch.arange(kv, device="cuda")[None, :, None]
    dst = torch.arange(src.shape[2], device="cuda").expand_as(src)
    # a sequence within the budget stays as it is: its rows are their own sources
    for name in ("k1", "k2", "v", "weights"):  # four tensors
        pool = _bits(s[name])
        pool[table[b, dst // page], h, dst % page] = pool[table[b, src // page], h, src % page]
    s["kv_len"].copy_(torch.minimum(kv_len, torch.full_like(kv_len, keep)))


# ---- the work that cannot be left out ------------------------------------------------------

def work(case):
    lens, kv, d = _lengths(case), case["kv"], case["d"]
    row = _row_bytes(case)
    if case["op"] == "attend":
        H, N, B = case["H"], case["N"], case["B"]
        qk = 1 if case["kind"] == "e4m3" else 2
        keys = sum(lens)
        nbytes = keys * kv * row + B * H * N * (2 * d * qk + 4 * d) + H * 4 + 8 * H * d
        if case["weights"]:
            nbytes += keys * kv * 8
        pairs = sum(sum(max(0, min(n, n - N + i + 1)) if case["causal"] else n * (n - N + i >= 0)
                        for i in range(N)) for n in lens)
        return {"bytes": nbytes, "flops": 8 * d * H * pairs}
    if case["op"] == "append":
        rows = sum(min(n, case["N"]) for n in lens) * kv
        return {"bytes": rows * (8 * d + row + 4), "flops": 0}
    over = [n for n in lens if n > case["keep"]]
    return {"bytes": sum(4 * n + case["keep"] * (2 * row + 4) for n in over) * kv + 8 * len(lens),
            "flops": 0}


# ---- the definitions in 64 bits ------------------------------------------------------------

def _places(s, b, n):
    """Page and slot of the first n positions of sequence b."""
    at = torch.arange(n, device="cuda")
    page = s["case"]["page"]
    return s["table"][b].long()[torch.div(at, page, rounding_mode="floor")], at % page


def _exact_attend(s):
    case = s["case"]
    B, H, N, d, kv = case["B"], case["H"], case["N"], case["d"], case["kv"]
    G = H // kv
    out = torch.zeros(B, H, N, 2 * d, dtype=torch.float64, device="cuda")
    total = s["weights"].double()
    lens = s["kv_len"].tolist()
    for b in range(B):
        n = lens[b]
        pg, sl = _places(s, b, n)
        for h in range(kv):
            heads = slice(h * G, h * G + G)
            k1, k2, v = (s[t][:, h][pg, sl].double() if s[t].dtype != E4M3 else
                         s[t].view(torch.uint8)[:, h][pg, sl].view(E4M3).double()
                         for t in ("k1", "k2", "v"))
            for i in range(N):
                at = n - N + i
                if at < 0:
                    continue
                seen = at + 1 if case["causal"] else n
                m = []
                for q, k in ((s["q1"], k1), (s["q2"], k2)):
                    x = q[b, heads, i].double() @ k[:seen].T / math.sqrt(d)
                    m.append(torch.exp(x - torch.logsumexp(x, -1, keepdim=True)))
                w = m[0] - s["lam"][heads].double()[:, None] * m[1]
                out[b, heads, i] = w @ v[:seen]
                if case["weights"]:
                    total[pg[:seen], h, sl[:seen]] += w.abs().sum(0)
    if case["norm"] == 2:
        out -= out.sum(-1, keepdim=True) / (2 * d)
    if case["norm"]:
        gain = s["norm_w"].double()[:, None] * (1.0 - LAMBDA_INIT)
        out = out * gain * ((out * out).sum(-1, keepdim=True) / (2 * d) + EPS).rsqrt()
    return {"out": out, "weights": total} if case["weights"] else {"out": out}


def _to_e4m3(x):
    """The nearest e4m3 value (3 bits behind the point, ties to even, 448 the largest)."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_append(s):
    case = s["case"]
    got = {t: (s[t].float() if s[t].dtype == E4M3 else s[t]).double() for t in ("k1", "k2", "v")}
    got["weights"] = s["weights"].double()
    lens = s["kv_len"].tolist()
    for b in range(case["B"]):
        n = lens[b]
        first = max(0, n - case["N"])
        pg, sl = (x[first:] for x in _places(s, b, n))
        for t in ("k1", "k2", "v"):
            rows = s[t + "_new"][b, :, case["N"] - (n - first):].double()
            got[t][pg, :, sl] = (_to_e4m3(rows) if s[t].dtype == E4M3 else rows).transpose(0, 1)
        got["weights"][pg, :, sl] = 0.0
    return got


def _exact_evict(s):
    case = s["case"]
    got = {t: (s[t].float() if s[t].dtype == E4M3 else s[t]).double() for t in ("k1", "k2", "v")}
    got["weights"] = s["weights"].double()
    lens = s["full_len"].tolist()
    for b in range(case["B"]):
        n, keep = lens[b], case["keep"]
        if n <= keep:
            continue
        pg, sl = _places(s, b, n)
        old = n - case["recent"]
        for h in range(case["kv"]):
            w = s["weights"][:, h][pg, sl][:old].double()
            best = torch.topk(w, min(old, keep - case["recent"]), sorted=True).values
            least = best[-1] if best.numel() else math.inf
            stay = w > least
            equal = torch.nonzero(w == least).flatten()
            stay[equal[: best.numel() - int(stay.sum())]] = True
            src = torch.cat([torch.nonzero(stay).flatten(), torch.arange(old, n, device="cuda")])
            for t in got:
                got[t][pg[:keep], h, sl[:keep]] = got[t][pg[src], h, sl[src]]
    got["kv_len"] = torch.tensor([min(n, case["keep"]) for n in lens], dtype=torch.int32)
    return got


def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "evict": _exact_evict}[case["op"]](s)
