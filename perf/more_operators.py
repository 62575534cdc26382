"""Rotary positions and the operators of a serving step over a packed ("ragged") batch, as a
training or serving program calls them: what is timed, on which sizes, and each operator's plain
form.

A packed batch holds the new tokens of B sequences behind one another: sequence b's are rows
q_start[b] .. q_start[b + 1] - 1 of tensors with T rows; rows behind q_start[B] belong to none.
They stand at the positions kv_len[b] - n + i of a paged cache of the differential-attention head
(k1, k2 [pages, kv_heads, page, d], v [pages, kv_heads, page, 2d], page table [B, max_pages]).

  rotary  turns the first `rot` channels of q1, q2, k1, k2 by their token's position (pairs of the
          two halves, or of neighbours); backward turns the gradients back.
  step    from the sequences' new tokens: lengths, pages taken from and given back to a stack of
          free ones, the page table, q_start, and each token's position and slot in the cache.
  append  rotates the packed q1, q2, k1, k2 (q to the type of the cache's keys) and writes k1, k2,
          v into the cache through the slots.
  attend  out = norm((map1 - lambda map2) V) w (1 - lambda_init) of all new tokens, causal, over
          their sequences' pages.
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
EPS = 1e-5
LAMBDA_INIT = 0.8 - 0.6 * math.exp(-0.3 * 23.0)  # layer 24
BASE = 10000.0
ORIGINAL = 4096  # positions that the unscaled frequencies were trained on
FAST, SLOW = 32.0, 1.0


def _named(name, **case):
    return dict(case, **({"name": name} if name else {}))


def _rotary(name, B, H, kv, N, d, rot, kind="bf16", pairs="half", scaling="none", factor=1.0,
            offset=0, layout="head", backward=False):
    return _named(name, op="rotary", B=B, H=H, kv=kv, N=N, d=d, rot=rot, kind=kind, pairs=pairs,
                  scaling=scaling, factor=factor, offset=offset, layout=layout, backward=backward)


def _step(name, B, page, lo, hi, chunks, n, ended, pad):
    return _named(name, op="step", B=B, page=page, min_len=lo, max_len=hi, chunks=chunks, n=n,
                  ended=ended, pad=pad)


def _append(name, B, H, kv, d, page, lo, hi, chunks, n, rot, pad=0, kind="bf16", pairs="half",
            scaling="none", factor=1.0, layout="head"):
    return _named(name, op="append", B=B, H=H, kv=kv, d=d, page=page, min_len=lo, max_len=hi,
                  chunks=chunks, n=n, rot=rot, pad=pad, kind=kind, pairs=pairs, scaling=scaling,
                  factor=factor, layout=layout)


def _attend(name, B, H, kv, d, page, lo, hi, chunks, n, pad=0, kind="bf16", layout="head", norm=1):
    return _named(name, op="attend", B=B, H=H, kv=kv, d=d, page=page, min_len=lo, max_len=hi,
                  chunks=chunks, n=n, pad=pad, kind=kind, layout=layout, norm=norm)


def listed():
    return [
        # a training step's queries and keys: this repository's 4K workload
        _rotary("rotary_train_4k", 2, 16, 16, 4096, 64, 64),
        # their gradients at the wide head, half of it rotated, context stretched fourfold
        _rotary("rotary_grads_wide", 2, 8, 8, 4096, 128, 64, pairs="neighbours", scaling="parts",
                factor=4.0, layout="token", backward=True),
        # one new token of each of a batch, far into long contexts
        _rotary("rotary_token_far", 1, 32, 8, 48, 64, 64, offset=1000003, layout="token"),
        # every decoding step's bookkeeping
        _step("step_decode", 64, 16, 17, 2000, 0, 1, 0, 0),
        # a large server's step: prompts' chunks, single tokens, sequences that have ended
        _step("step_many", 768, 16, 1600, 6000, 40, 1531, 60, 77),
        # every decoding step's new tokens
        _append("append_tokens", 64, 32, 8, 64, 16, 17, 2000, 0, 1, 64, layout="token"),
        # prompts, four query heads to a key/value head
        _append("append_prompts", 4, 32, 8, 64, 64, 3001, 4096, 4, 3001, 64),
        # the wide head, e4m3 keys, chunks between single tokens in a padded buffer
        _append("append_wide_e4m3", 20, 16, 4, 128, 32, 2049, 9000, 4, 2049, 64, pad=61,
                kind="e4m3", pairs="neighbours", scaling="linear", factor=2.0),
        # the rest of one short prompt: latency alone
        _attend("attend_short", 1, 16, 16, 64, 16, 200, 200, 1, 33),
        # a server's batch: chunks of prompts between single tokens of sequences of all ages
        _attend("attend_mixed", 24, 32, 8, 64, 16, 700, 9001, 3, 613, pad=19, norm=2),
        # the last chunk of a long document
        _attend("attend_long", 1, 32, 8, 64, 64, 32768, 32768, 1, 2048),
        # the wide head, e4m3 keys, prompts being read in
        _attend("attend_wide_e4m3", 6, 16, 4, 128, 32, 2000, 5003, 6, 1025, kind="e4m3"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


MOST_PAIRS = 32 * 2048 * 30000 * 64  # (query, key) pairs times d that an attention may cost


def draw(rng):
    op = rng.choice(["rotary", "step", "append", "attend", "attend"])
    d = rng.choice([64, 64, 128])
    kind = rng.choice(["bf16", "bf16", "e4m3"])
    layout = rng.choice(["head", "token"])
    pairs = rng.choice(["half", "neighbours"])
    scaling = rng.choice(["none", "none", "linear", "ntk", "parts"])
    factor = 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 7.5])
    rot = rng.choice([d, d, d // 2, 16, 48])
    page = 16 * rng.choice([1, 2, 3, 4, 8])
    kv = rng.choice([1, 2, 4, 5, 8, 16])
    G = rng.choice([1, 1, 2, 4, 7, 8])
    if op == "rotary":
        B = rng.choice([1, 1, 2, 3, 4])
        kind = rng.choice(["bf16", "bf16", "fp32"])
        most = (128 << 20) // (4 * B * kv * (G + 1) * d * (4 if kind == "fp32" else 2))
        return _rotary("", B, kv * G, kv, _log(rng, 1, max(1, most)), d, rot, kind, pairs, scaling,
                       factor, rng.choice([0, 0, _log(rng, 1, 1 << 20)]), layout,
                       rng.random() < 0.5)
    if op == "step":
        B = _log(rng, 1, 1024)
        n = _log(rng, 1, 2000)
        chunks = min(B, rng.choice([0, 1, 3, 10, 20]))
        hi = n + _log(rng, 16, 20000)
        return _step("", B, page, n + int((hi - n) * rng.uniform(0.0, 0.9)), hi, chunks, n,
                     int((B - chunks) * rng.choice([0.0, 0.1, 0.5])), rng.choice([0, 0, 13, 100]))
    B = _log(rng, 1, 48)
    chunks = min(B, rng.choice([0, 1, 1, 2, 4, 8]))
    pad = rng.choice([0, 0, 5, 50])
    most = (512 << 20) // (B * kv * 8 * d)  # keys that one sequence may have: 512 MB of bf16 rows
    hi = _log(rng, 16, min(32768, most))
    n = _log(rng, 1, min(hi, 4096))
    if op == "append":
        n = min(n, max(1, (24 << 20) // (max(1, chunks) * kv * (G + 2) * d)))
    else:
        n = min(n, max(1, MOST_PAIRS // (max(1, chunks) * kv * G * hi * d)))
    lo = n + int((hi - n) * rng.uniform(0.0, 1.0))
    if op == "append":
        return _append("", B, kv * G, kv, d, page, lo, hi, chunks, n, rot, pad, kind, pairs,
                       scaling, factor, layout)
    return _attend("", B, kv * G, kv, d, page, lo, hi, chunks, n, pad, kind, layout,
                   rng.choice([0, 1, 2]))


# ---- lengths --------------------------------------------------------------------------------

def _batch(case, seed=0):
    """Each sequence's length with its new tokens, and those: `chunks` of them bring between half
    of n and n, the others one (for `step`: -1 where they have ended).  In an order of the seed."""
    B, lo, hi, chunks, n = (case[k] for k in ("B", "min_len", "max_len", "chunks", "n"))
    lens = [hi - (hi - lo) * i // max(1, B - 1) for i in range(B)]
    new = [n - (n // 2) * i // max(1, chunks - 1) for i in range(chunks)] + [1] * (B - chunks)
    for i in range(case.get("ended", 0)):
        new[B - 1 - i] = -1
    random.Random(B).shuffle(new)  # which length goes with which count is the case's
    order = random.Random(seed).sample(range(B), B)
    return [lens[i] for i in order], [new[i] for i in order]


def _rows(case):
    """Rows of the packed tensors: the new tokens and the padding behind them."""
    return sum(max(0, n) for n in _batch(case)[1]) + case["pad"]


def _starts(new):
    at = [0]
    for n in new:
        at.append(at[-1] + max(0, n))
    return at


# ---- frequencies ----------------------------------------------------------------------------

def _frequencies(case):
    """Radians per position of each pair, and the factor of the rotated channels."""
    rot, scaling, factor = case["rot"], case["scaling"], case["factor"]
    base, m = BASE, 1.0
    if scaling == "ntk":
        base = BASE * factor ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "parts":  # pairs that turn often keep their frequency, slow ones are stretched
        m = 0.1 * math.log(factor) + 1.0
        for i, x in enumerate(f):
            keep = min(1.0, max(0.0, (ORIGINAL * x / (2 * math.pi) - SLOW) / (FAST - SLOW)))
            f[i] = x * (keep + (1.0 - keep) / factor)
    return f, m


# ---- inputs ---------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    def whole(values, dtype=torch.int32):
        return torch.tensor(values, dtype=dtype, device="cuda")

    s = dict(case=case)
    if "rot" in case:
        s["freq"], s["m"] = _frequencies(case)
        s["freq"] = torch.tensor(s["freq"], dtype=torch.float64, device="cuda")
    if case["op"] == "rotary":
        B, H, kv, N, d = (case[k] for k in ("B", "H", "kv", "N", "d"))
        dtype = torch.float32 if case["kind"] == "fp32" else torch.bfloat16

        def rows(heads):
            if case["layout"] == "token":
                return randn(B, N, heads, d, dtype=dtype).permute(0, 2, 1, 3)
            return randn(B, heads, N, d, dtype=dtype)

        s["x"] = [rows(h) for h in (H, H, kv, kv)]
        s["positions"] = case["offset"] + torch.arange(N, dtype=torch.int32, device="cuda")
    else:
        lens, new = _batch(case, seed)
        s.update(lens=lens, new=new)
        B, page, T = case["B"], case["page"], _rows(case)
        max_pages = -(-case["max_len"] // page)
        if case["op"] == "step":
            _prepare_step(s, g, lens, new, B, page, T, max_pages, whole)
        else:
            _prepare_packed(s, g, lens, new, B, page, T, max_pages, randn, whole)
    if own:
        from differential_attention_attn_gb300 import ops
        if "rot" in case:
            s["rotary"] = ops.RotaryTable(
                case["rot"], base=BASE, neighbours=case["pairs"] == "neighbours",
                scaling=None if case["scaling"] == "none" else case["scaling"],
                factor=case["factor"], original=ORIGINAL, fast=FAST, slow=SLOW)
        if case["op"] == "step":
            s["page_book"] = ops.PageBook(s["table"], s["kv_len"], s["held"], s["free_pages"],
                                          s["free_count"], case["page"])
        elif case["op"] != "rotary":
            s["cache"] = ops.PagedCache(s["k1"], s["k2"], s["v"], s["table"], s["kv_len"],
                                        weights=s.get("weights"))
        if case["op"] == "attend":
            need = ops.ragged_fwd_plan(s["cache"], case["H"], s["q1"].shape[0])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


def _prepare_step(s, g, lens, new, B, page, T, max_pages, whole):
    # the sequences' pages before the step, drawn from a pool with a quarter to spare
    old = [n if m < 0 else n - m for n, m in zip(lens, new)]
    held = [-(-n // page) for n in old]
    most = sum(-(-n // page) for n in lens) * 5 // 4 + 8
    order = torch.randperm(most, generator=g, device="cuda").to(torch.int32)
    inside = torch.arange(max_pages, device="cuda")[None] < whole(held)[:, None]
    # one buffer for all that a step changes, so that one copy brings the state before it back
    sizes = [B, B, 1, most, B * max_pages]
    book = torch.zeros(sum(sizes), dtype=torch.int32, device="cuda")
    kv_len, held_t, count, free, table = book.split(sizes)
    kv_len.copy_(whole(old))
    held_t.copy_(whole(held))
    used = sum(held)
    table = table.view(B, max_pages)
    table[inside] = order[:used]
    free[: most - used] = order[used:]
    count.fill_(most - used)
    s.update(book=book, before=book.clone(), kv_len=kv_len, held=held_t, free_count=count,
             free_pages=free, table=table, new_len=whole(new),
             q_start=torch.zeros(B + 1, dtype=torch.int32, device="cuda"),
             positions=torch.zeros(T, dtype=torch.int32, device="cuda"),
             slots=torch.zeros(T, dtype=torch.int64, device="cuda"))


def _prepare_packed(s, g, lens, new, B, page, T, max_pages, randn, whole):
    case = s["case"]
    H, kv, d = case["H"], case["kv"], case["d"]
    P = B * max_pages + 3
    qk = E4M3 if case["kind"] == "e4m3" else torch.bfloat16

    def pool(width, dtype):
        if case["layout"] == "token":
            return randn(P, page, kv, width, dtype=dtype).permute(0, 2, 1, 3)
        return randn(P, kv, page, width, dtype=dtype)

    starts = _starts(new)
    table = torch.randperm(P, generator=g, device="cuda")[: B * max_pages].reshape(B, max_pages)
    s.update(k1=pool(d, qk), k2=pool(d, qk), v=pool(2 * d, torch.bfloat16),
             table=table.to(torch.int32), kv_len=whole(lens), q_start=whole(starts), starts=starts)
    if case["op"] == "attend":
        # logits of standard deviation 2: maps with a few strong keys over many weak ones
        s.update(q1=randn(T, H, d, scale=2.0, dtype=qk), q2=randn(T, H, d, scale=2.0, dtype=qk),
                 lam=torch.rand(H, generator=g, device="cuda") * 0.3 + 0.6,
                 norm_w=1.0 + 0.02 * torch.randn(H, 2 * d, generator=g, device="cuda"),
                 out=torch.zeros(T, H, 2 * d, dtype=torch.bfloat16, device="cuda"))
        return
    # the projections' output, one row a token, and its parts as views
    x = randn(T, (2 * H + 4 * kv) * d)
    at = 0
    for name, heads, width in (("q1", H, d), ("q2", H, d), ("k1_new", kv, d), ("k2_new", kv, d),
                               ("v_new", kv, 2 * d)):
        s[name] = x[:, at: at + heads * width].unflatten(1, (heads, width))
        at += heads * width
    b = torch.repeat_interleave(torch.arange(B, device="cuda"), whole(new))
    i = torch.arange(starts[-1], device="cuda") - s["q_start"].long()[b]
    pos = s["kv_len"].long()[b] - whole(new).long()[b] + i
    s["positions"] = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    s["slots"] = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    s["positions"][: starts[-1]] = pos.to(torch.int32)
    s["slots"][: starts[-1]] = table[b, pos // page] * page + pos % page
    s["weights"] = torch.rand(P, kv, page, generator=g, device="cuda")
    s["q1_out"] = torch.zeros(T, H, d, dtype=torch.bfloat16, device="cuda").to(qk)
    s["q2_out"] = torch.zeros(T, H, d, dtype=torch.bfloat16, device="cuda").to(qk)


# ---- one pass -------------------------------------------------------------------------------

BOOK = ("kv_len", "held", "free_count", "free_pages", "table", "q_start", "positions", "slots")
WRITTEN = ("k1", "k2", "v", "weights", "q1_out", "q2_out")


def run(s):
    case = s["case"]
    if case["op"] == "step":
        s["book"].copy_(s["before"])  # the state before the step again
    if not own:
        return {"rotary": _plain_rotary, "step": _plain_step, "append": _plain_append,
                "attend": _plain_attend}[case["op"]](s)
    from differential_attention_attn_gb300 import ops
    if case["op"] == "rotary":
        call = ops.rotary_bwd if case["backward"] else ops.rotary
        return list(call(s["rotary"], s["x"], s["positions"]))
    if case["op"] == "step":
        ops.ragged_step(s["page_book"], s["new_len"], q_start=s["q_start"],
                        positions=s["positions"], slots=s["slots"])
        return {t: s[t] for t in BOOK}
    if case["op"] == "append":
        ops.ragged_append(s["cache"], s["k1_new"], s["k2_new"], s["v_new"], s["slots"],
                          rotary=s["rotary"], positions=s["positions"], q=(s["q1"], s["q2"]),
                          q_out=(s["q1_out"], s["q2_out"]))
        return {t: s[t] for t in WRITTEN}
    return ops.ragged_fwd(s["cache"], s["q1"], s["q2"], s["lam"], s["q_start"],
                          headnorm=case["norm"], norm_w=s["norm_w"], eps=EPS,
                          lambda_init=LAMBDA_INIT, workspace=s["workspace"], out=s["out"])


# ---- plain forms ----------------------------------------------------------------------------

def _turn(x, positions, s, sign=1.0):
    """x [..., tokens, d] in 32 bits, its first `rot` channels rotated by positions [tokens]; the
    angles in 64 bits, as far positions need."""
    case = s["case"]
    r = case["rot"]
    angle = positions.double()[:, None] * s["freq"]
    cos, sin = (torch.cos(angle) * s["m"]).float(), (torch.sin(angle) * (sign * s["m"])).float()
    x = x.float()
    a, b = (x[..., : r // 2], x[..., r // 2: r]) if case["pairs"] == "half" else \
        (x[..., 0:r:2], x[..., 1:r:2])
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.cat((a, b), -1) if case["pairs"] == "half" else \
        torch.stack((a, b), -1).flatten(-2)
    return torch.cat((turned, x[..., r:]), -1)


def _plain_rotary(s):
    sign = -1.0 if s["case"]["backward"] else 1.0
    return [_turn(x, s["positions"], s, sign).to(x.dtype) for x in s["x"]]


def _plain_step(s):
    case, page = s["case"], s["case"]["page"]
    new, held, kv_len, table = s["new_len"].long(), s["held"].long(), s["kv_len"], s["table"]
    lens = torch.where(new < 0, 0, kv_len.long() + new)
    need = (lens + page - 1) // page
    take, give = (need - held).clamp_min(0), (held - need).clamp_min(0)
    at = torch.arange(table.shape[1], device="cuda")
    # pages given back: on top of the stack, by sequence and place
    back = (at >= need[:, None]) & (at < held[:, None])
    place = give.cumsum(0) - give
    k = torch.where(back, s["free_count"].long() + place[:, None] + at - need[:, None], 0)
    last = s["free_pages"].shape[0]
    padded = torch.cat((s["free_pages"], s["free_pages"][:1]))  # one place more, for the others
    padded[torch.where(back, k, last)] = table
    s["free_pages"].copy_(padded[:last])
    # pages taken: from the top down
    count = s["free_count"].long() + give.sum()
    want = (at >= held[:, None]) & (at < need[:, None])
    place = take.cumsum(0) - take
    k = torch.where(want, count - 1 - place[:, None] - (at - held[:, None]), 0)
    table.copy_(torch.where(want, s["free_pages"][k], table))
    s["free_count"].copy_(count - take.sum())
    s["held"].copy_(need)
    kv_len.copy_(lens)
    n = new.clamp_min(0)
    ends = n.cumsum(0)
    s["q_start"][0] = 0
    s["q_start"][1:] = ends
    # each packed row's sequence, position and slot
    row = torch.arange(s["slots"].shape[0], device="cuda")
    b = torch.searchsorted(ends, row, right=True)
    real = b < case["B"]
    b = b.clamp_max(case["B"] - 1)
    pos = lens[b] - ends[b] + row
    pos = torch.where(real, pos, -1)
    page_of = table[b, (pos // page).clamp_min(0)].long()
    s["positions"].copy_(pos)
    s["slots"].copy_(torch.where(real, page_of * page + pos % page, -1))
    return {t: s[t] for t in BOOK}


def _bits(t):
    return t.view(torch.uint8) if t.dtype == E4M3 else t


def _to_type(x, dtype):
    return x.clamp(-448.0, 448.0).to(dtype) if dtype == E4M3 else x.to(dtype)


def _plain_append(s):
    case, page, n = s["case"], s["case"]["page"], s["starts"][-1]
    pos, slots = s["positions"][:n], s["slots"][:n]

    def turned(name):  # [tokens, heads, d]
        return _turn(s[name][:n].transpose(0, 1), pos, s).transpose(0, 1)

    for name in ("q1", "q2"):
        out = s[name + "_out"]
        _bits(out)[:n] = _bits(_to_type(turned(name), out.dtype))
    where, slot = slots // page, slots % page
    for name in ("k1", "k2"):
        _bits(s[name])[where, :, slot] = _bits(_to_type(turned(name + "_new"), s[name].dtype))
    s["v"][where, :, slot] = s["v_new"][:n]
    s["weights"][where, :, slot] = 0.0
    return {t: s[t] for t in WRITTEN}


def _gather(pool, pages):
    """[kv, len(pages) * page, width] of a pool."""
    x = _bits(pool)[pages].transpose(0, 1)
    return x.reshape(x.shape[0], -1, x.shape[3]).view(pool.dtype)


def _plain_attend(s):
    case, page = s["case"], s["case"]["page"]
    H, kv, d = case["H"], case["kv"], case["d"]
    G = H // kv
    lam = s["lam"].reshape(kv, G, 1, 1)
    for b in range(case["B"]):
        L, start, end = s["lens"][b], s["starts"][b], s["starts"][b + 1]
        pages = s["table"][b, : -(-L // page)].long()
        k = [_gather(s[t], pages)[:, :L].float().transpose(1, 2) for t in ("k1", "k2")]
        v = _gather(s["v"], pages)[:, :L].float()
        j = torch.arange(L, device="cuda")
        rows = max(1, (1 << 28) // (H * L))  # tokens whose maps are held at a time
        for t in range(start, end, rows):
            u = min(end, t + rows)
            last = L - (end - start) + torch.arange(t - start, u - start, device="cuda")
            see = j <= last[:, None]

            def softmax(q, k):
                q = q[t:u].float().reshape(u - t, kv, G, d).permute(1, 2, 0, 3)
                x = (q.reshape(kv, G * (u - t), d) @ k * d ** -0.5).reshape(kv, G, u - t, L)
                x = torch.where(see, x, -math.inf)
                p = torch.exp(x - x.amax(-1, keepdim=True))
                return p / p.sum(-1, keepdim=True)

            w = softmax(s["q1"], k[0]) - lam * softmax(s["q2"], k[1])
            o = (w.reshape(kv, G * (u - t), L) @ v).reshape(H, u - t, 2 * d)
            if case["norm"]:
                if case["norm"] == 2:
                    o = o - o.mean(-1, keepdim=True)
                o = o / torch.sqrt(o.square().mean(-1, keepdim=True) + EPS)
                o = o * s["norm_w"][:, None] * (1.0 - LAMBDA_INIT)
            s["out"][t:u] = o.transpose(0, 1).to(torch.bfloat16)
    return s["out"]


# ---- the work that cannot be left out -------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "rotary":
        rows = case["B"] * case["N"] * 2 * (case["H"] + case["kv"])
        size = 4 if case["kind"] == "fp32" else 2
        return {"bytes": 2 * rows * case["d"] * size + 4 * case["N"],
                "flops": 3 * rows * case["rot"]}
    lens, new = _batch(case)
    T = _rows(case)
    if op == "step":
        page = case["page"]
        changed = touched = 0
        for n, m in zip(lens, new):
            old = n if m < 0 else n - m
            changed += -(-old // page) if m < 0 else -(-n // page) - -(-old // page)
            touched += 0 if m < 0 else -(-n // page) - old // page
        return {"bytes": 4 * (6 * case["B"] + 2 * changed + touched) + 12 * T, "flops": 0}
    n, d, H, kv = sum(new), case["d"], case["H"], case["kv"]
    qk = 1 if case["kind"] == "e4m3" else 2
    if op == "append":
        return {"bytes": n * ((2 * H + 2 * kv) * d * (2 + qk) + kv * (8 * d + 4) + 12),
                "flops": 3 * n * 2 * (H + kv) * case["rot"]}
    keys = sum(lens)
    pairs = sum(m * (L - m) + m * (m + 1) // 2 for L, m in zip(lens, new))
    return {"bytes": keys * kv * (2 * d * qk + 4 * d) + n * H * (2 * d * qk + 4 * d) + H * 4
            + 8 * H * d, "flops": 8 * d * H * pairs}


# ---- the definitions in 64 bits -------------------------------------------------------------

def _wide(t):
    return (t.float() if t.dtype == E4M3 else t).double()


def _exact_turn(x, positions, s, sign):
    """x [..., tokens, d] as complex pairs times m exp(i p f)."""
    case = s["case"]
    r = case["rot"]
    angle = sign * torch.outer(positions.double(), s["freq"])
    turn = torch.polar(torch.full_like(angle, s["m"]), angle)
    y = x.double().clone()
    if case["pairs"] == "half":
        even, odd = slice(0, r // 2), slice(r // 2, r)
    else:
        even, odd = slice(0, r, 2), slice(1, r, 2)
    z = torch.complex(y[..., even].contiguous(), y[..., odd].contiguous()) * turn
    y[..., even], y[..., odd] = z.real, z.imag
    return y


def _exact_step(s):
    """Sequence by sequence, page by page, on the host."""
    page = s["case"]["page"]
    lens, held, free = s["kv_len"].tolist(), s["held"].tolist(), s["free_pages"].tolist()
    count, table, new = int(s["free_count"]), s["table"].tolist(), s["new_len"].tolist()
    for b, n in enumerate(new):
        lens[b] = 0 if n < 0 else lens[b] + n
        for k in range(-(-lens[b] // page), held[b]):
            free[count] = table[b][k]
            count += 1
    positions, slots, q_start = [], [], [0]
    for b, n in enumerate(new):
        for k in range(held[b], -(-lens[b] // page)):
            count -= 1
            table[b][k] = free[count]
        held[b] = -(-lens[b] // page)
        for t in range(lens[b] - max(0, n), lens[b]):
            positions.append(t)
            slots.append(table[b][t // page] * page + t % page)
        q_start.append(len(slots))
    left = [-1] * (s["slots"].shape[0] - len(slots))
    got = dict(kv_len=lens, held=held, free_count=[count], free_pages=free, table=table,
               q_start=q_start, positions=positions + left, slots=slots + left)
    return {t: torch.tensor(got[t], dtype=s[t].dtype).reshape(s[t].shape) for t in BOOK}


def _to_e4m3(x):
    """The nearest e4m3 value (3 bits behind the point, ties to even, 448 the largest)."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_append(s):
    n, page = s["starts"][-1], s["case"]["page"]
    got = {t: _wide(s[t]) for t in WRITTEN}
    pos = s["positions"][:n]
    narrow = _to_e4m3 if s["case"]["kind"] == "e4m3" else (lambda x: x)
    pg, sl = s["slots"][:n] // page, s["slots"][:n] % page
    for t in ("q1", "q2"):
        got[t + "_out"][:n] = narrow(_exact_turn(s[t][:n].transpose(0, 1), pos, s, 1)
                                     .transpose(0, 1))
    for t in ("k1", "k2"):
        got[t][pg, :, sl] = narrow(_exact_turn(s[t + "_new"][:n].transpose(0, 1), pos, s, 1)
                                   .transpose(0, 1))
    got["v"][pg, :, sl] = s["v_new"][:n].double()
    got["weights"][pg, :, sl] = 0.0
    return got


def _exact_attend(s):
    case = s["case"]
    H, kv, d, page = case["H"], case["kv"], case["d"], case["page"]
    if work(case)["flops"] > 3e12:  # some 20 seconds in 64 bits
        return None
    G = H // kv
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        L, start, end = s["lens"][b], s["starts"][b], s["starts"][b + 1]
        at = torch.arange(L, device="cuda")
        pg = s["table"][b].long()[torch.div(at, page, rounding_mode="floor")]
        for h in range(kv):
            heads = slice(h * G, h * G + G)
            k1, k2, v = (_wide(_bits(s[t])[:, h][pg, at % page].view(s[t].dtype))
                         for t in ("k1", "k2", "v"))
            for t in range(start, end, 256):
                u = min(end, t + 256)
                seen = at[None] <= (L - (end - t) + torch.arange(u - t, device="cuda"))[:, None]
                m = []
                for q, k in ((s["q1"], k1), (s["q2"], k2)):
                    x = torch.einsum("thc,jc->htj", _wide(q[t:u, heads]), k) / math.sqrt(d)
                    x.masked_fill_(~seen, -math.inf)
                    m.append(torch.exp(x - torch.logsumexp(x, -1, keepdim=True)))
                w = m[0] - s["lam"][heads].double()[:, None, None] * m[1]
                out[t:u, heads] = torch.einsum("htj,jc->thc", w, v)
    if case["norm"] == 2:
        out -= out.sum(-1, keepdim=True) / (2 * d)
    if case["norm"]:
        gain = s["norm_w"].double() * (1.0 - LAMBDA_INIT)
        out = out * gain * ((out * out).sum(-1, keepdim=True) / (2 * d) + EPS).rsqrt()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        sign = -1 if case["backward"] else 1
        return [_exact_turn(x, s["positions"], s, sign) for x in s["x"]]
    return {"step": _exact_step, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)
