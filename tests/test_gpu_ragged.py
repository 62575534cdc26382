"""The packed-batch operators on the GPU against float64 references."""
import math
import random

import pytest
import torch

from differential_attention_attn_gb300 import ops
from tests import paged_ref as R
from tests import ragged_ref as G

pytestmark = pytest.mark.gpu
INF = float("inf")
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
BOOK = ("kv_len", "held", "page_table", "free_pages", "free_count")


def _int(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


# ---- step -------------------------------------------------------------------------------------

class Book:
    def __init__(self, seed, lens, page, max_pages, spare, extra_held=0, room=0):
        rng = random.Random(seed)
        self.page, self.max_pages = page, max_pages
        held = [min(max_pages, -(-n // page) + (rng.random() < 0.5) * extra_held) for n in lens]
        ids = list(range(sum(held) + spare))
        rng.shuffle(ids)
        table = [[ids.pop() if k < h else -7 for k in range(max_pages)] for h in held]
        free = ids + [-9] * (sum(held) + room)
        self.lists = dict(lens=list(lens), held=held, table=table, free=free, count=len(ids))
        self.kv_len, self.held, self.page_table = _int(lens), _int(held), _int(table)
        self.free_pages, self.free_count = _int(free), _int([len(ids)])
        self.ops = ops.PageBook(self.page_table, self.kv_len, self.held, self.free_pages,
                                self.free_count, page)


def _step(book, new, N, status=True):
    B = len(new)
    q = torch.full((B + 1,), 77, dtype=torch.int32, device="cuda")
    pos = torch.full((N,), 77, dtype=torch.int32, device="cuda")
    slots = torch.full((N,), 77, dtype=torch.int64, device="cuda")
    word = _int([0])
    before = {t: getattr(book, t).clone() for t in BOOK}
    want = G.step(new, **book.lists, page=book.page, max_pages=book.max_pages, N=N)
    ops.ragged_step(book.ops, _int(new), q_start=q, positions=pos, slots=slots, status=word)
    torch.cuda.synchronize()
    assert int(word) == (ops.ERR_PAGE if want is None else 0)
    if want is None:
        want = dict(q_start=[0] * (B + 1), positions=[-1] * N, slots=[-1] * N)
        for t in BOOK:
            assert torch.equal(getattr(book, t), before[t]), t
    got = dict(q_start=q, positions=pos, slots=slots, **{t: getattr(book, t) for t in BOOK})
    for t, w in want.items():
        assert got[t].tolist() == w, t
    return want


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("B,page", [(1, 16), (7, 1), (40, 48), (1024, 16), (2300, 16)])
def test_step_random(seed, B, page):
    rng = random.Random(seed * 100 + B)
    lens = [rng.choice([0, 1, page, page - 1, rng.randint(0, 20 * page)]) for _ in range(B)]
    new = [rng.choice([0, 1, 1, -1, rng.randint(0, 4 * page)]) for _ in range(B)]
    book = Book(seed, lens, page, 30, spare=4 * B + 3, extra_held=rng.choice([0, 3]))
    want = _step(book, new, sum(max(0, n) for n in new) + rng.choice([0, 5]))
    assert "kv_len" in want or max(lens) + max(new) > 30 * page


def test_step_rows_in_a_second_kernel():
    """More rows than the first kernel writes itself, and rows of no sequence behind them."""
    book = Book(3, [5, 0, 100, 31, 900], 32, 200, spare=400)
    _step(book, [4000, 3333, 1, 0, -1], 8000)
    _step(Book(3, [5, 0, 100], 32, 200, spare=3), [4000, 1, 1], 5000)  # does not fit


@pytest.mark.parametrize("what", ["pages", "rows", "table", "capacity", "new", "held", "len", "count"])
def test_step_that_does_not_fit_changes_nothing(what):
    new, N, spare = [17, 1, -1, 3], 30, 4
    book = Book(5, [10, 16, 40, 0], 16, 5, spare=spare)
    if what == "pages":
        book.free_count.fill_(0)
        book.lists["count"] = 0
        new = [70, 1, -1, 3]
    elif what == "rows":
        N = 20
    elif what == "table":
        new = [71, 1, -1, 3]
    elif what == "capacity":
        book.lists["free"] = book.lists["free"][:book.lists["count"] + 2]
        book.free_pages = _int(book.lists["free"])
        book.ops = ops.PageBook(book.page_table, book.kv_len, book.held, book.free_pages,
                                book.free_count, 16)
    elif what == "new":
        new = [17, 1, -2, 3]
    elif what == "held":
        book.held[1] = book.lists["held"][1] = 0
    elif what == "len":
        book.kv_len[3] = book.lists["lens"][3] = -1
    elif what == "count":
        book.free_count.fill_(-1)
        book.lists["count"] = -1
    assert "kv_len" not in _step(book, new, N)


def test_step_pages_given_back_are_taken_again():
    book = Book(6, [64, 0], 16, 8, spare=0)
    want = _step(book, [-1, 60], 60)
    assert sorted(want["page_table"][1][:4]) == sorted(book.lists["table"][0][:4])


def test_step_outputs_left_out_graph_and_empty():
    book = Book(7, [3, 20], 16, 4, spare=4)
    q, new = _int([9, 9, 9]), _int([2, 1])
    ops.ragged_step(book.ops, new, q_start=q)  # compiled and loaded before the capture
    assert q.tolist() == [0, 2, 3] and book.kv_len.tolist() == [5, 21]
    pos = _int([0] * 6)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.ragged_step(book.ops, new, q_start=q, positions=pos)
    new.copy_(_int([0, 4]))
    graph.replay()
    graph.replay()
    assert pos.tolist() == [25, 26, 27, 28, -1, -1] and book.kv_len.tolist() == [5, 29]
    e = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    z = torch.empty(0, dtype=torch.int32, device="cuda")
    empty = ops.PageBook(e, z, z, z, _int([0]), 16)
    for n in (3, 5000):
        pos, q0 = _int([5] * n), _int([4])
        ops.ragged_step(empty, z, q_start=q0, positions=pos)
        assert q0.tolist() == [0] and set(pos.tolist()) == {-1}


@pytest.mark.parametrize("N", [4096, 4097])
@pytest.mark.parametrize("B", [256, 257, 1024, 1025])
def test_step_at_the_borders_of_its_launch_shapes(B, N):
    """One block or a cluster of eight, 1024 sequences at a time: from 4097 rows or 257 sequences on
    the cluster, from 1025 sequences on a second round.  The pool has only the pages that others give
    back in the same step; with one page less it does not fit."""
    rng = random.Random(B + N)
    lens = [rng.randint(1, 16) if b % 2 == 0 else rng.choice([0, 16]) for b in range(B)]
    new = [-1 if b % 2 == 0 else 1 for b in range(B)]
    taking = range(1, B, 2)
    if B % 2:  # one ends more than take: two pages
        new[1] = 17
    left = N - sum(n for n in new if n > 0)
    for b in taking:
        more = min(left, -new[b] % 16, rng.randint(0, 30))
        new[b], left = new[b] + more, left - more
    want = _step(Book(B, lens, 16, 4, spare=0), new, N)
    assert want["free_count"] == [0]
    new[B - 2 if B % 2 else B - 1] += 16  # a page more than there is
    assert "kv_len" not in _step(Book(B, lens, 16, 4, spare=0), new, N + 16)


def test_step_without_rows_that_does_not_fit():
    """Neither positions nor slots: any number of rows, but no more pages than there are."""
    for B in (3, 300):
        book = Book(8, [20] * B, 16, 6, spare=B - 1)
        before = {t: getattr(book, t).clone() for t in BOOK}
        q, word = torch.full((B + 1,), 77, dtype=torch.int32, device="cuda"), _int([0])
        ops.ragged_step(book.ops, _int([13] * B), q_start=q, status=word)  # a page each
        torch.cuda.synchronize()
        assert int(word) == ops.ERR_PAGE and q.tolist() == [0] * (B + 1)
        for t in BOOK:
            assert torch.equal(getattr(book, t), before[t]), t
        word.zero_()
        ops.ragged_step(book.ops, _int([13] * (B - 1) + [12]), q_start=q, status=word)
        torch.cuda.synchronize()
        assert int(word) == 0 and book.kv_len.tolist() == [33] * (B - 1) + [32]
        assert q.tolist() == [13 * b for b in range(B)] + [13 * B - 1] and int(book.free_count) == 0


# ---- append -----------------------------------------------------------------------------------

def _packed(seed, T, heads_widths, layout="packed", scale=1.0):
    """Tensors [T, heads, width], all in one row a token ("packed") or each for itself."""
    g = torch.Generator().manual_seed(seed)
    if layout == "packed":
        x = (torch.randn(T, sum(h * w for h, w in heads_widths), generator=g) * scale).to(BF16).cuda()
        out, at = [], 0
        for h, w in heads_widths:
            out.append(x[:, at: at + h * w].unflatten(1, (h, w)))
            at += h * w
        return out
    if layout == "head":
        return [(torch.randn(h, T, w, generator=g) * scale).to(BF16).cuda().transpose(0, 1)
                for h, w in heads_widths]
    return [(torch.randn(T, h, w, generator=g) * scale).to(BF16).cuda() for h, w in heads_widths]


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (128, 32), (64, 0)])
@pytest.mark.parametrize("layout,pool,neighbours", [("packed", "token", False), ("head", "head", True),
                                                    ("plain", "head", False)])
@pytest.mark.parametrize("T", [1, 5, 333])
def test_append(dtype, d, rot, layout, pool, neighbours, T):
    H, kv, page = 6, 2, 16
    c = R.Cache(1, lens=[400], kv=kv, d=d, page=page, dtype=dtype, layout=pool, weights=True, fill=3.0)
    q1, q2, k1, k2, v = _packed(2, T, [(H, d), (H, d), (kv, d), (kv, d), (kv, 2 * d)], layout, 30.0)
    g = torch.Generator().manual_seed(3)
    P = c.k1.shape[0]
    slots = torch.randperm(P * page, generator=g)[:T].cuda()
    pos = torch.randint(0, 100000, (T,), dtype=torch.int32, generator=g).cuda()
    if T > 4:
        slots[3] = -1
    names = ("k1", "k2", "v", "weights")
    want = {t: R.f64(getattr(c, t)).clone() for t in names}
    tol = {t: torch.zeros_like(want[t]) for t in names}
    table = ops.RotaryTable(rot, neighbours=neighbours) if rot else None
    freq, m = G.frequencies(rot) if rot else (torch.zeros(0, dtype=torch.float64), 1.0)

    def turned(x, to):
        y, t = G.turn(x.double().transpose(0, 1), pos, freq, m, neighbours,
                      short=dtype == BF16)
        y, t = y.transpose(0, 1), t.transpose(0, 1)
        if to == E4M3:
            y = y.clamp(-448.0, 448.0)
        return y, (G.rounded(y, t, to) if rot or to == E4M3 else t)

    live = slots >= 0
    pg, sl = slots[live] // page, slots[live] % page
    for t, x in (("k1", k1), ("k2", k2)):
        y, a = turned(x, dtype)
        want[t][pg, :, sl], tol[t][pg, :, sl] = y[live], a[live]
    want["v"][pg, :, sl] = v[live].double()
    want["weights"][pg, :, sl] = 0
    outs = [torch.full((T, H, d), 5.0, device="cuda").to(dtype) for _ in range(2)]
    word = _int([0])
    got = ops.ragged_append(c.ops_cache(), k1, k2, v, slots, rotary=table, positions=pos, q=(q1, q2),
                            q_out=outs, status=word)
    torch.cuda.synchronize()
    assert int(word) == 0 and got is outs
    for t in names:
        assert float(((R.f64(getattr(c, t)) - want[t]).abs() - tol[t]).max()) <= 0, t
    for q, o in zip((q1, q2), outs):
        y, a = turned(q, dtype)
        assert float(((R.f64(o) - y).abs() - a)[live].max()) <= 0
        assert torch.all(R.f64(o)[~live] == 5.0)


def test_append_many_tokens_without_queries_and_in_place():
    c = R.Cache(4, lens=[6000], kv=5, d=64, page=48, fill=0.0)
    k1, k2, v = _packed(5, 6000, [(5, 64), (5, 64), (5, 128)])
    at = torch.arange(6000, device="cuda")
    slots = c.table[0].long()[at // 48] * 48 + at % 48
    ops.ragged_append(c.ops_cache(), k1, k2, v, slots)
    for t, x in (("k1", k1), ("k2", k2), ("v", v)):
        assert torch.equal(c.rows(t, 0), x.transpose(0, 1))
    table = ops.RotaryTable(64)
    q = _packed(6, 6000, [(20, 64), (20, 64)])
    pos = at.to(torch.int32)
    want = ops.ragged_append(c.ops_cache(), k1, k2, v, slots, rotary=table, positions=pos, q=q)
    assert torch.equal(want[0], ops.rotary(table, [q[0].transpose(0, 1)[None]], pos)[0][0]
                       .transpose(0, 1))
    ops.ragged_append(c.ops_cache(), k1, k2, v, slots, rotary=table, positions=pos, q=q, q_out=q)
    assert torch.equal(q[0], want[0]) and torch.equal(q[1], want[1])


@pytest.mark.parametrize("bad", [-2, 1 << 20, -(1 << 40), 1 << 40])
def test_append_bad_slot(bad):
    c = R.Cache(7, lens=[40], kv=2, d=64, page=16, fill=0.0)
    k1, k2, v = _packed(8, 3, [(2, 64), (2, 64), (2, 128)])
    slots = torch.tensor([5, bad, 9], device="cuda")
    word = _int([0])
    ops.ragged_append(c.ops_cache(), k1, k2, v, slots, status=word)
    torch.cuda.synchronize()
    assert int(word) == ops.ERR_PAGE
    assert torch.equal(c.k1[0, :, 5], k1[0]) and torch.equal(c.v[0, :, 9], v[2])


def test_append_refusals():
    c = R.Cache(9, lens=[40], kv=2, d=64, page=16, fill=0.0)
    cache = c.ops_cache()
    k1, k2, v = _packed(8, 3, [(2, 64), (2, 64), (2, 128)])
    q = _packed(8, 3, [(4, 64), (4, 64)])
    slots, pos = torch.zeros(3, dtype=torch.int64, device="cuda"), _int([0, 0, 0])
    table = ops.RotaryTable(64)
    call = lambda *a, **k: ops.ragged_append(cache, *a, **k)
    for a, k in (((k1, k2, v, slots.int()), {}), ((k1, k2, v, slots[:2]), {}),
                 ((k1[:2], k2, v, slots), {}), ((k1, k2, k1, slots), {}),
                 ((k1.float(), k2, v, slots), {}), ((k1, k2, v, slots), dict(rotary=table)),
                 ((k1, k2, v, slots), dict(q=(q[0], q[1][:2]))),
                 ((k1, k2, v, slots), dict(q=q, q_out=[x.to(E4M3) for x in q])),
                 ((k1, k2, v, slots.cpu()), {}), ((k1.transpose(1, 2), k2, v, slots), {})):
        with pytest.raises(ValueError):
            call(*a, **k)
    with pytest.raises(ops.DiffAttnError):
        call(k1, k2, v, slots, rotary=ops.RotaryTable(128), positions=pos)
    with pytest.raises(ops.DiffAttnError):
        call(k1, k2, v, slots, q=[x[:, :3].contiguous() for x in q])  # 3 heads over 2
    with pytest.raises(ops.DiffAttnError):
        call(k1, k2, v, slots, q=q, q_out=[q[0], q[0].transpose(0, 0).as_strided((3, 4, 64), (256, 63, 1))])


# ---- attention --------------------------------------------------------------------------------

LI = 0.5


def _queries(seed, T, H, d, dtype, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    q = [(torch.randn(T, H, d, generator=g) * scale).to(dtype).cuda() for _ in range(2)]
    lam = (torch.rand(H, generator=g) * 0.8 + 0.1).cuda()
    w = (1.0 + 0.1 * torch.randn(H, 2 * d, generator=g)).cuda()
    return q[0], q[1], lam, w


def _starts(new, before=0):
    at = [before]
    for n in new:
        at.append(at[-1] + n)
    return at


def _parity(c, H, new, seed=3, before=0, behind=0, causal=True, headnorm=1, scale=1.5, q=None, **kw):
    starts = _starts(new, before)
    T = starts[-1] + behind
    q1, q2, lam, w = _queries(seed, T, H, c.d, c.dtype, scale) if q is None else q
    out = torch.full((T, H, 2 * c.d), 7.0, dtype=BF16, device="cuda")
    word = _int([0])
    got = ops.ragged_fwd(c.ops_cache(), q1, q2, lam, _int(starts), norm_w=w, lambda_init=LI,
                         causal=causal, headnorm=headnorm, out=out, status=word, **kw)
    torch.cuda.synchronize()
    assert int(word) == 0 and got is out
    ref, tol = G.attend(c, starts, q1, q2, lam, causal=causal, headnorm=headnorm, norm_w=w,
                        lambda_init=LI)
    R.check(out[starts[0]: starts[-1]], ref[starts[0]: starts[-1]], tol[starts[0]: starts[-1]], "out")
    assert torch.all(out[: starts[0]] == 7.0) and torch.all(out[starts[-1]:] == 7.0)
    return out


KINDS = [(64, BF16), (64, E4M3), (128, BF16), (128, E4M3)]


@pytest.mark.parametrize("d,dtype", KINDS)
@pytest.mark.parametrize("H,kv", [(2, 2), (4, 1), (6, 2), (7, 1), (64, 1)])
def test_short_ragged_batch(d, dtype, H, kv):
    """Whole items; groups that do not divide 128; rows outside the batch."""
    lens, new = [1, 0, 16, 17, 63, 64, 65, 128, 200, 5], [1, 0, 3, 17, 1, 64, 40, 1, 130, 2]
    c = R.Cache(11, lens=lens, kv=kv, d=d, page=16, dtype=dtype)
    _parity(c, H, new, before=2, behind=3)


@pytest.mark.parametrize("d,dtype", KINDS)
@pytest.mark.parametrize("page,layout", [(16, "token"), (48, "head"), (64, "head"), (128, "token"),
                                         (256, "head")])
def test_long_ragged_batch(d, dtype, page, layout):
    """Items cut by borders between shares and joined."""
    c = R.Cache(12, lens=[1500, 1, 3, 700, 65, 2049], kv=2, d=d, page=page, dtype=dtype,
                layout=layout)
    _parity(c, 4, [900, 1, 0, 1, 60, 130])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("headnorm", [0, 1, 2])
def test_norms_and_masks(d, causal, headnorm):
    c = R.Cache(13, lens=[3, 400, 0, 61, 1, 66, 2100], kv=2, d=d, page=16)
    _parity(c, 4, [3, 200, 0, 1, 1, 66, 300], causal=causal, headnorm=headnorm)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_padding_positions(d, causal):
    """More tokens than the sequence is long: rows that see no key are zero, whole tiles of them
    too."""
    c = R.Cache(14, lens=[2, 0, 40, 130], kv=1, d=d, page=16)
    out = _parity(c, 1, [5, 300, 200, 131], causal=causal)
    assert torch.all(out[:3] == 0) and torch.all(out[5:305] == 0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv,H,n,new", [(1, 1, 20001, 1), (1, 8, 12000, 33), (2, 2, 9000, 300),
                                        (8, 8, 3000, 3000)])
def test_one_sequence(d, kv, H, n, new):
    c = R.Cache(15, lens=[n], kv=kv, d=d, page=64)
    _parity(c, H, [new])


def test_many_sequences():
    """More sequences than threads that look for a share, most of them idle or single tokens."""
    rng = random.Random(2)
    lens = [rng.choice([0, 1, 20, 33]) for _ in range(1500)]
    new = [min(n, rng.choice([0, 1, 1, 5])) for n in lens]
    c = R.Cache(16, lens=lens, kv=1, d=64, page=16)
    _parity(c, 1, new)


class _Shared(R.Cache):
    """Sequences far longer than the pool: pages that are only read may stand in a table many times."""

    def __init__(self, seed, pages, page, d, dtype, tables, lens, scales=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        k = [torch.randn(pages, 1, page, d, generator=g, device="cuda") for _ in range(2)]
        if scales is not None:
            k = [x * torch.tensor(scales, device="cuda")[:, None, None, None] for x in k]
        self.k1, self.k2 = (x.to(dtype) for x in k)
        self.v = (torch.randn(pages, 1, page, 2 * d, generator=g, device="cuda") + 1).to(BF16)
        self.table, self.lens, self.kv_len = tables.to(torch.int32).cuda(), list(lens), _int(lens)
        self.B, self.kv, self.d, self.page, self.dtype = len(lens), 1, d, page, dtype

    def ops_cache(self):
        return ops.PagedCache(self.k1, self.k2, self.v, self.table, self.kv_len)


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _alike_rows(B, n, page, d, dtype):
    """B rows of n keys each, all of whose weights and values are alike, so that what sums drop adds
    up.

    With every page as often in the table, each map is the softmax over the pool.  Beside a row's
    E = 2^-8 of every p |v| (P as bf16) and of |out| (its own rounding), a product with V drops at
    most two steps of O, 2 * 2^-23, per 16 keys of a piece of 2^17 keys, a sum one in each of its
    2^17 / 128 tiles, and joining the pieces and parts of both rounds twice each, 2^-24."""
    pages, H, pieces = 8, 2, n // 2 ** 17 + 6
    table = torch.arange(n // page).remainder(pages).expand(B, -1).contiguous()
    c = _Shared(51, pages, page, d, dtype, table, [n] * B)
    q1, q2, _, _ = _queries(52, B, H, d, dtype, 0.7)
    lam, word = torch.tensor([0.1, 0.4], device="cuda"), _int([0])
    out = ops.ragged_fwd(c.ops_cache(), q1, q2, lam, _int(range(B + 1)), headnorm=0, status=word)
    torch.cuda.synchronize()
    assert int(word) == 0
    v, o, tol = R.f64(c.v).reshape(-1, 2 * d), 0.0, 0.0
    for q, k, w in ((q1, c.k1, torch.ones_like(lam)), (q2, c.k2, -lam)):
        q, k = R.f64(q), R.f64(k).reshape(-1, d)
        x = q @ k.T / math.sqrt(d)
        p = torch.softmax(x, -1)
        dx = (q.abs() @ k.abs().T).amax(-1) / math.sqrt(d) * 1.4427 * (d / 16 + 2) * 2.0 ** -22
        rel = 2 * (math.log(2) * dx + 2.0 ** -21) + 2 * (2 ** 13 + 2 ** 10 + pieces) * 2.0 ** -23 + 2.0 ** -8
        o = o + w.double()[:, None] * (p @ v)
        tol = tol + w.double().abs()[:, None] * (p @ v.abs()) * rel[..., None]
    R.check(out, o, tol * 1.01 + o.abs() * 2.0 ** -8, "out")


@pytest.mark.parametrize("d,dtype", KINDS)
@pytest.mark.parametrize("fewer", [0, 2])
def test_rows_of_millions_of_keys(d, dtype, fewer):
    """As many rows as SMs (each item whole) or a few less (all cut)."""
    _alike_rows(_sms() - fewer, 2 ** 23, 4096, d, dtype)


@pytest.mark.parametrize("d", [64, 128])
def test_items_that_take_longer_than_a_wait(d):
    """Some 2.6 million key tiles in each item, about three seconds: every wait is for a piece."""
    _alike_rows(_sms() if d == 64 else _sms() // 2, 5 * 2 ** 26, 65536, d, BF16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("alike", [True, False])
@pytest.mark.parametrize("headnorm", [0, 2])
def test_long_ranges_in_pieces(d, alike, headnorm):
    """Ranges of keys that are walked in three pieces: logits that climb, fall or stay from piece to
    piece, a value that is not finite in the first piece or seen by the last token alone, whole
    items (alike) and cut ones."""
    page, pages, H, kinds = 2048, 40, 2, 5
    n = 2 * 2 ** 17 + 3 * page + 777
    lens = [n - (0 if alike else 64 * b) for b in range(kinds)]
    rng, cols = random.Random(53), -(-n // page)
    ids = [[rng.randrange(3, pages - 1) for _ in range(cols)] for _ in range(kinds)]
    ids[0].sort()
    ids[1].sort(reverse=True)
    ids[3][7] = 0    # NaN in a column that all rows see, in the first piece
    ids[4][-1] = 1   # an infinite value at the last token's row
    scales = [1.0] * 3 + [0.3 + 0.05 * i for i in range(pages - 4)] + [1.0]
    few = _Shared(54, pages, page, d, BF16, torch.tensor(ids), lens, scales)
    few.v[0, 0, 100, 9] = float("nan")
    few.v[1, 0, (lens[4] - 1) % page, 2 * d - 1] = INF
    B = _sms() + (0 if alike else 3)
    kind = [b % kinds for b in range(B)]
    c = _Shared(54, pages, page, d, BF16, torch.tensor([ids[k] for k in kind]),
                [lens[k] for k in kind], scales)
    c.v = few.v
    new = 3
    q1, q2, lam, w = _queries(55, new * kinds, H, d, BF16)
    lam = lam * 0.5
    rows = torch.tensor([new * k + i for k in kind for i in range(new)], device="cuda")
    word = _int([0])
    out = ops.ragged_fwd(c.ops_cache(), q1[rows], q2[rows], lam, _int(range(0, new * B + 1, new)),
                         norm_w=w, lambda_init=LI, headnorm=headnorm, status=word)
    torch.cuda.synchronize()
    assert int(word) == 0
    ref, tol = G.attend(few, list(range(0, new * kinds + 1, new)), q1, q2, lam, norm_w=w,
                        lambda_init=LI, headnorm=headnorm)
    R.check(out, ref[rows], tol[rows], "out")
    # a page outside the pool in the first piece: all rows of its sequences are NaN, and no other's
    c.table[::kinds, 3] = pages
    bad = ops.ragged_fwd(c.ops_cache(), q1[rows], q2[rows], lam, _int(range(0, new * B + 1, new)),
                         norm_w=w, lambda_init=LI, headnorm=headnorm, status=word)
    torch.cuda.synchronize()
    assert int(word) == ops.ERR_PAGE
    hit = torch.tensor(kind, device="cuda").repeat_interleave(new) == 0
    assert torch.isnan(bad[hit].float()).all()
    R.check(bad[~hit], ref[rows][~hit], tol[rows][~hit], "others")


@pytest.mark.parametrize("d,causal", [(64, True), (64, False), (128, True), (128, False)])
def test_long_ranges_of_several_row_tiles(d, causal):
    """Heads with two tiles of rows, so that a share walks the end of an item that another one begins
    last, after whole and cut items of its own: all of them in pieces."""
    page, pages, H, kinds, new = 2048, 20, 32, 2, 5
    lens = [2 ** 17 + 999, 2 ** 18 + 5000]
    rng, cols = random.Random(56), -(-lens[1] // page)
    few = _Shared(57, pages, page, d, BF16,
                  torch.tensor([[rng.randrange(pages) for _ in range(cols)] for _ in range(kinds)]),
                  lens)
    B = _sms() + 11
    kind = [rng.randrange(kinds) for _ in range(B)]
    c = _Shared(57, pages, page, d, BF16, few.table[kind], [lens[k] for k in kind])
    q1, q2, lam, w = _queries(58, new * kinds, H, d, BF16)
    lam = lam * 0.5
    rows = torch.tensor([new * k + i for k in kind for i in range(new)], device="cuda")
    out = ops.ragged_fwd(c.ops_cache(), q1[rows], q2[rows], lam, _int(range(0, new * B + 1, new)),
                         norm_w=w, lambda_init=LI, causal=causal)
    ref, tol = G.attend(few, [0, new, 2 * new], q1, q2, lam, norm_w=w, lambda_init=LI, causal=causal)
    R.check(out, ref[rows], tol[rows], "out")


@pytest.mark.parametrize("d", [64, 128])
def test_large_and_climbing_logits(d):
    c = R.Cache(17, lens=[1900, 130], kv=2, d=d, page=16, fill=0.0)
    for t in ("k1", "k2"):
        for b, n in enumerate(c.lens):
            pages = c.table[b].long()[torch.arange(n, device="cuda") // 16]
            x = getattr(c, t)
            ramp = torch.linspace(0.1, 6.0, n, device="cuda")[:, None, None]
            x[pages, :, torch.arange(n, device="cuda") % 16] = (
                x[pages, :, torch.arange(n, device="cuda") % 16].float() * ramp).to(BF16)
    _parity(c, 4, [700, 130], scale=4.0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("headnorm", [0, 1])
@pytest.mark.parametrize("n", [130, 2500])
def test_values_that_are_not_finite_reach_only_rows_that_see_them(d, headnorm, n):
    """Also through the join, and whatever lies behind the sequences (R.Cache fills NaN)."""
    c = R.Cache(18, lens=[n, 40], kv=2, d=d, page=16)
    new = min(n, 600)
    for k, (back, col, x) in enumerate([(1, 0, INF), (new // 2, 5, float("nan")),
                                        (new - 2, 2 * d - 1, -INF), (17, 64, float("nan"))]):
        t = n - back
        c.v[int(c.table[0, t // 16]), k % 2, t % 16, col] = x
    _parity(c, 4, [new, 40], headnorm=headnorm)


@pytest.mark.parametrize("d", [64, 128])
def test_keys_and_queries_that_are_not_finite(d):
    """A NaN in a masked key has no influence; a NaN query row is its own row's."""
    c = R.Cache(19, lens=[300], kv=1, d=d, page=16)
    t = 290
    c.k1[int(c.table[0, t // 16]), 0, t % 16, 3] = float("nan")
    q = _queries(5, 40, 2, d, BF16)
    q[0][7, 1, 0] = float("nan")
    out = _parity(c, 2, [40], q=q)
    bad = torch.isnan(out.float()).any(-1)
    assert bad[30:].all() and bad[7, 1] and int(bad[:30].sum()) == 1


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,new", [([300, 40, 9], [40, 1, 3]), ([2500, 1300], [70, 5])])
def test_rows_of_none_have_no_influence(d, lens, new):
    """Not on a bit of the others: the rows of a tile behind a sequence's last are other sequences'
    or nobody's."""
    c = R.Cache(25, lens=lens, kv=1, d=d, page=16)
    starts = _starts(new, 2)
    T = starts[-1] + 60
    q1, q2, lam, w = _queries(5, T, 2, d, BF16)
    got = []
    for x in (0.0, float("nan"), 3e4):
        for q in (q1, q2):
            q[:2], q[starts[-1]:] = x, x
        out = torch.zeros(T, 2, 2 * d, dtype=BF16, device="cuda")
        got.append(ops.ragged_fwd(c.ops_cache(), q1, q2, lam, _int(starts), norm_w=w, lambda_init=LI,
                                  out=out))
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


@pytest.mark.parametrize("d,dtype", KINDS)
def test_a_row_of_one_key_gets_its_value(d, dtype):
    """(1 - lambda) v in fp32, however near lambda is to one: a weight's rounding is in the sum too.
    Both maps' quotients and products, lambda's and the difference are 2^-24 each of (1 + lambda) |v|
    at most four in a row."""
    c = R.Cache(31, lens=[90, 1, 1, 300], kv=2, d=d, page=16, dtype=dtype)
    starts = _starts([90, 1, 1, 300])
    q1, q2, lam, _ = _queries(9, starts[-1], 4, d, dtype)
    lam = torch.tensor([0.99, 0.8, 1.003, 0.0], device="cuda")
    out = ops.ragged_fwd(c.ops_cache(), q1, q2, lam, _int(starts), headnorm=0)
    for b in range(4):
        v = R.f64(c.rows("v", b, 1))[:, 0].repeat_interleave(2, 0)
        x = lam.double()[:, None]
        y = (1 - x) * v
        tol = (1 + x) * v.abs() * 4 * 2.0 ** -24 * 1.01 + y.abs() * 2.0 ** -8
        R.check(out[starts[b]], y, tol, f"sequence {b}")


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("n", [90, 1000, 5000])
def test_rows_that_lean_on_one_key_at_d_128(dtype, n):
    """Both maps have nearly all weight on one key, anywhere, and lambda is near one: the weights that
    the values are multiplied with add up to one, so their roundings cancel as the maps do.

    With weights w_j (1 + e_j) over their sum, |e_j| <= E = 2^-8, a map's output changes by
    sum_j w_j (e_j - sum_i w_i e_i) v_j to first order, and |e_j - sum_i w_i e_i| =
    |sum_i w_i (e_j - e_i)| <= 2 E (1 - w_j).  The rest as in ragged_ref.attend."""
    d, T = 128, 24
    c = R.Cache(61, lens=[n], kv=1, d=d, page=16, dtype=dtype)
    q1, q2, lam, _ = _queries(62, T, 1, d, dtype)
    lam = torch.full((1,), 0.95, device="cuda")
    at = torch.linspace(0, n - 1, T).round().long().cuda()
    q1[:, 0], q2[:, 0] = (R.f64(c.rows(t, 0))[0][at].mul(1.2).to(dtype) for t in ("k1", "k2"))
    out = ops.ragged_fwd(c.ops_cache(), q1, q2, lam, _int([0, T]), headnorm=0, causal=False)
    v, o, tol = R.f64(c.rows("v", 0))[0], 0.0, 0.0
    for q, t, x in ((q1, "k1", 1.0), (q2, "k2", -0.95)):
        q, k = R.f64(q)[:, 0], R.f64(c.rows(t, 0))[0]
        w = torch.softmax(q @ k.T / math.sqrt(d), -1)
        assert float(w.gather(1, at[:, None]).min()) > 0.9
        dx = (q.abs() @ k.abs().T).amax(-1, keepdim=True) / math.sqrt(d) * 1.4427 * (d / 16 + 2) * 2.0 ** -22
        rel = 2 * (math.log(2) * dx + 2.0 ** -21) + 2 * (n / 16 + 8) * 2.0 ** -23
        o = o + x * (w @ v)
        tol = tol + abs(x) * ((w * (1 - w)) @ v.abs() * 2 * 2.0 ** -8 + (w @ v.abs()) * rel)
    R.check(out[:, 0], o, tol * 1.02 + o.abs() * 2.0 ** -8, "out")


@pytest.mark.parametrize("d", [64, 128])
def test_strided_queries_and_output(d):
    c = R.Cache(20, lens=[500, 90], kv=2, d=d, page=32)  # NaN behind the sequences
    starts = [0, 70, 90]
    q1, q2, lam, w = _queries(6, 90, 4, d, BF16)
    want = ops.ragged_fwd(c.ops_cache(), q1, q2, lam, _int(starts), norm_w=w, lambda_init=LI)
    wide = torch.zeros(90, 4, 3 * d, dtype=BF16, device="cuda")
    wide[:, :, d: 2 * d] = q1
    heads_first = q2.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.zeros(4, 90, 2 * d, dtype=BF16, device="cuda").transpose(0, 1)
    ops.ragged_fwd(c.ops_cache(), wide[:, :, d: 2 * d], heads_first, lam, _int(starts), norm_w=w,
                   lambda_init=LI, out=out)
    assert torch.equal(out, want)


def _far_rows(T, heads, width, dtype=BF16):
    """[T, heads, width] with 2^31 elements from token to token."""
    x = torch.empty((T - 1) * 2 ** 31 + heads * width, dtype=dtype, device="cuda")
    return x.as_strided((T, heads, width), (2 ** 31, width, 1))


@pytest.mark.parametrize("d", [64, 128])
def test_offsets_past_32_bits(d):
    """Pages, packed rows and outputs whose byte and element offsets do not fit 32 bits."""
    page, H, T, n = 64, 2, 3, 150
    P = 2 ** 32 // (page * 2 * d)  # v: 2^32 elements
    pools = [torch.empty(P, 1, page, w, dtype=BF16, device="cuda") for w in (d, d, 2 * d)]
    far = [P - 1, P - 7, P // 2 + 3]
    c = R.Cache(41, lens=[n], kv=1, d=d, page=page)
    for k, f in enumerate(far):
        for big, t in zip(pools, (c.k1, c.k2, c.v)):
            big[f] = t[int(c.table[0, k])]
    cache = ops.PagedCache(*pools, torch.tensor([far], dtype=torch.int32, device="cuda"), c.kv_len)
    new = _packed(42, T, [(1, d), (1, d), (1, 2 * d)], "plain")
    rows = [_far_rows(T, 1, w) for w in (d, d, 2 * d)]
    slots = torch.empty(T, dtype=torch.int64, device="cuda")
    for i in range(T):  # the last three tokens: in both caches
        at = n - T + i
        slots[i] = far[at // page] * page + at % page
        for x, y, t in zip(rows, new, (c.k1, c.k2, c.v)):
            x[i] = y[i]
            t[int(c.table[0, at // page]), :, at % page] = y[i]
    q1, q2, lam, w = _queries(43, T, H, d, BF16)
    q_far, q_out = [_far_rows(T, H, d) for _ in range(2)], [_far_rows(T, H, d) for _ in range(2)]
    for x, y in zip(q_far, (q1, q2)):
        x.copy_(y)
    ops.ragged_append(cache, *rows, slots, q=q_far, q_out=q_out)
    assert torch.equal(q_out[0], q1) and torch.equal(q_out[1], q2)
    out = ops.ragged_fwd(cache, *q_out, lam, _int([0, T]), norm_w=w, lambda_init=LI,
                         out=_far_rows(T, H, 2 * d))
    ref, tol = G.attend(c, [0, T], q1, q2, lam, norm_w=w, lambda_init=LI)
    R.check(out, ref, tol, "out")


@pytest.mark.parametrize("d", [64, 128])
def test_two_streams_at_once(d):
    """Calls that run side by side, each with a workspace of its own."""
    calls = []
    for seed, lens, new in ((44, [3000, 70, 900], [200, 1, 33]), (45, [500, 2500], [130, 7])):
        c = R.Cache(seed, lens=lens, kv=2, d=d, page=16)
        starts = _starts(new)
        q1, q2, lam, w = _queries(seed, starts[-1], 4, d, BF16)
        cache, at = c.ops_cache(), _int(starts)

        def call(stream=None, cache=cache, q1=q1, q2=q2, lam=lam, w=w, at=at):
            return ops.ragged_fwd(cache, q1, q2, lam, at, norm_w=w, lambda_init=LI, stream=stream)
        calls.append((call, call(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [(call(stream), want) for _ in range(10) for call, want, stream in calls]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x, want in got)


@pytest.mark.parametrize("d", [64, 128])
def test_bad_pages_lengths_and_rows(d):
    """Reported, and nothing outside the pool or the batch is touched."""
    c = R.Cache(21, lens=[200, 300, 100, 50, 2000], kv=2, d=d, page=16, fill=0.0)
    new = [30, 40, 10, 5, 200]
    starts = _starts(new)
    q1, q2, lam, w = _queries(7, starts[-1] + 2, 4, d, BF16)
    good, tol = G.attend(c, starts, q1, q2, lam, norm_w=w, lambda_init=LI)
    for what, seq in (("page", 0), ("page", 4), ("length", 1), ("rows", 2)):
        table, kv_len, q_start = c.table.clone(), c.kv_len.clone(), _int(starts)
        if what == "page":
            table[seq, 1] = c.k1.shape[0] if seq else -5
        elif what == "length":
            kv_len[seq] = c.max_pages * 16 + 1
        else:
            q_start[3] = starts[-1] + 3  # sequence 2 ends behind the rows, sequence 3 falls
        cache = ops.PagedCache(c.k1, c.k2, c.v, table, kv_len)
        word, out = _int([0]), torch.full(good.shape, 7.0, dtype=BF16, device="cuda")
        ops.ragged_fwd(cache, q1, q2, lam, q_start, norm_w=w, lambda_init=LI, status=word, out=out)
        torch.cuda.synchronize()
        assert int(word) == ops.ERR_PAGE, what
        for b in range(5):
            mine = slice(starts[b], starts[b + 1])
            if what == "rows" and b in (2, 3):
                assert torch.all(out[mine] == 7.0)
            elif b == seq:
                assert torch.isnan(out[mine].float()).all(), (what, b)
            else:
                R.check(out[mine], good[mine], tol[mine], f"{what} {b}")
        assert torch.all(out[starts[-1]:] == 7.0)


@pytest.mark.parametrize("B", [40, 90])
def test_sequences_on_top_of_one_another(B):
    """Every other one of them is right by itself; together they have many times the rows there are
    (and could have more steps than 31 bits): reported, and nothing is written."""
    T = 200
    c = R.Cache(26, lens=[300] * B, kv=2, d=64, page=16, fill=0.0)
    q1, q2, lam, w = _queries(7, T, 4, 64, BF16)
    out, word = torch.full((T, 4, 128), 7.0, dtype=BF16, device="cuda"), _int([0])
    ops.ragged_fwd(c.ops_cache(), q1, q2, lam, _int([0, T] * (B // 2) + [0]), norm_w=w, out=out,
                   status=word)
    torch.cuda.synchronize()
    assert int(word) == ops.ERR_PAGE and torch.all(out == 7.0)


@pytest.mark.parametrize("d", [64, 128])
def test_repeated_runs_graphs_and_stale_workspaces(d):
    c = R.Cache(22, lens=[3000, 700, 1], kv=2, d=d, page=16)
    q1, q2, lam, w = _queries(8, 400, 4, d, BF16)
    cache = c.ops_cache()
    q_start = _int([0, 390, 398, 399])
    kw = dict(norm_w=w, lambda_init=LI)
    need = ops.ragged_fwd_plan(cache, 4, 400)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN bits
    out = torch.zeros(400, 4, 2 * d, dtype=BF16, device="cuda")
    want = ops.ragged_fwd(cache, q1, q2, lam, q_start, workspace=ws, out=out, **kw).clone()
    for _ in range(3):
        assert torch.equal(ops.ragged_fwd(cache, q1, q2, lam, q_start, workspace=ws, out=out, **kw),
                           want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.ragged_fwd(cache, q1, q2, lam, q_start, workspace=ws, out=out, **kw)
    for x in (c.k1, c.k2, c.v):  # finite places behind the sequences, to compare whole tensors
        x.nan_to_num_(nan=0.0)
    for lens, starts in (([3000, 700, 1], [0, 390, 398, 399]), ([128, 700, 1], [0, 3, 399, 400]),
                         ([2999, 0, 0], [0, 1, 1, 1]), ([3000, 600, 1], [5, 5, 400, 400])):
        cache.kv_len.copy_(_int(lens))
        q_start.copy_(_int(starts))
        out.zero_()
        graph.replay()
        fresh = torch.zeros_like(out)
        ops.ragged_fwd(cache, q1, q2, lam, q_start, out=fresh, **kw)
        assert torch.equal(out, fresh)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.ragged_fwd(cache, q1, q2, lam, q_start, stream=side, **kw)
    side.synchronize()
    assert torch.equal(got[5:], out[5:])


def test_fwd_refusals():
    c = R.Cache(23, lens=[400], kv=2, d=64, page=16, fill=0.0)
    cache = c.ops_cache()
    q1, q2, lam, w = _queries(9, 6, 4, 64, BF16)
    qs = _int([0, 6])
    call = lambda *a, **k: ops.ragged_fwd(cache, *a, **k)
    for a, k in (((q1, q2[:5], lam, qs), {}), ((q1.float(), q2.float(), lam, qs), {}),
                 ((q1, q2, lam[:3], qs), {}), ((q1, q2, lam, qs.long()), {}),
                 ((q1, q2, lam, _int([0, 3, 6])), {}), ((q1, q2, lam, qs), dict(norm_w=w[:, :64])),
                 ((q1, q2, lam, qs), dict(out=torch.zeros(6, 4, 64, dtype=BF16, device="cuda"))),
                 ((q1[:, :, :32], q2[:, :, :32], lam, qs), {}), ((q1[0], q2[0], lam, qs), {}),
                 ((q1, q2, lam.cpu(), qs), {}),
                 ((q1.transpose(1, 2).contiguous().transpose(1, 2), q2, lam, qs), {})):
        with pytest.raises(ValueError):
            call(*a, **k)
    with pytest.raises(ops.DiffAttnError):
        call(q1[:, :3].contiguous(), q2[:, :3].contiguous(), lam[:3].contiguous(), qs)
    with pytest.raises(ops.DiffAttnError):
        call(q1, q2, lam, qs, norm_w=torch.ones(4 * 128 + 1, device="cuda")[1:].view(4, 128))
    big = R.Cache(23, lens=[4000], kv=2, d=64, page=16, fill=0.0).ops_cache()
    need = ops.ragged_fwd_plan(big, 4, 6)
    assert need > 0
    with pytest.raises(ops.DiffAttnError):
        ops.ragged_fwd(big, q1, q2, lam, qs,
                       workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    out = ops.ragged_fwd(cache, q1[:0], q2[:0], lam, _int([0, 0]))
    assert out.shape == (0, 4, 128)


@pytest.mark.parametrize("seed", range(16))
def test_random_batches(seed):
    """Head groups, pages, lengths and counts by chance: whole, uncut and cut items."""
    rng = random.Random(seed)
    d, dtype = KINDS[seed % 4]
    kv, group = rng.choice([1, 2, 3]), rng.choice([1, 2, 3, 4, 5, 8, 16, 40])
    B = rng.choice([1, 2, 5, 20, 70, 130])
    most = rng.choice([30, 200, 1500, 5000]) if B < 20 else rng.choice([30, 300])
    lens = [rng.choice([0, 1, rng.randint(1, most), most]) for _ in range(B)]
    new = [rng.choice([0, 1, 1, rng.randint(0, 150), n]) for n in lens]
    while sum(new) * kv * group * most > 3e8:  # the reference's time
        new = [n // 2 for n in new]
    c = R.Cache(100 + seed, lens=lens, kv=kv, d=d, page=rng.choice([16, 32, 48, 80, 128]),
                dtype=dtype, layout=rng.choice(["head", "token"]))
    _parity(c, kv * group, new, before=rng.choice([0, 3]), behind=rng.choice([0, 7]),
            causal=rng.random() < 0.8, headnorm=rng.choice([0, 1, 2]))


def test_share_search_over_many_sequences():
    """More sequences than one warp looks through, long ones among them, so that items are cut."""
    lens = [1 + 37 * i % 400 for i in range(100)]
    lens[7], lens[93] = 9000, 4000
    new = [1] * 100
    new[7], new[50], new[93] = 260, 100, 33
    c = R.Cache(24, lens=lens, kv=2, d=64, page=16)
    _parity(c, 8, [min(a, b) for a, b in zip(new, lens)])


@pytest.mark.parametrize("d,dtype", KINDS)
def test_steps_of_a_server_together(d, dtype):
    """step, append and fwd over several steps of growing, idle and ending sequences, against
    sequences kept on the side: prompts in chunks, single tokens, pages handed on, one graph."""
    B, kv, H, page, T = 5, 2, 6, 16, 160
    g = torch.Generator().manual_seed(3)
    pages, max_pages = 60, 30
    qk = dtype
    pools = [torch.full((pages, kv, page, w), float("nan"), device="cuda").to(t)
             for w, t in ((d, qk), (d, qk), (2 * d, BF16))]
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    kv_len, held = _int([0] * B), _int([0] * B)
    free, count = _int(list(range(pages))), _int([pages])
    cache = ops.PagedCache(*pools, table, kv_len)
    book = ops.PageBook(table, kv_len, held, free, count, page)
    rot = ops.RotaryTable(64 if d == 64 else 96, neighbours=d == 128)
    freq, m = G.frequencies(rot.rot)
    new_len, q_start = _int([0] * B), _int([0] * (B + 1))
    positions, slots = _int([0] * T), _int([0] * T, torch.int64)
    x = [torch.zeros(T, h, w, dtype=BF16, device="cuda")
         for h, w in ((H, d), (H, d), (kv, d), (kv, d), (kv, 2 * d))]
    q_out = [torch.zeros(T, H, d, device="cuda").to(qk) for _ in range(2)]
    out = torch.zeros(T, H, 2 * d, dtype=BF16, device="cuda")
    lam, w = torch.rand(H, generator=g).cuda(), (1 + 0.1 * torch.randn(H, 2 * d, generator=g)).cuda()
    word = _int([0])
    ws = torch.empty(ops.ragged_fwd_plan(cache, H, T), dtype=torch.uint8, device="cuda")

    def step():
        ops.ragged_step(book, new_len, q_start=q_start, positions=positions, slots=slots, status=word)
        ops.ragged_append(cache, x[2], x[3], x[4], slots, rotary=rot, positions=positions,
                          q=(x[0], x[1]), q_out=q_out, status=word)
        ops.ragged_fwd(cache, q_out[0], q_out[1], lam, q_start, norm_w=w, lambda_init=LI, out=out,
                       workspace=ws, status=word)

    step()  # nothing new; loads the kernels
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    seqs = [[torch.zeros(kv, 0, w, dtype=torch.float64) for w in (d, d, 2 * d)] for _ in range(B)]
    for new in ([100, 7, 0, 1, 33], [60, 1, 50, 1, 40], [1, 1, 1, 0, -1], [0, 90, -1, 16, 20],
                [1, 1, 31, 1, 1], [-1, 1, 1, 1, 120]):
        for t in x:
            t.copy_(torch.randn(t.shape, generator=g))
        new_len.copy_(_int(new))
        if new[0] == 1:
            graph.replay()
        else:
            step()
        torch.cuda.synchronize()
        assert int(word) == 0
        starts = _starts([max(0, n) for n in new])
        assert q_start.tolist() == starts
        got, kc = out.clone(), []
        for b, n in enumerate(new):
            if n < 0:
                seqs[b] = [torch.zeros(kv, 0, w, dtype=torch.float64) for w in (d, d, 2 * d)]
                continue
            old = seqs[b][0].shape[1]
            pos = torch.arange(old, old + n)
            for i, t in enumerate((2, 3, 4)):
                rows = x[t][starts[b]: starts[b + 1]].double().cpu().transpose(0, 1)
                if i < 2:  # what the cache holds of them: turned and rounded
                    y, tol = G.turn(rows, pos, freq, m, rot.neighbours,
                                    short=qk == BF16)
                    held_rows = _cache_rows(pools[i], table[b], page, old, old + n)
                    assert float(((held_rows - y).abs() - G.rounded(y, tol, qk)).max() if n else 0) <= 0
                    rows = held_rows
                seqs[b][i] = torch.cat((seqs[b][i], rows), 1)
        # the attention against the rows that the cache holds and the queries that were written
        lens = [s[0].shape[1] for s in seqs]
        assert kv_len.tolist() == lens and held.tolist() == [-(-n // page) for n in lens]
        c = _Held(pools, table, lens, kv, d, page, qk)
        ref, tol = G.attend(c, starts, q_out[0], q_out[1], lam, norm_w=w, lambda_init=LI)
        R.check(got[: starts[-1]], ref[: starts[-1]], tol[: starts[-1]], "out")
    assert int(count) + int(held.sum()) == pages
    ids = free[: int(count)].tolist() + [p for b in range(B) for p in
                                         table[b, : int(held[b])].tolist()]
    assert sorted(ids) == list(range(pages))


def _cache_rows(pool, table, page, begin, end):
    at = torch.arange(begin, end, device="cuda")
    raw = pool.view(torch.uint8) if pool.dtype == E4M3 else pool
    x = raw[table.long()[at // page], :, at % page].transpose(0, 1).contiguous()
    return R.f64(x.view(E4M3) if pool.dtype == E4M3 else x).cpu()


class _Held(R.Cache):
    """What a paged cache holds, as paged_ref.Cache has it."""

    def __init__(self, pools, table, lens, kv, d, page, dtype):
        self.k1, self.k2, self.v = pools
        self.table, self.lens, self.kv, self.d, self.page, self.dtype = table, lens, kv, d, page, dtype
        self.B = len(lens)
