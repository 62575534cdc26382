"""The packed-batch operators on the GPU against float64 references."""
import random

import pytest
import torch

from differential_attention_attn_gb300 import ops
from tests import paged_ref as R
from tests import ragged_ref as G

pytestmark = pytest.mark.gpu
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
        y, t = G.turn(x.double().transpose(0, 1), pos, freq, m, neighbours)
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
