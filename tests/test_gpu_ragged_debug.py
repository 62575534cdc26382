"""The packed batch's kernels in the bounds-checked build: no check fails, and the results are the
release library's bits."""
import ctypes

import pytest
import torch

from differential_attention_attn_gb300 import build as libbuild
from differential_attention_attn_gb300 import ops
from tests import paged_ref as R

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dbg():
    return ops.bind(ctypes.CDLL(libbuild.build(debug=True)))


def _same(dbg, run):
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = run(None)
    with ops.using(dbg):
        got = run(word)
    torch.cuda.synchronize()
    assert int(word) == 0
    for a, b in zip(want, got):
        a, b = (x.view(torch.uint8) if x.dtype == E4M3 else x for x in (a, b))
        assert torch.equal(a, b)


@pytest.mark.parametrize("d,dtype", [(64, BF16), (64, E4M3), (128, BF16), (128, E4M3)])
@pytest.mark.parametrize("lens,new", [([1, 200, 0, 33], [1, 130, 0, 5]), ([3000, 700], [500, 1])])
def test_append_and_fwd(dbg, d, dtype, lens, new):
    c = R.Cache(31, lens=lens, kv=2, d=d, page=32, dtype=dtype, fill=0.0)
    g = torch.Generator().manual_seed(1)
    T, H = sum(new) + 3, 6
    x = [torch.randn(T, h, w, generator=g).to(BF16).cuda()
         for h, w in ((H, d), (H, d), (2, d), (2, d), (2, 2 * d))]
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    starts = [0]
    for b, n in enumerate(new):
        at = torch.arange(lens[b] - n, lens[b], device="cuda")
        slots[starts[-1]: starts[-1] + n] = c.table[b].long()[at // 32] * 32 + at % 32
        starts.append(starts[-1] + n)
    q_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
    lam = torch.rand(H, generator=g).cuda()
    rot = ops.RotaryTable(64)

    def run(word):
        cache = c.ops_cache()
        q = ops.ragged_append(cache, x[2], x[3], x[4], slots, rotary=rot, positions=pos,
                              q=(x[0], x[1]), status=word)
        out = torch.zeros(T, H, 2 * d, dtype=BF16, device="cuda")
        ops.ragged_fwd(cache, q[0], q[1], lam, q_start, lambda_init=0.3, out=out, status=word)
        return out, q[0][: starts[-1]], q[1][: starts[-1]], c.k1, c.k2, c.v
    _same(dbg, run)


@pytest.mark.parametrize("d", [64, 128])
def test_long_ranges_in_pieces(dbg, d):
    """Two pieces of 2^17 keys or less in each item; the pool's pages many times in each table."""
    g = torch.Generator(device="cuda").manual_seed(2)
    B, page, n = torch.cuda.get_device_properties(0).multi_processor_count + 1, 1024, 2 ** 17 + 300
    pools = [torch.randn(9, 1, page, w, generator=g, device="cuda").to(BF16) for w in (d, d, 2 * d)]
    table = torch.randint(0, 9, (B, -(-n // page)), generator=g, device="cuda", dtype=torch.int32)
    lens = n - torch.arange(B, dtype=torch.int32, device="cuda") % 250
    cache = ops.PagedCache(*pools, table, lens)
    q = [torch.randn(2 * B, 1, d, generator=g, device="cuda").to(BF16) for _ in range(2)]
    q_start = torch.arange(0, 2 * B + 1, 2, dtype=torch.int32, device="cuda")
    lam = torch.full((1,), 0.5, device="cuda")
    _same(dbg, lambda word: [ops.ragged_fwd(cache, *q, lam, q_start, lambda_init=0.3, status=word)])


@pytest.mark.parametrize("B,n", [(3, 40), (300, 30)])
def test_step(dbg, B, n):
    def run(word):
        i32 = dict(dtype=torch.int32, device="cuda")
        table = torch.full((B, 8), -1, **i32)
        kv_len, held = torch.zeros(B, **i32), torch.zeros(B, **i32)
        free, count = torch.arange(8 * B, **i32), torch.full((1,), 8 * B, **i32)
        book = ops.PageBook(table, kv_len, held, free, count, 16)
        q, pos = torch.zeros(B + 1, **i32), torch.zeros(B * n + 5, **i32)
        slots = torch.zeros(B * n + 5, dtype=torch.int64, device="cuda")
        for k in range(3):
            new = (torch.arange(B, **i32) * 7 + k) % n
            if k == 2:
                new[::3] = -1
            ops.ragged_step(book, new, q_start=q, positions=pos, slots=slots, status=word)
        return q, pos, slots, kv_len, held, table, free, count
    _same(dbg, run)


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_rotary(dbg, dtype):
    x = [torch.randn(2, h, 50, 128, device="cuda", dtype=dtype) for h in (5, 1)]
    rot = ops.RotaryTable(48, neighbours=True)
    _same(dbg, lambda word: ops.rotary(rot, x, start=5, status=word))
