"""The paged key/value-cache operators on the GPU against float64 references."""
import pytest
import torch

from differential_attention_attn_gb300 import ops
from tests import paged_ref as R

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
LI = 0.5


def _fwd(c, q1, q2, lam, w, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ops.paged_fwd(c.ops_cache(), q1, q2, lam, norm_w=w, lambda_init=LI, status=status, **kw)
    torch.cuda.synchronize()
    assert int(status) == 0
    return out


def _parity(c, H, N, seed=3, causal=True, headnorm=1, scale=1.5, **kw):
    q1, q2, lam, w = R.queries(seed, c.B, H, N, c.d, c.dtype, scale)
    out = _fwd(c, q1, q2, lam, w, causal=causal, headnorm=headnorm, **kw)
    ref, tol, _, _ = R.attend(c, q1, q2, lam, causal=causal, headnorm=headnorm, norm_w=w,
                              lambda_init=LI)
    R.check(out, ref, tol, "out")
    return out


# ---- append ---------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("N", [1, 3, 70])
def test_append_writes_the_newest_positions_and_nothing_else(dtype, d, layout, N):
    lens = [1, 70, 0, 33, 129, 2]
    c = R.Cache(1, lens=lens, kv=3, d=d, page=32, dtype=dtype, layout=layout, weights=True,
                fill=7.0)
    want = {t: R.f64(getattr(c, t)).clone() for t in ("k1", "k2", "v", "weights")}
    g = torch.Generator().manual_seed(5)
    new = {t: (torch.randn(6, N, 3, w, generator=g) * 20).to(torch.bfloat16).cuda()
           .permute(0, 2, 1, 3) for t, w in (("k1", d), ("k2", d), ("v", 2 * d))}
    for b, n in enumerate(lens):
        for i in range(N):
            t = n - N + i
            if t < 0:
                continue
            page, slot = int(c.table[b, t // 32]), t % 32
            for name in ("k1", "k2", "v"):
                row = R.f64(new[name][b, :, i])
                want[name][page, :, slot] = R.to_e4m3(row) if dtype == E4M3 and name != "v" else row
            want["weights"][page, :, slot] = 0
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.paged_append(c.ops_cache(), new["k1"], new["k2"], new["v"], status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    for t in want:
        assert torch.equal(R.f64(getattr(c, t)), want[t]), t


def test_append_many_rows():
    """More rows than the one-row-per-warp variant takes."""
    c = R.Cache(2, lens=[4100, 4033], kv=4, d=64, page=64, fill=0.0)
    g = torch.Generator().manual_seed(6)
    new = [torch.randn(2, 4, 4099, w, generator=g).to(torch.bfloat16).cuda() for w in (64, 64, 128)]
    before = [c.rows(t, 0, 1).clone() for t in ("k1", "k2", "v")]
    ops.paged_append(c.ops_cache(), *new)
    for t, x, old in zip(("k1", "k2", "v"), new, before):
        assert torch.equal(c.rows(t, 0)[:, 1:], x[0])
        assert torch.equal(c.rows(t, 0)[:, :1], old)
        assert torch.equal(c.rows(t, 1), x[1, :, 4099 - 4033:])


def test_append_rounds_to_e4m3():
    """Ties, subnormals, values at and past the largest, infinities and NaN."""
    c = R.Cache(3, lens=[1], kv=1, d=64, page=16, dtype=E4M3)
    x = torch.zeros(64)
    vals = [0.0, -0.0, 1.0625, 1.1875, 447.0, 448.0, 464.0, 466.0, -1e4, float("inf"),
            float("-inf"), float("nan"), 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11,
            -5 * 2.0 ** -10, 0.0146484375, 17.0, 19.0, 240.0, 248.0]
    x[:len(vals)] = torch.tensor(vals)
    x = x.to(torch.bfloat16)
    k = x.reshape(1, 1, 1, 64).cuda()
    ops.paged_append(c.ops_cache(), k, k, torch.zeros(1, 1, 1, 128, dtype=torch.bfloat16,
                                                      device="cuda"))
    got, want = R.f64(c.rows("k1", 0))[0, 0].cpu(), R.to_e4m3(x.double())
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~torch.isnan(want)], want[~torch.isnan(want)])


# ---- attention ------------------------------------------------------------------------------

@pytest.mark.parametrize("d,dtype", [(64, torch.bfloat16), (128, torch.bfloat16), (64, E4M3),
                                     (128, E4M3)])
@pytest.mark.parametrize("H,kv,N", [(2, 2, 1), (4, 1, 1), (6, 2, 3), (7, 1, 1), (9, 1, 1),
                                    (8, 2, 5), (3, 3, 16)])
def test_short_ragged_batch(d, dtype, H, kv, N):
    """Up to four tiles a sequence: one CTA per item."""
    c = R.Cache(11, lens=[1, 0, 16, 17, 63, 64, 65, 128, 200, 5], kv=kv, d=d, page=16,
                dtype=dtype)
    _parity(c, H, N)


@pytest.mark.parametrize("d,dtype", [(64, torch.bfloat16), (128, torch.bfloat16), (64, E4M3),
                                     (128, E4M3)])
@pytest.mark.parametrize("page,layout", [(16, "token"), (48, "head"), (64, "head"),
                                         (128, "token")])
def test_long_ragged_batch(d, dtype, page, layout):
    """Shares of all tiles: items cut by CTA boundaries and joined."""
    c = R.Cache(12, lens=[1500, 1, 0, 700, 65, 2049], kv=2, d=d, page=page, dtype=dtype,
                layout=layout)
    _parity(c, 4, 2)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("headnorm", [0, 1, 2])
@pytest.mark.parametrize("N", [1, 4])
def test_norms_and_masks(causal, headnorm, N):
    c = R.Cache(13, lens=[3, 400, 0, 61, 1, 66], kv=2, d=64, page=16)
    _parity(c, 2, N, causal=causal, headnorm=headnorm)
    c = R.Cache(14, lens=[2, 3, 1, 0, 130], kv=2, d=128, page=16)
    _parity(c, 4, N, causal=causal, headnorm=headnorm)


@pytest.mark.parametrize("kv,H,n", [(1, 1, 20001), (1, 8, 30000), (1, 20, 9000), (2, 2, 16384)])
def test_one_long_sequence(kv, H, n):
    """One item cut over many CTAs; with 20 query heads three row blocks of it."""
    c = R.Cache(15, lens=[n], kv=kv, d=64, page=64)
    _parity(c, H, 1)


def test_group_of_64_and_16_tokens():
    c = R.Cache(16, lens=[90, 10], kv=1, d=64, page=16)
    _parity(c, 64, 16)


def test_large_and_climbing_logits():
    """Logits of +-100s that grow along the keys move the reference maximum at every tile."""
    c = R.Cache(17, lens=[900, 130], kv=2, d=64, page=16, fill=0.0)
    for b in range(2):
        n = c.lens[b]
        for t in range(n):
            page, slot = int(c.table[b, t // 16]), t % 16
            c.k1[page, :, slot] *= 0.02 * t
            c.k2[page, :, slot] *= 6.0
    _parity(c, 4, 2, scale=3.0)


def test_garbage_in_unused_places_has_no_influence():
    lens = [70, 0, 200, 1, 129]
    a = R.Cache(18, lens=lens, kv=2, d=64, page=32, fill=float("nan"))
    b = R.Cache(18, lens=lens, kv=2, d=64, page=32, fill=float("inf"))
    z = R.Cache(18, lens=lens, kv=2, d=64, page=32, fill=0.0)
    outs = [_parity(c, 4, 3) for c in (a, b, z)]
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[2])


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("where", ["v", "k1", "k2"])
def test_non_finite_newest_token_reaches_only_rows_that_see_it(bad, where):
    """A masked key is left out, not multiplied by zero: earlier tokens stay finite."""
    for lens in ([66, 300], [64, 1], [3, 40]):
        c = R.Cache(19, lens=lens, kv=1, d=64, page=16)
        for b, n in enumerate(lens):
            pool = getattr(c, where)
            pool[int(c.table[b, (n - 1) // 16]), 0, (n - 1) % 16, 5] = bad
        q1, q2, lam, w = R.queries(4, 2, 2, 4, 64)
        out = _fwd(c, q1, q2, lam, w, headnorm=0).double()
        ref, tol, _, _ = R.attend(c, q1, q2, lam, headnorm=0)
        for b, n in enumerate(lens):
            R.check(out[b, :, :3], ref[b, :, :3], tol[b, :, :3], "rows before it")
            if where == "v":
                last = out[b, :, 3]
                assert bool(torch.isfinite(last[:, [4, 6]]).all())
                assert not bool(torch.isfinite(last[:, 5]).any())
            else:  # a logit of +inf or NaN makes the row NaN, one of -inf drops the key
                R.check(out[b, :, 3], ref[b, :, 3], tol[b, :, 3], "the newest row")


def test_strided_queries_and_output():
    c = R.Cache(20, lens=[300, 40], kv=2, d=64, page=16)
    q1, q2, lam, w = R.queries(7, 2, 6, 3, 64)
    v1, v2 = (q.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for q in (q1, q2))
    big = torch.full((2, 3, 6, 160), 9.0, dtype=torch.bfloat16, device="cuda")
    out = big[..., 16:144].permute(0, 2, 1, 3)
    want = _fwd(c, q1, q2, lam, w)
    got = _fwd(c, v1, v2, lam, w, out=out)
    assert got is out and torch.equal(got, want)
    assert bool((big[..., :16] == 9).all()) and bool((big[..., 144:] == 9).all())


def test_offsets_past_32_bits():
    """Pages whose byte and element offsets do not fit 32 bits."""
    page, d, P = 64, 64, 1 << 19  # v: 2^32 elements
    k1, k2 = (torch.empty(P, 1, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    v = torch.empty(P, 1, page, 2 * d, dtype=torch.bfloat16, device="cuda")
    small = R.Cache(21, lens=[150], kv=1, d=d, page=page, weights=True)
    far = [P - 1, P - 7, P // 2 + 3]
    weights = torch.zeros(P, 1, page, device="cuda")
    for k, f in enumerate(far):
        s = int(small.table[0, k])
        for big, t in ((k1, small.k1), (k2, small.k2), (v, small.v)):
            big[f] = t[s]
    table = torch.tensor([far], dtype=torch.int32, device="cuda")
    cache = ops.PagedCache(k1, k2, v, table, small.kv_len, weights=weights)
    q1, q2, lam, w = R.queries(8, 1, 2, 1, d)
    out = ops.paged_fwd(cache, q1, q2, lam, norm_w=w, lambda_init=LI, accumulate=True)
    ref, tol, add, add_tol = R.attend(small, q1, q2, lam, norm_w=w, lambda_init=LI)
    R.check(out, ref, tol, "out")
    got = torch.cat([weights[f, 0] for f in far])[:150]
    R.check(got, add[0][0], add_tol[0][0] + 2.0 ** -23, "weights")
    new = [torch.ones(1, 1, 1, x, dtype=torch.bfloat16, device="cuda") for x in (d, d, 2 * d)]
    ops.paged_append(cache, *new)
    assert bool((v[far[2], 0, 149 - 128] == 1).all()) and float(weights[far[2], 0, 21]) == 0
    weights[far[0], 0, :10] = 5.0
    rows = v[far[0], 0, 0:10].clone()
    last = v[far[2], 0, 21].clone()
    ops.paged_evict(cache, keep=11, recent=1)
    assert torch.equal(v[far[0], 0, :10], rows) and torch.equal(v[far[0], 0, 10], last)
    assert small.kv_len.tolist() == [11]


# ---- weights --------------------------------------------------------------------------------

@pytest.mark.parametrize("lens,H,kv,N,d,page,dtype", [
    ([100, 0, 1, 64, 130], 4, 2, 1, 64, 16, torch.bfloat16),
    ([3, 700, 1100], 6, 2, 3, 64, 48, torch.bfloat16),
    ([2300], 12, 1, 2, 128, 32, torch.bfloat16),
    ([1030, 33], 2, 2, 1, 64, 64, E4M3),
])
def test_accumulated_weights(lens, H, kv, N, d, page, dtype):
    c = R.Cache(31, lens=lens, kv=kv, d=d, page=page, dtype=dtype, weights=True)
    before = c.weights.clone()
    q1, q2, lam, w = R.queries(9, c.B, H, N, d, dtype)
    out = _fwd(c, q1, q2, lam, w, accumulate=True)
    ref, tol, add, add_tol = R.attend(c, q1, q2, lam, norm_w=w, lambda_init=LI)
    R.check(out, ref, tol, "out")
    after = c.weights.clone()
    touched = torch.zeros_like(before, dtype=torch.bool)
    for b, n in enumerate(lens):
        if not n:
            continue
        c.weights = before
        old = c.rows("weights", b).double()
        c.weights = after
        want = old + add[b]
        # R N fp32 additions and one to the old value
        tol_w = add_tol[b] + want.abs() * (H // kv * N + 2) * 2.0 ** -23
        R.check(c.rows("weights", b), want, tol_w, f"weights of sequence {b}")
        for t in range(n):
            touched[int(c.table[b, t // page]), :, t % page] = True
    assert torch.equal(after[~touched], before[~touched])
    # a fixed order of addition: the same bits again
    c.weights = before.clone()
    assert torch.equal(_fwd(c, q1, q2, lam, w, accumulate=True), out)
    assert torch.equal(c.weights, after)


@pytest.mark.parametrize("lens,H,kv,N,d,page,causal", [
    ([20001], 1, 1, 1, 64, 64, True),          # an item cut over every CTA
    ([9000, 0, 300], 3, 1, 1, 64, 64, True),   # a plane of three rows
    ([700, 3, 260], 10, 2, 1, 64, 16, True),   # five rows
    ([700, 1, 500], 7, 1, 2, 128, 16, False),  # fourteen rows, some see no key
    ([1300, 30], 40, 1, 1, 64, 16, True),      # two row blocks
    ([90, 10], 64, 1, 16, 64, 16, True),       # 32 row blocks
    ([70000, 100], 16, 2, 1, 64, 64, True),    # logits past what L2 holds back
])
def test_accumulated_weights_by_rows_and_parts(lens, H, kv, N, d, page, causal):
    c = R.Cache(33, lens=lens, kv=kv, d=d, page=page, weights=True)
    before = c.weights.clone()
    old = [c.rows("weights", b).double() for b in range(c.B)]
    q1, q2, lam, w = R.queries(34, c.B, H, N, d)
    lam[0] = 0.0
    out = _fwd(c, q1, q2, lam, w, accumulate=True, causal=causal)
    ref, tol, add, add_tol = R.attend(c, q1, q2, lam, norm_w=w, lambda_init=LI, causal=causal)
    R.check(out, ref, tol, "out")
    for b, n in enumerate(lens):
        if n:
            want = old[b] + add[b]
            tol_w = add_tol[b] + want.abs() * (H // kv * N + 2) * 2.0 ** -23
            R.check(c.rows("weights", b), want, tol_w, f"weights of sequence {b}")
    after = c.weights.clone()
    for _ in range(3):  # the same bits again, in memory that the call before has used
        c.weights.copy_(before)
        assert torch.equal(_fwd(c, q1, q2, lam, w, accumulate=True, causal=causal), out)
        assert torch.equal(c.weights, after)


def test_weights_of_calls_in_a_row_on_one_workspace():
    """Logits past what L2 holds back, written, read and dropped by call after call without a wait
    between them: the weights are those of the same calls one at a time."""
    d, kv, H, n = 64, 4, 16, 80000
    caches = [R.Cache(120 + k, lens=[n - k, 3000], kv=kv, d=d, page=64, weights=True, fill=0.0)
              for k in range(2)]
    ops_caches = [c.ops_cache() for c in caches]
    queries = [R.queries(122 + k, 2, H, 1, d) for k in range(2)]
    start = [c.weights.clone() for c in caches]
    need = max(ops.paged_fwd_plan(c, H, accumulate=True) for c in ops_caches)
    assert need > 16 << 20
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    results = []
    for wait in (True, False):
        for c, w0 in zip(caches, start):
            c.weights.copy_(w0)
        torch.cuda.synchronize()
        for step in range(24):
            q1, q2, lam, w = queries[step % 2]
            ops.paged_fwd(ops_caches[step % 2], q1, q2, lam, norm_w=w, accumulate=True,
                          workspace=ws)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        results.append([c.weights.clone() for c in caches])
    for x, y in zip(*results):
        assert torch.equal(x, y)


# ---- bad pages and lengths ------------------------------------------------------------------

@pytest.mark.parametrize("lens", [[100, 90, 33], [1000, 900, 33]])
@pytest.mark.parametrize("bad", [-1, 1 << 20])
def test_bad_page_is_reported_and_kept_apart(lens, bad):
    c = R.Cache(41, lens=lens, kv=2, d=64, page=16, weights=True)
    q1, q2, lam, w = R.queries(10, 3, 4, 1, 64)
    want = _fwd(c, q1, q2, lam, w)
    c.table[1, 2] = bad
    pools = {t: getattr(c, t).clone() for t in ("k1", "k2", "v", "weights")}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ops.paged_fwd(c.ops_cache(), q1, q2, lam, norm_w=w, lambda_init=LI, status=status,
                        accumulate=True)
    assert int(status) == ops.ERR_PAGE
    assert bool(torch.isnan(out[1]).all())
    assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2])
    for t in range(lens[1]):
        if t // 16 != 2:
            page, slot = int(c.table[1, t // 16]), t % 16
            assert torch.equal(c.weights[page, :, slot], pools["weights"][page, :, slot])
    status.zero_()
    lens_before = c.kv_len.clone()
    kept = {t: c.rows(t, 0).clone() for t in ("k1", "v")}
    ops.paged_evict(c.ops_cache(), keep=60, recent=4, status=status)
    assert int(status) == ops.ERR_PAGE
    assert c.kv_len.tolist() == [min(60, lens[0]), lens[1], min(60, lens[2])]
    assert lens_before.tolist() == lens
    status.zero_()
    c.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
    c.kv_len[1] = 48
    new = [torch.ones(3, 2, 20, x, dtype=torch.bfloat16, device="cuda") for x in (64, 64, 128)]
    ops.paged_append(c.ops_cache(), *new, status=status)
    assert int(status) == ops.ERR_PAGE
    assert bool((c.v[int(c.table[1, 1]), :, 12:] == 1).all())
    del kept


@pytest.mark.parametrize("bad", [-1, 161, 2 ** 31 - 1, -2 ** 31])
def test_bad_length_is_reported_and_kept_apart(bad):
    c = R.Cache(42, lens=[100, 90, 33], kv=2, d=64, page=16, weights=True, extra_pages=3)
    q1, q2, lam, w = R.queries(10, 3, 4, 2, 64)
    want = _fwd(c, q1, q2, lam, w)
    c.kv_len[1] = bad
    pools = {t: getattr(c, t).clone() for t in ("k1", "k2", "v", "weights")}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ops.paged_fwd(c.ops_cache(), q1, q2, lam, norm_w=w, lambda_init=LI, status=status)
    assert int(status) == ops.ERR_PAGE
    assert bool(torch.isnan(out[1]).all())
    assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2])
    status.zero_()
    ops.paged_evict(c.ops_cache(), keep=120, recent=4, status=status)
    assert int(status) == ops.ERR_PAGE
    new = [torch.ones(3, 2, 1, x, dtype=torch.bfloat16, device="cuda") for x in (64, 64, 128)]
    status.zero_()
    ops.paged_append(c.ops_cache(), *new, status=status)
    assert int(status) == ops.ERR_PAGE
    mine = [int(x) for x in c.table[1] if x >= 0]
    for t in pools:
        raw = getattr(c, t).view(torch.int16 if t != "weights" else torch.int32)
        old = pools[t].view(raw.dtype)
        assert torch.equal(raw[mine], old[mine]), t
    assert c.kv_len.tolist() == [100, bad, 33]


# ---- eviction -------------------------------------------------------------------------------

def _check_evict(c, keep, recent, **kw):
    before = {t: getattr(c, t).clone() for t in ("k1", "k2", "v", "weights")}
    kept = [R.evict(c, b, keep, recent) for b in range(c.B)]
    want = {t: x.view(torch.uint8).clone() if x.dtype == E4M3 else
            x.view(torch.int16).clone() if x.dtype == torch.bfloat16 else
            x.view(torch.int32).clone() for t, x in before.items()}
    for b, rows in enumerate(kept):
        if rows is None:
            continue
        for h, src in enumerate(rows):
            s = torch.tensor(src, dtype=torch.long, device="cuda")
            dst = torch.arange(len(src), device="cuda")
            tab = c.table[b].long()
            for t in want:
                want[t][tab[dst // c.page], h, dst % c.page] = \
                    want[t][tab[s // c.page], h, s % c.page].clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.paged_evict(c.ops_cache(), keep=keep, recent=recent, status=status, **kw)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert c.kv_len.tolist() == [min(n, keep) for n in c.lens]
    for t in want:
        got = getattr(c, t)
        assert torch.equal(got.view(want[t].dtype), want[t]), t
    c.lens = c.kv_len.tolist()


@pytest.mark.parametrize("keep,recent", [(0, 0), (1, 0), (1, 1), (64, 0), (64, 64), (100, 17),
                                         (1024, 100), (2999, 5), (3000, 0)])
def test_evict_keeps_the_largest_weights(keep, recent):
    c = R.Cache(51, lens=[3000, 100, 0, 65, 1025, 2048], kv=2, d=64, page=16, weights=True)
    _check_evict(c, keep, recent)


@pytest.mark.parametrize("d,dtype,layout,page", [(128, torch.bfloat16, "token", 48),
                                                 (64, E4M3, "head", 64),
                                                 (128, E4M3, "token", 16)])
def test_evict_layouts(d, dtype, layout, page):
    c = R.Cache(52, lens=[777, 300, 12], kv=3, d=d, page=page, dtype=dtype, layout=layout,
                weights=True)
    _check_evict(c, 256, 32)
    _check_evict(c, 255, 0)


def test_evict_ties_and_special_values():
    """Equal weights: the lower position stays; NaN as +infinity; -0 equals 0; negatives last."""
    c = R.Cache(53, lens=[1500, 1500, 40, 1500], kv=1, d=64, page=16, weights=True)

    def put(b, values):
        for t, x in enumerate(values):
            c.weights[int(c.table[b, t // 16]), 0, t % 16] = x

    put(0, [1.0] * 1500)
    put(1, [0.0 if t % 3 else -0.0 for t in range(1500)])
    special = [float("nan"), float("inf"), -1.0, 0.0, -0.0, 1e-45, -float("inf"), 3.0, 3.0, 3.0]
    put(2, special * 4)
    put(3, [float((t * 7919) % 13) for t in range(1500)])
    _check_evict(c, 37, 5)
    _check_evict(c, 20, 3)


def test_evict_large_cache():
    c = R.Cache(54, lens=[40000], kv=1, d=64, page=64, weights=True)
    _check_evict(c, 20000, 1000)


# ---- a run of them --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])
def test_prompt_decode_and_evict_together(dtype):
    """Prompts of different lengths, then decoding steps with eviction whenever a sequence passes
    its budget, the whole state followed by the float64 operators on the stored values."""
    B, H, kv, d, page, budget, recent = 3, 4, 2, 64, 16, 96, 24
    c = R.Cache(61, lens=[160, 160, 160], kv=kv, d=d, page=page, dtype=dtype, weights=True,
                fill=0.0)
    prompt = [70, 95, 1]
    c.kv_len.copy_(torch.tensor(prompt, dtype=torch.int32))
    cache = c.ops_cache()
    g = torch.Generator().manual_seed(62)

    def new(N):
        return [torch.randn(B, kv, N, w, generator=g).to(torch.bfloat16).cuda()
                for w in (d, d, 2 * d)]

    ops.paged_append(cache, *new(95))
    for step in range(40):
        N = 1 if step % 4 else 3
        c.kv_len.add_(N)
        c.lens = c.kv_len.tolist()
        ops.paged_append(cache, *new(N))
        q1, q2, lam, w = R.queries(100 + step, B, H, N, d, dtype)
        old = [c.rows("weights", b).double() for b in range(B)]
        ref, tol, add, add_tol = R.attend(c, q1, q2, lam, norm_w=w, lambda_init=LI)
        out = ops.paged_fwd(cache, q1, q2, lam, norm_w=w, lambda_init=LI, accumulate=True)
        R.check(out, ref, tol, f"step {step}")
        for b in range(B):
            want = old[b] + add[b]
            R.check(c.rows("weights", b), want,
                    add_tol[b] + want * (H // kv * N + 2) * 2.0 ** -23, f"weights, step {step}")
        if max(c.lens) > budget:
            _check_evict(c, budget - 8, recent)
    assert c.kv_len.tolist() != prompt


def test_captured_step_replays_with_new_lengths():
    """append, fwd with weights and evict in one CUDA graph, replayed while kv_len moves on."""
    B, H, kv, d, page = 2, 4, 2, 64, 16
    make = lambda: R.Cache(71, lens=[400, 400], kv=kv, d=d, page=page, weights=True, fill=0.0)
    a, b = make(), make()
    for c in (a, b):
        c.kv_len.copy_(torch.tensor([100, 260], dtype=torch.int32))
    q1, q2, lam, w = R.queries(72, B, H, 1, d)
    g = torch.Generator().manual_seed(73)
    steps = [[torch.randn(B, kv, 1, x, generator=g).to(torch.bfloat16).cuda()
              for x in (d, d, 2 * d)] for _ in range(6)]
    buf = [t.clone() for t in steps[0]]

    def step(cache, kv_len, new):
        kv_len.add_(1)
        ops.paged_append(cache, *new)
        out = ops.paged_fwd(cache, q1, q2, lam, norm_w=w, lambda_init=LI, accumulate=True)
        ops.paged_evict(cache, keep=262, recent=10)
        return out

    ca, cb = a.ops_cache(), b.ops_cache()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    saved = {t: getattr(a, t).clone() for t in ("k1", "k2", "v", "weights", "kv_len")}
    with torch.cuda.stream(side):
        step(ca, a.kv_len, buf)  # warm-up on the capture stream
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(ca, a.kv_len, buf)
    for t, x in saved.items():
        getattr(a, t).copy_(x)
    for new in steps:
        for dst, src in zip(buf, new):
            dst.copy_(src)
        graph.replay()
        want = step(cb, b.kv_len, new)
        assert torch.equal(out, want)
    for t in saved:
        assert torch.equal(getattr(a, t), getattr(b, t)), t
    assert b.kv_len.tolist() == [106, 262]


def test_other_stream_and_two_at_once():
    """Calls on a stream of their own, and two at once with a workspace each."""
    c = R.Cache(81, lens=[3000, 500], kv=2, d=64, page=16)
    cache = c.ops_cache()
    q1, q2, lam, w = R.queries(82, 2, 4, 1, 64)
    want = _fwd(c, q1, q2, lam, w)
    streams = [torch.cuda.Stream() for _ in range(2)]
    need = ops.paged_fwd_plan(cache, 4, 1)
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for k in range(20):
        s = streams[k % 2]
        outs.append(ops.paged_fwd(cache, q1, q2, lam, norm_w=w, lambda_init=LI, stream=s,
                                  workspace=ws[k % 2] if k < 10 else None))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_empty_calls():
    c = R.Cache(91, lens=[5], kv=2, d=64, page=16, weights=True)
    cache = c.ops_cache()
    q = torch.empty(1, 4, 0, 64, dtype=torch.bfloat16, device="cuda")
    lam = torch.ones(4, device="cuda")
    assert ops.paged_fwd(cache, q, q, lam).shape == (1, 4, 0, 128)
    k = torch.empty(1, 2, 0, 64, dtype=torch.bfloat16, device="cuda")
    ops.paged_append(cache, k, k, torch.empty(1, 2, 0, 128, dtype=torch.bfloat16, device="cuda"))
    ops.paged_evict(cache, keep=16)
    assert c.kv_len.tolist() == [5]


def test_calls_that_do_not_fit_are_refused():
    """Wrong shapes, types, devices, layouts and workspaces, also right after a good call of the
    same numbers; nothing is launched."""
    c = R.Cache(92, lens=[40, 7], kv=2, d=64, page=16, weights=True)
    cache = c.ops_cache()
    q1, q2, lam, w = R.queries(93, 2, 4, 1, 64)
    new = [torch.ones(2, 2, 1, x, dtype=torch.bfloat16, device="cuda") for x in (64, 64, 128)]
    pools = [getattr(c, t).clone() for t in ("k1", "k2", "v", "weights")]
    good = ops.paged_fwd(cache, q1, q2, lam)
    for bad in ((q1[:1], q2, lam), (q1, q2[:, :2], lam), (q1[..., :32], q2[..., :32], lam),
                (q1.float(), q2, lam), (q1, q2.half(), lam), (q1.cpu(), q2, lam),
                (q1, q2, lam[:3]), (q1, q2, lam.double()), (q1, q2, lam.cpu()),
                (q1[0], q2[0], lam),
                (q1, torch.zeros(2, 4, 1, 128, dtype=torch.bfloat16, device="cuda")[..., ::2],
                 lam)):
        with pytest.raises(ValueError):
            ops.paged_fwd(cache, *bad)
    for kw in (dict(norm_w=w[:, :64]), dict(norm_w=w.half()), dict(out=good[:1]),
               dict(out=good.float()), dict(out=good.cpu()),
               dict(workspace=torch.empty(64, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            ops.paged_fwd(cache, q1, q2, lam, **kw)
    with pytest.raises(ops.DiffAttnError):  # N past 16 tokens
        ops.paged_fwd(cache, *(torch.zeros(2, 4, 17, 64, dtype=torch.bfloat16, device="cuda"),) * 2,
                      lam)
    assert ops.paged_fwd(cache, q1, q2, lam, eps=-1.0, raw_status=True) == ops.ERR_INVALID_ARG
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    assert ops.paged_fwd(cache, q1, q2, lam, accumulate=True, workspace=small,
                         raw_status=True) == ops.ERR_INVALID_ARG
    for bad in ((new[0][:1], new[1], new[2]), (new[0], new[1][:, :1], new[2]),
                (new[0], new[1], new[0]), (new[0].float(), new[1], new[2]),
                (new[0], new[1], new[2].cpu())):
        with pytest.raises(ValueError):
            ops.paged_append(cache, *bad)
    assert ops.paged_evict(cache, keep=4, recent=5, raw_status=True) == ops.ERR_INVALID_ARG
    assert ops.paged_evict(cache, keep=-1, raw_status=True) == ops.ERR_INVALID_ARG
    torch.cuda.synchronize()
    for t, before in zip(("k1", "k2", "v", "weights"), pools):
        assert torch.equal(getattr(c, t).view(torch.uint8), before.view(torch.uint8))
    assert c.kv_len.tolist() == [40, 7]


def test_many_sequences():
    """More sequences than one warp scans at a time, most of them short, some idle."""
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 260, (300,), generator=g).tolist()
    c = R.Cache(101, lens=lens, kv=1, d=64, page=16)
    _parity(c, 2, 1)


@pytest.mark.parametrize("lens", [[5, 300, 0], [0, 0, 0], [129]])
@pytest.mark.parametrize("kv,H", [(2, 4), (1, 40)])
def test_capacity_far_beyond_the_lengths(lens, kv, H):
    c = R.Cache(102, lens=lens, kv=kv, d=64, page=32, extra_pages=500, weights=True)
    out = _parity(c, H, 1)
    if not any(lens):
        assert not bool(out.any())
    before = c.weights.clone()
    q1, q2, lam, w = R.queries(3, c.B, H, 1, 64)
    _, _, add, add_tol = R.attend(c, q1, q2, lam, norm_w=w)
    _fwd(c, q1, q2, lam, w, accumulate=True)
    after = c.weights
    for b, n in enumerate(lens):
        c.weights = before
        old = c.rows("weights", b).double()
        c.weights = after
        R.check(c.rows("weights", b), old + add[b],
                add_tol[b] + (old + add[b]) * (H // kv + 2) * 2.0 ** -23, "weights")


@pytest.mark.parametrize("d,dtype,H,N,top", [
    (64, torch.bfloat16, 2, 1, 130), (128, E4M3, 4, 3, 40), (64, E4M3, 40, 1, 130),
    (128, torch.bfloat16, 2, 1, 700)])
def test_many_short_items(d, dtype, H, N, top):
    """More items than SMs, taken whole (or cut, the longest): idle sequences and bad ones among
    them, with weights and without."""
    g = torch.Generator().manual_seed(118)
    lens = torch.randint(0, top + 1, (190,), generator=g).tolist()
    lens[:5] = [0, 1, top, 0, top - 1]
    lens[-2:] = [top, 0]
    c = R.Cache(119, lens=lens, kv=2, d=d, page=16, dtype=dtype, weights=True)
    out = _parity(c, H, N)
    before = c.weights.clone()
    q1, q2, lam, w = R.queries(3, c.B, H, N, d, dtype)
    assert torch.equal(_fwd(c, q1, q2, lam, w, accumulate=True), out)
    _, _, add, add_tol = R.attend(c, q1, q2, lam, norm_w=w, lambda_init=LI)
    after = c.weights
    for b in (1, 2, 4, 90, 188):
        if lens[b]:
            c.weights = before
            want = c.rows("weights", b).double() + add[b]
            c.weights = after
            R.check(c.rows("weights", b), want,
                    add_tol[b] + want.abs() * (H // 2 * N + 2) * 2.0 ** -23, f"weights of {b}")
    page = c.table[2, 0].item()
    c.table[2, 0] = -7
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ops.paged_fwd(c.ops_cache(), q1, q2, lam, norm_w=w, lambda_init=LI, status=status)
    assert int(status) == ops.ERR_PAGE and bool(torch.isnan(got[2]).all())
    got[2] = out[2]
    assert torch.equal(got, out)
    c.table[2, 0] = page


def test_two_row_blocks_share_a_head():
    """40 and 64 rows a key/value head, joined, with weights over all of them."""
    for H, N in ((40, 1), (16, 4)):
        c = R.Cache(103, lens=[3000, 700], kv=1, d=64, page=64, weights=True)
        before = c.weights.clone()
        q1, q2, lam, w = R.queries(104, 2, H, N, 64)
        out = _fwd(c, q1, q2, lam, w, accumulate=True)
        ref, tol, add, add_tol = R.attend(c, q1, q2, lam, norm_w=w, lambda_init=LI)
        R.check(out, ref, tol, "out")
        after = c.weights
        for b in range(2):
            c.weights = before
            old = c.rows("weights", b).double()
            c.weights = after
            want = old + add[b]
            R.check(c.rows("weights", b), want,
                    add_tol[b] + want * (H * N + 2) * 2.0 ** -23, "weights")


def test_sequences_that_share_a_prefix():
    """A page may stand in several sequences' tables where a call only reads it."""
    c = R.Cache(105, lens=[200, 150, 70], kv=2, d=64, page=16)
    c.table[1, :4] = c.table[0, :4]
    c.table[2, :2] = c.table[0, :2]
    _parity(c, 4, 2)


@pytest.mark.parametrize("seed", range(16))
def test_random_problems(seed):
    g = torch.Generator().manual_seed(200 + seed)
    pick = lambda *x: x[int(torch.randint(len(x), (1,), generator=g))]
    kv, group, N = pick(1, 2, 3), pick(1, 2, 3, 5, 8), pick(1, 1, 2, 4, 7)
    B, hi = pick(1, 2, 5), pick(40, 400, 1500)
    lens = torch.randint(0, hi + 1, (B,), generator=g).tolist()
    c = R.Cache(300 + seed, lens=lens, kv=kv, d=pick(64, 128), page=pick(16, 32, 48, 80, 128),
                dtype=pick(torch.bfloat16, E4M3), layout=pick("head", "token"),
                extra_pages=pick(0, 3))
    _parity(c, kv * group, N, seed=seed, causal=pick(True, False), headnorm=pick(0, 1, 2))


def test_workspace_contents_do_not_matter():
    c = R.Cache(106, lens=[900, 20, 2000], kv=2, d=64, page=16, weights=True)
    cache = c.ops_cache()
    q1, q2, lam, w = R.queries(107, 3, 8, 2, 64)
    kw = dict(norm_w=w, lambda_init=LI, accumulate=True)
    before = c.weights.clone()
    need = ops.paged_fwd_plan(cache, 8, 2, accumulate=True)
    got = []
    for fill in (0, 255, 127):
        c.weights.copy_(before)
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        got.append((ops.paged_fwd(cache, q1, q2, lam, workspace=ws, **kw), c.weights.clone()))
    for out, weights in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(weights, got[0][1])
    pools = {t: getattr(c, t).clone() for t in ("k1", "k2", "v", "weights", "kv_len")}
    got = []
    for fill in (0, 255, 127):
        for t, x in pools.items():
            getattr(c, t).copy_(x)
        ws = torch.full((ops.paged_evict_plan(cache, keep=500),), fill, dtype=torch.uint8,
                        device="cuda")
        ops.paged_evict(cache, keep=500, recent=20, workspace=ws)
        got.append([getattr(c, t).clone() for t in pools])
    for other in got[1:]:
        for x, y in zip(other, got[0]):
            bits = torch.int16 if x.dtype == torch.bfloat16 else torch.int32
            assert torch.equal(x.view(bits), y.view(bits))


def test_steps_without_waiting_are_those_with():
    """Lengths raised, rows appended, attention, eviction, back to back on the stream: kernels that
    start before the ones ahead of them end see what those wrote."""
    outs = []
    for wait in (True, False):
        c = R.Cache(108, lens=[700, 700, 700], kv=2, d=64, page=16, weights=True, fill=0.0)
        c.kv_len.copy_(torch.tensor([3, 600, 250], dtype=torch.int32))
        cache = c.ops_cache()
        g = torch.Generator(device="cuda").manual_seed(109)
        q1, q2, lam, w = R.queries(110, 3, 4, 1, 64)
        torch.cuda.synchronize()
        got = []
        for step in range(60):
            new = [torch.randn(3, 2, 1, x, generator=g, device="cuda").to(torch.bfloat16)
                   for x in (64, 64, 128)]
            c.kv_len.add_(1)
            ops.paged_append(cache, *new)
            got.append(ops.paged_fwd(cache, q1, q2, lam, norm_w=w, accumulate=True))
            ops.paged_evict(cache, keep=610, recent=30)
            if wait:
                torch.cuda.synchronize()
        outs.append(got + [c.weights, c.kv_len])
    for x, y in zip(*outs):
        assert torch.equal(x, y)


def test_next_kernel_waits_where_no_item_is_cut():
    """Items that fill the CTAs' shares exactly, so that the second kernel has nothing to join: what
    follows on the stream still sees the outputs."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    c = R.Cache(116, lens=[1024] * (2 * sms), kv=1, d=64, page=64)
    cache = c.ops_cache()
    q1, q2, lam, w = R.queries(117, 2 * sms, 1, 1, 64)
    want = _fwd(c, q1, q2, lam, w)
    out = torch.empty_like(want)
    ws = torch.empty(ops.paged_fwd_plan(cache, 1), dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(50):
        out.fill_(float("nan"))
        ops.paged_fwd(cache, q1, q2, lam, norm_w=w, lambda_init=LI, workspace=ws, out=out)
        got.append(out.clone())
    torch.cuda.synchronize()
    for x in got:
        assert torch.equal(x, want)


def test_two_graphs_with_a_workspace_each_replay_at_once():
    c = R.Cache(111, lens=[3000, 500], kv=2, d=64, page=16)
    cache = c.ops_cache()
    graphs, outs, want = [], [], []
    for k in range(2):
        q1, q2, lam, w = R.queries(112 + k, 2, 4, 1, 64)
        want.append(_fwd(c, q1, q2, lam, w))
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            ops.paged_fwd(cache, q1, q2, lam, norm_w=w, lambda_init=LI)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(ops.paged_fwd(cache, q1, q2, lam, norm_w=w, lambda_init=LI))
        graphs.append((graph, side, (q1, q2, lam, w)))
    for _ in range(20):
        for graph, side, _ in graphs:
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    for out, ref in zip(outs, want):
        assert torch.equal(out, ref)


def test_bounds_checked_build_agrees():
    """The debug build's checks find nothing, and its results are the release build's."""
    import ctypes

    from differential_attention_attn_gb300 import build as libbuild
    debug = ops.bind(ctypes.CDLL(libbuild.build(debug=True)))
    for d, dtype, N, H in ((64, torch.bfloat16, 3, 8), (128, E4M3, 1, 2), (64, E4M3, 1, 24),
                           (128, torch.bfloat16, 5, 8)):
        both = []
        for lib in (ops.load(), debug):
            with ops.using(lib):
                c = R.Cache(113, lens=[1500, 0, 70, 129], kv=2, d=d, page=48, dtype=dtype,
                            weights=True, fill=0.0)
                cache = c.ops_cache()
                q1, q2, lam, w = R.queries(114, 4, H, N, d, dtype)
                g = torch.Generator().manual_seed(115)
                new = [torch.randn(4, 2, N, x, generator=g).to(torch.bfloat16).cuda()
                       for x in (d, d, 2 * d)]
                status = torch.zeros(1, dtype=torch.int32, device="cuda")
                ops.paged_append(cache, *new, status=status)
                out = ops.paged_fwd(cache, q1, q2, lam, norm_w=w, accumulate=True, status=status)
                ops.paged_evict(cache, keep=100, recent=9, status=status)
                torch.cuda.synchronize()
                assert int(status) == 0
                both.append([out, c.weights, c.v, c.kv_len])
        for x, y in zip(*both):
            assert torch.equal(x, y)


def test_numbers_given_as_tensors_are_read_at_every_call():
    """eps and lambda_init as tensors of one element that change in place between calls."""
    c = R.Cache(125, lens=[40, 7], kv=2, d=64, page=16)
    cache = c.ops_cache()
    q1, q2, lam, w = R.queries(126, 2, 4, 1, 64)
    li, eps = torch.tensor(0.25), torch.tensor(1e-5)
    for a, b in ((0.25, 1e-5), (0.75, 1e-5), (0.75, 0.5)):
        li.fill_(a)
        eps.fill_(b)
        got = ops.paged_fwd(cache, q1, q2, lam, norm_w=w, lambda_init=li, eps=eps)
        ref, tol, _, _ = R.attend(c, q1, q2, lam, norm_w=w, lambda_init=a, eps=b)
        R.check(got, ref, tol, f"lambda_init {a}, eps {b}")


@pytest.mark.parametrize("lens,upto,kv,H", [
    ([600, 300], 128, 2, 4),    # the whole first tile
    ([600, 300], 290, 1, 1),    # two tiles and a part of the third
    ([9000, 40], 7000, 1, 8),   # whole parts of a joined item
    ([3000, 200], 2999, 1, 40),  # one key is left; two row blocks
])
def test_keys_with_logits_of_minus_infinity_weigh_nothing(lens, upto, kv, H):
    """Visible keys whose logits are -infinity, over whole tiles: the softmax of the others."""
    c = R.Cache(127, lens=lens, kv=kv, d=64, page=16, weights=True)
    for b, n in enumerate(lens):
        t = torch.arange(min(upto, n - 1), device="cuda")
        for pool in (c.k1, c.k2):
            pool[c.table[b].long()[t // 16], :, t % 16, 3] = -float("inf")
    q1, q2, lam, w = R.queries(128, 2, H, 1, 64)
    for q in (q1, q2):
        q[..., 3] = 0.5
    old = [c.rows("weights", b).double() for b in range(2)]
    out = _fwd(c, q1, q2, lam, w, accumulate=True)
    ref, tol, add, add_tol = R.attend(c, q1, q2, lam, norm_w=w, lambda_init=LI)
    assert bool(torch.isfinite(ref).all())
    R.check(out, ref, tol, "out")
    for b in range(2):
        want = old[b] + add[b]
        R.check(c.rows("weights", b), want,
                add_tol[b] + want * (H // kv + 2) * 2.0 ** -23, "weights")


@pytest.mark.parametrize("B,kv", [(3, 2), (40, 8)])
def test_evict_then_append_and_attend_with_nothing_between(B, kv):
    """The next kernels start while the eviction runs, and see the lengths that it writes: with keys
    replaced at the end of what stays."""
    lens = [700 - 3 * b for b in range(B)]
    results = []
    for wait in (True, False):
        c = R.Cache(129, lens=lens, kv=kv, d=64, page=16, weights=True, fill=0.0)
        cache = c.ops_cache()
        pools = {t: getattr(c, t).clone() for t in ("k1", "k2", "v", "weights", "kv_len")}
        q1, q2, lam, w = R.queries(130, B, 2 * kv, 2, 64)
        g = torch.Generator().manual_seed(131)
        new = [torch.randn(B, kv, 2, x, generator=g).to(torch.bfloat16).cuda()
               for x in (64, 64, 128)]
        got = []
        for step in range(20):
            for t, x in pools.items():
                getattr(c, t).copy_(x)
            torch.cuda.synchronize()
            ops.paged_evict(cache, keep=300 + step, recent=30)
            if wait:
                torch.cuda.synchronize()
            ops.paged_append(cache, *new)
            if wait:
                torch.cuda.synchronize()
            got.append(ops.paged_fwd(cache, q1, q2, lam, norm_w=w, accumulate=True))
            torch.cuda.synchronize()
            got.append(c.weights.clone())
            assert c.kv_len.tolist() == [300 + step] * B
        results.append(got)
        c.lens = c.kv_len.tolist()
        for b in (0, B - 1):
            assert torch.equal(c.rows("v", b)[:, -2:], new[2][b])
    for x, y in zip(*results):
        assert torch.equal(x, y)


@pytest.mark.parametrize("H,kv,N", [(2, 2, 1), (4, 1, 1), (1, 1, 8), (8, 1, 2)])
@pytest.mark.parametrize("top", [40, 700])
def test_ends_of_items_behind_values_in_flight(H, kv, N, top):
    """d = 128 with bf16 keys has three value buffers for two a tile: the garbage behind a sequence's
    end is cleared in the tile's own values, not in those of the tile before, which may still be on
    their way.  Call after call on many short items, with other traffic beside them."""
    g = torch.Generator().manual_seed(132)
    lens = torch.randint(0, top + 1, (200,), generator=g).tolist()
    c = R.Cache(133, lens=lens, kv=kv, d=128, page=16)
    out = _parity(c, H, N)
    cache = c.ops_cache()
    q1, q2, lam, w = R.queries(3, c.B, H, N, 128)
    noise = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(100):
            noise.add_(1)
    got = [ops.paged_fwd(cache, q1, q2, lam, norm_w=w, lambda_init=LI) for _ in range(60)]
    torch.cuda.synchronize()
    for x in got:
        assert torch.equal(x, out)


@pytest.mark.parametrize("keep", [119, 160, 161, 1 << 40])
@pytest.mark.parametrize("bad", [-1, 161, 2 ** 31 - 1, -2 ** 31])
def test_evict_reports_a_bad_length_whatever_the_budget(keep, bad):
    """Budgets below, at and past the 160 keys that the table has room for, among 300 sequences."""
    c = R.Cache(134, lens=[100] + [30] * 299, kv=1, d=64, page=16, weights=True, extra_pages=3)
    cache = c.ops_cache()
    assert c.max_pages * 16 == 160
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pools = [getattr(c, t).clone() for t in ("k1", "k2", "v", "weights")]
    ops.paged_evict(cache, keep=keep, recent=3, status=status)
    assert int(status) == 0
    c.kv_len[299] = bad
    ops.paged_evict(cache, keep=keep, recent=3, status=status)
    assert int(status) == ops.ERR_PAGE
    ops.paged_evict(cache, keep=keep, recent=3)  # no status word: nothing to report to
    torch.cuda.synchronize()
    assert c.kv_len.tolist() == [100] + [30] * 298 + [bad]
    for t, x in zip(("k1", "k2", "v", "weights"), pools):
        assert torch.equal(getattr(c, t).view(torch.uint8), x.view(torch.uint8)), t


def _longest_share(lens, heads, ctas):
    """Steps (a tile each, two more an item) of the longest share and of an equal one, for items
    taken whole by one CTA each, whole in the equal shares that they begin in, and cut."""
    item = [2 + max(1, -(-n // 128)) for n in lens for _ in range(heads)]
    total = sum(item)
    alone = max(item) if len(item) <= ctas else None
    each, more = divmod(total, ctas)
    begins = [c * each + min(c, more) for c in range(ctas + 1)]
    at, c, uncut = 0, 0, [0] * ctas
    for x in item:
        while c + 1 < ctas and begins[c + 1] <= at:
            c += 1
        uncut[c] += x
        at += x
    return alone, max(uncut), total / ctas


@pytest.mark.parametrize("B,kv,lo,hi,big", [
    (18, 8, 100, 9001, 0), (19, 8, 100, 9001, 0), (38, 8, 100, 9001, 0), (19, 8, 200, 200, 32768),
    (38, 8, 200, 200, 32768), (16, 8, 200, 200, 4800), (57, 8, 500, 900, 0), (64, 16, 100, 700, 0),
    (8, 8, 1024, 1024, 0), (1, 16, 200, 200, 0)])
def test_ragged_batches_are_balanced(B, kv, lo, hi, big):
    """The kernels take items whole only where no CTA has many steps more than in equal shares: told
    from the parts that a call leaves in its workspace, as the second kernel would read them."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    lens = [hi - (hi - lo) * b // max(1, B - 1) for b in range(B)]
    if big:
        lens[B // 2] = big
    page, d = 64, 64
    max_pages = -(-max(lens) // page) + 600  # far more room than any sequence takes
    need = [-(-n // page) for n in lens]
    P = sum(need)
    table = torch.full((B, max_pages), -1, dtype=torch.int32)
    ids = iter(torch.randperm(P, generator=torch.Generator().manual_seed(135)).tolist())
    for b in range(B):
        for k in range(need[b]):
            table[b, k] = next(ids)
    g = torch.Generator(device="cuda").manual_seed(136)
    pool = lambda w: torch.randn(P, kv, page, w, generator=g, device="cuda").to(torch.bfloat16)
    cache = ops.PagedCache(pool(d), pool(d), pool(2 * d), table.cuda(),
                           torch.tensor(lens, dtype=torch.int32, device="cuda"))
    q1, q2, lam, w = R.queries(137, B, kv, 1, d)
    need_ws = ops.paged_fwd_plan(cache, kv)
    slots = 2 * sms * 2  # partial states: [2 CTAs][2 maps], a row of 2 d each; then their (m, l)
    part_bytes = -(-slots * 2 * d * 4 // 256) * 256
    assert need_ws == part_bytes + -(-slots * 8 // 256) * 256
    mark = 12345.0
    ws = torch.full((need_ws // 4,), mark, device="cuda")
    out = ops.paged_fwd(cache, q1, q2, lam, norm_w=w, workspace=ws)
    parts = ws[part_bytes // 4:][:slots * 2].view(2 * sms, 2, 2)
    cut = bool((parts != mark).any())
    alone, uncut, equal = _longest_share(lens, kv, sms)
    if not cut:  # at most as far from equal shares as the rules have it
        assert (alone is not None and alone - 2 <= equal + 6) or uncut <= equal + 5
    elif alone is not None:
        assert alone - 2 > equal - 2 * B * kv / sms + 6 - 1e-9
    # the same values as one sequence after another
    for b in sorted({0, B // 2, B - 1}):
        one = ops.PagedCache(cache.k1, cache.k2, cache.v, table[b:b + 1].cuda(),
                             cache.kv_len[b:b + 1].clone())
        ref = ops.paged_fwd(one, q1[b:b + 1], q2[b:b + 1], lam, norm_w=w).float()
        # each within a bf16 rounding and its fp32 sums of the value: 2^-8 and 2^-12 apart at most
        err = (out[b:b + 1].float() - ref).abs()
        assert bool((err <= ref.abs() * 2.0 ** -7 + 2.0 ** -12 * ref.abs().amax(-1, True)).all())


def test_modes_follow_the_lengths_under_one_graph():
    """One captured call, replayed with lengths that have its items taken one to a CTA, whole in
    shares, and cut: the values are the definition's, and those of a call with these lengths."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for B, kv, sets in (
            (20, 2, ([100] * 20, [1500] + [90] * 19, [1500] * 20, [0] * 20, [7, 1200] * 10)),
            (sms, 2, ([150] * sms, [1500] + [90] * (sms - 1), [0, 300] * (sms // 2) + [1] * (sms % 2)))):
        c = R.Cache(138, lens=[1500] * B, kv=kv, d=64, page=64, weights=True)
        cache = c.ops_cache()
        q1, q2, lam, w = R.queries(139, B, kv, 1, 64)
        call = lambda: ops.paged_fwd(cache, q1, q2, lam, norm_w=w, lambda_init=LI, accumulate=True)
        start = c.weights.clone()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        for lens in sets:
            c.lens = lens
            c.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
            c.weights.copy_(start)
            graph.replay()
            got, weights = out.clone(), c.weights.clone()
            c.weights.copy_(start)
            assert torch.equal(call(), got) and torch.equal(c.weights, weights)
            some = sorted({0, 1, B // 2, B - 1})
            sub = R.Cache.__new__(R.Cache)
            sub.__dict__.update(c.__dict__)
            sub.lens, sub.table = [lens[b] for b in some], c.table[some]
            ref, tol, add, add_tol = R.attend(sub, q1[some], q2[some], lam, norm_w=w,
                                              lambda_init=LI)
            R.check(got[some], ref, tol, f"lengths {lens[:3]}")
            for k, b in enumerate(some):
                if not lens[b]:
                    continue
                sub.weights = start
                want = sub.rows("weights", k).double() + add[k]
                sub.weights = weights
                R.check(sub.rows("weights", k), want, add_tol[k] + want.abs() * 3 * 2.0 ** -23,
                        f"weights of {b}")


@pytest.mark.parametrize("lens,kv,H", [([200], 16, 16), ([90, 0, 33], 2, 8), ([130] * 100, 3, 3)])
def test_room_beyond_the_lengths_changes_nothing(lens, kv, H):
    """Items taken whole because of the lengths give the bits of those that no length would cut."""
    outs = []
    for extra in (0, 600):
        c = R.Cache(140, lens=lens, kv=kv, d=64, page=16, extra_pages=extra)
        outs.append(_fwd(c, *R.queries(141, len(lens), H, 1, 64)))
        assert (ops.paged_fwd_plan(c.ops_cache(), H) > 0) == (extra > 0)
    assert torch.equal(*outs)


@pytest.mark.parametrize("kind", ["one to a CTA", "between items"])
def test_next_kernel_waits_where_the_second_finds_nothing_to_join(kind):
    """The second kernel is launched, because other lengths would have items cut, and has nothing to
    do: what follows on the stream still sees the outputs."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    extra = 0
    if kind == "one to a CTA":  # 64 items of eight tiles, with room for more
        lens, kv, extra = [1024] * 8, 8, 20
    else:  # steps of 20, 10 and 10: the bounds of equal shares fall between items
        lens, kv = [18 * 128, 8 * 128, 8 * 128] * (sms // 2), 1
    c = R.Cache(142, lens=lens, kv=kv, d=64, page=128, extra_pages=extra)
    cache = c.ops_cache()
    q1, q2, lam, w = R.queries(143, len(lens), kv, 1, 64)
    need = ops.paged_fwd_plan(cache, kv)
    assert need > 0
    want = _fwd(c, q1, q2, lam, w)
    out = torch.empty_like(want)
    ws = torch.full((need,), 1, dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(50):
        out.fill_(float("nan"))
        ops.paged_fwd(cache, q1, q2, lam, norm_w=w, lambda_init=LI, workspace=ws, out=out)
        got.append(out.clone())
    torch.cuda.synchronize()
    for x in got:
        assert torch.equal(x, want)
    assert bool((ws == 1).all())  # no partial state was left: nothing was cut


@pytest.mark.parametrize("B,kv,d,dtype,layout,page", [
    (5, 8, 64, torch.bfloat16, "head", 16),    # 40 heads: slices of 128 bytes
    (13, 3, 128, torch.bfloat16, "token", 48),  # 39
    (10, 8, 64, E4M3, "token", 64), (4, 10, 128, E4M3, "head", 16),
    (6, 4, 64, torch.bfloat16, "head", 32),    # 24: slices of 64 bytes
    (5, 3, 128, torch.bfloat16, "head", 16), (7, 3, 64, E4M3, "head", 16)])  # the last: of 32
def test_evict_of_many_heads(B, kv, d, dtype, layout, page):
    """As many heads as a served batch has: the move takes wider slices of the rows then."""
    lens = [800 - 61 * b for b in range(B)]
    c = R.Cache(144, lens=lens, kv=kv, d=d, page=page, dtype=dtype, layout=layout, weights=True)
    _check_evict(c, 300, 32)
    _check_evict(c, 299, 0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])
@pytest.mark.parametrize("layout,page", [("head", 48), ("token", 64)])
def test_append_many_rows_of_every_type(d, dtype, layout, page):
    """More than 16384 rows, an odd number a head, with padding in front and strided sources."""
    N, kv = 1639, 5
    lens = [1700, 1639, 3, 0]
    c = R.Cache(145, lens=lens, kv=kv, d=d, page=page, dtype=dtype, layout=layout, weights=True,
                fill=7.0)
    assert 4 * kv * N > 16384
    want = {t: R.f64(getattr(c, t)).clone() for t in ("k1", "k2", "v", "weights")}
    g = torch.Generator().manual_seed(146)
    new = {t: (torch.randn(4, N, kv, w, generator=g) * 200).to(torch.bfloat16).cuda()
           .permute(0, 2, 1, 3) for t, w in (("k1", d), ("k2", d), ("v", 2 * d))}
    for b, n in enumerate(lens):
        at = torch.arange(max(0, n - N), n, device="cuda")
        pages, slots = c.table[b].long()[at // page], at % page
        for t in ("k1", "k2", "v"):
            rows = R.f64(new[t][b, :, N - len(at):]).transpose(0, 1)
            want[t][pages, :, slots] = R.to_e4m3(rows) if dtype == E4M3 and t != "v" else rows
        want["weights"][pages, :, slots] = 0
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.paged_append(c.ops_cache(), new["k1"], new["k2"], new["v"], status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    for t in want:
        assert torch.equal(R.f64(getattr(c, t)), want[t]), t


def test_many_items_that_are_cut():
    """More items than SMs, long enough to be cut, with idle sequences and a bad one among them."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    lens = torch.randint(0, 1101, (sms,), generator=torch.Generator().manual_seed(147)).tolist()
    lens[:5] = [0, 1, 1100, 0, 1099]
    lens[-2:] = [1100, 0]
    _, uncut, equal = _longest_share(lens, 2, sms)
    assert uncut > equal + 5
    c = R.Cache(148, lens=lens, kv=2, d=64, page=16, weights=True)
    before = c.weights.clone()
    out = _parity(c, 4, 2)
    q1, q2, lam, w = R.queries(3, c.B, 4, 2, 64)
    assert torch.equal(_fwd(c, q1, q2, lam, w, accumulate=True), out)
    _, _, add, add_tol = R.attend(c, q1, q2, lam, norm_w=w, lambda_init=LI)
    after = c.weights
    for b in range(sms):
        if lens[b]:
            c.weights = before
            want = c.rows("weights", b).double() + add[b]
            c.weights = after
            R.check(c.rows("weights", b), want, add_tol[b] + want.abs() * 6 * 2.0 ** -23,
                    f"weights of {b}")
    c.table[4, 60] = -7
    kept = c.weights.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ops.paged_fwd(c.ops_cache(), q1, q2, lam, norm_w=w, lambda_init=LI, status=status,
                        accumulate=True)
    assert int(status) == ops.ERR_PAGE and bool(torch.isnan(got[4]).all())
    got[4] = out[4]
    assert torch.equal(got, out)
    mine = [int(x) for x in c.table[4] if x >= 0]
    assert torch.equal(c.weights[mine], kept[mine])


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("d", [64, 128])
def test_non_finite_newest_values_of_a_joined_item(bad, d):
    """Values kept out of the product reach the rows that see them through the partial states."""
    lens = [9003, 5000, 130]
    c = R.Cache(149, lens=lens, kv=1, d=d, page=16)
    for b, n in enumerate(lens):
        for back in (1, 2):
            c.v[int(c.table[b, (n - back) // 16]), 0, (n - back) % 16, 5] = bad
    q1, q2, lam, w = R.queries(150, 3, 2, 4, d)
    out = _fwd(c, q1, q2, lam, w, headnorm=0).double()
    ref, tol, _, _ = R.attend(c, q1, q2, lam, headnorm=0)
    R.check(out[:, :, :2], ref[:, :, :2], tol[:, :, :2], "rows before them")
    others = [x for x in range(2 * d) if x != 5]
    assert not bool(torch.isfinite(out[:, :, 2:, 5]).any())
    clean = R.Cache.__new__(R.Cache)
    clean.__dict__.update(c.__dict__)
    clean.v = c.v.clone()
    clean.v[..., 5] = 0
    ref, tol, _, _ = R.attend(clean, q1, q2, lam, headnorm=0)
    R.check(out[:, :, 2:][..., others], ref[:, :, 2:][..., others], tol[:, :, 2:][..., others],
            "the other columns")
