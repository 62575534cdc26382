"""Rotary positions on the GPU against float64."""
import math

import pytest
import torch

from differential_attention_attn_gb300 import ops
from tests import ragged_ref as G

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _rows(seed, B, heads, N, d, dtype, layout):
    g = torch.Generator().manual_seed(seed)
    if layout == "token":
        x = torch.randn(B, N, heads, d, generator=g).permute(0, 2, 1, 3)
    elif layout == "wide":  # a slice of rows twice as wide
        x = torch.randn(B, heads, N, 2 * d, generator=g)
    else:
        x = torch.randn(B, heads, N, d, generator=g)
    x = x.to(dtype).cuda()
    return x[..., d:] if layout == "wide" else x


def _check(table, kw, xs, ys, pos, inverse=False):
    freq, m = G.frequencies(**kw)
    for x, y in zip(xs, ys):
        ref, tol = G.turn(x.double(), pos[:, None], freq, m, table.neighbours, inverse,
                          short=x.dtype == BF16)
        tol = G.rounded(ref, tol, x.dtype)
        assert y.dtype == x.dtype and float(((y.double() - ref).abs() - tol).max()) <= 0
        r = kw["rot"]
        assert torch.equal(y[..., r:], x[..., r:])  # channels that are only copied


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 48)])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("layout,N", [("head", 1), ("token", 77), ("wide", 300)])
def test_forward_and_back(dtype, d, rot, neighbours, layout, N):
    kw = dict(rot=rot)
    table = ops.RotaryTable(**kw, neighbours=neighbours)
    xs = [_rows(i, 3, h, N, d, dtype, layout) for i, h in enumerate((5, 5, 1, 2))]
    pos = torch.randint(0, 5000, (3, N), dtype=torch.int32, generator=torch.Generator().manual_seed(1))
    ys = ops.rotary(table, xs, pos.cuda())
    _check(table, kw, xs, ys, pos.cuda())
    _check(table, kw, xs, ops.rotary_bwd(table, xs, pos.cuda()), pos.cuda(), inverse=True)


@pytest.mark.parametrize("kw", [
    dict(rot=64, scaling="linear", factor=8.0), dict(rot=64, scaling="ntk", factor=4.0),
    dict(rot=128, scaling="parts", factor=4.0, original=4096.0),
    dict(rot=32, base=500000.0, scaling="parts", factor=7.5, original=8192.0, fast=4.0, slow=0.5)])
def test_scalings(kw):
    table = ops.RotaryTable(**kw)
    freq, m = G.frequencies(**kw)
    got = table.freq.cpu().double()  # fractions below a quarter turn: int64 holds them
    unit = 2 * math.pi / 2.0 ** 64  # a fraction is cut to a whole number of these; pow: a few ulp
    assert torch.allclose(got * unit, freq, rtol=2.0 ** -48, atol=unit)
    assert abs(table.scale - m) <= m * 2.0 ** -24
    xs = [_rows(4, 2, 3, 50, 128, F32, "head")]
    ys = ops.rotary(table, xs, start=100)
    pos = (100 + torch.arange(50)).expand(2, 50).cuda()
    _check(table, kw, xs, ys, pos)


@pytest.mark.parametrize("at", [-7, 2 ** 20 + 3, 2 ** 31 - 40])
def test_far_and_negative_positions(at):
    kw = dict(rot=64)
    table = ops.RotaryTable(**kw)
    xs = [_rows(5, 1, 2, 33, 64, F32, "head")]
    pos = torch.arange(at, at + 33, dtype=torch.int64)
    _check(table, kw, xs, ops.rotary(table, xs, pos.to(torch.int32).cuda()), pos[None].cuda())
    assert torch.equal(ops.rotary(table, xs, start=at)[0],
                       ops.rotary(table, xs, pos.to(torch.int32).cuda())[0])


@pytest.mark.parametrize("heads", [1, 33])
def test_in_place_and_many_rows(heads):
    """In place, and more rows than one head a thread takes."""
    kw = dict(rot=32)
    table = ops.RotaryTable(**kw, neighbours=True)
    xs = [_rows(6 + i, 2, h, 2100, 64, BF16, "token") for i, h in enumerate((heads, 7))]
    pos = torch.arange(2100, dtype=torch.int32, device="cuda")
    ys = ops.rotary(table, xs, pos)
    _check(table, kw, xs, ys, pos.expand(2, 2100))
    same = [x.clone() for x in xs]
    for s, x in zip(same, xs):
        assert s.stride() == x.stride()
    got = ops.rotary(table, same, pos, outs=same)
    assert got[0] is same[0] and all(torch.equal(a, b) for a, b in zip(same, ys))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_offsets_past_32_bits(dtype):
    """Rows 2^31 elements apart, from batch to batch, head to head or token to token, in place and
    into another tensor."""
    kw = dict(rot=64)
    table = ops.RotaryTable(**kw)
    for axis in range(3):
        shape = [1, 1, 1, 64]
        shape[axis] = 3
        strides = [64 * shape[1] * shape[2], 64 * shape[2], 64, 1]
        strides[axis] = 2 ** 31
        x = torch.empty(2 ** 32 + 64, dtype=dtype, device="cuda").as_strided(shape, strides)
        x.copy_(_rows(9 + axis, *shape, dtype, "head"))
        pos = torch.arange(7, 7 + shape[2], device="cuda")
        y = ops.rotary(table, [x], start=7)[0]
        _check(table, kw, [x], [y], pos.expand(shape[0], shape[2]))
        assert torch.equal(ops.rotary(table, [x], start=7, outs=[x])[0], y)


def test_gradient_against_differences():
    """sum(dy * rotary(x)) changes by the gradient: the map is linear, so one difference is exact
    up to fp32 (64-bit sums; each of the 2 * 3 * 20 * 64 terms is off by at most 12 * 2^-24 of the
    values it comes from)."""
    table = ops.RotaryTable(64, scaling="parts", factor=4.0, original=4096.0)
    x, dx, dy = (_rows(s, 2, 3, 20, 64, F32, "head") for s in (1, 2, 3))
    y0, y1 = ops.rotary(table, [x], start=9)[0], ops.rotary(table, [x + dx], start=9)[0]
    g = ops.rotary_bwd(table, [dy], start=9)[0]
    want = (dy.double() * (y1.double() - y0.double())).sum()
    got = (g.double() * ((x + dx).double() - x.double())).sum()
    bound = 24 * 2.0 ** -24 * 2 * table.scale * float((dy.abs() * (x.abs() + (x + dx).abs() + dx.abs())
                                                       .amax(-1, keepdim=True)).double().sum())
    assert abs(float(want - got)) <= bound


def test_streams_graphs_and_nothing_to_do():
    table = ops.RotaryTable(64)
    x = _rows(8, 1, 4, 40, 64, BF16, "head")
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    want = ops.rotary(table, [x], pos)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.rotary(table, [x], pos, stream=side)[0]
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.rotary(table, [x], pos, outs=[out])
    pos += 5
    graph.replay()
    assert torch.equal(out, ops.rotary(table, [x], start=5)[0])
    for B, H, N in ((0, 4, 3), (1, 0, 3), (2, 4, 0)):
        y = ops.rotary(table, [torch.empty(B, H, N, 64, dtype=BF16, device="cuda")], start=0)[0]
        assert y.shape == (B, H, N, 64)
    e = torch.empty(1, 0, 40, 64, dtype=BF16, device="cuda")  # one of several without heads
    assert torch.equal(ops.rotary(table, [e, x], start=5)[1], out)


def test_refusals():
    table = ops.RotaryTable(64)
    x = _rows(9, 2, 4, 8, 64, BF16, "head")
    for kw in (dict(rot=24), dict(rot=0), dict(rot=64, base=1.0), dict(rot=64, scaling="linear",
               factor=0.5), dict(rot=64, scaling="parts", factor=2.0)):
        with pytest.raises(ops.DiffAttnError):
            ops.RotaryTable(**kw)
    with pytest.raises(ValueError):
        ops.RotaryTable(64, scaling="other")
    with pytest.raises(ops.DiffAttnError):
        ops.rotary(ops.RotaryTable(128), [x])  # more channels than the row has
    with pytest.raises(ops.DiffAttnError):
        ops.rotary(table, [_rows(9, 1, 1, 8, 32, BF16, "head")])
    with pytest.raises(ops.DiffAttnError):
        ops.rotary(table, [x[:, :1].expand(2, 4, 8, 64)], outs=[x])  # a stride of zero
    for bad in (dict(tensors=[x] * 5), dict(tensors=[]), dict(tensors=[x.half()]),
                dict(tensors=[x, x.float()]), dict(tensors=[x, x[:, :, :4]]),
                dict(tensors=[x.cpu()]), dict(tensors=[x], outs=[x[:1]]),
                dict(tensors=[x.transpose(2, 3)]), dict(tensors=[x[0]]),
                dict(tensors=[x], positions=torch.zeros(8, dtype=torch.int64, device="cuda")),
                dict(tensors=[x], positions=torch.zeros(7, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            ops.rotary(table, **bad)
