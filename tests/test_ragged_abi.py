"""Rotary positions' and the packed batch's entry points: exported as declared, and refusing bad
arguments on the host."""
import ctypes
import glob
import math
import os
import re
import subprocess

import pytest
import torch

from differential_attention_attn_gb300 import build as libbuild
from differential_attention_attn_gb300 import ops
from tests import ragged_ref as G

FAKE = 0x10000  # never dereferenced: validation rejects or returns before any launch
I, U = ops.ERR_INVALID_ARG, ops.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return ops.load()


@pytest.mark.parametrize("header,prefix,names", [
    (ops.ROTARY_HEADER_PATH, "diffrotary_", {"diffrotary_frequencies", "diffrotary_apply"}),
    (ops.RAGGED_HEADER_PATH, "diffragged_", {"diffragged_step", "diffragged_append",
                                             "diffragged_fwd", "diffragged_fwd_plan"})])
def test_exports_what_the_header_declares(lib, header, prefix, names):
    text = re.sub(r"/\*.*?\*/", "", open(header).read(), flags=re.S)
    assert set(re.findall(r"\b(%s[a-z0-9_]+)\s*\(" % prefix, text)) == names
    out = subprocess.run(["nm", "-D", "--defined-only", libbuild.build()], capture_output=True,
                         text=True, check=True).stdout
    assert {x.split()[-1] for x in out.splitlines() if x.split()[-1].startswith(prefix)} == names


def test_struct_layouts():
    assert ctypes.sizeof(ops.RotaryTableStruct) == 8 + 4 * 4
    assert ctypes.sizeof(ops.PageBookStruct) == 5 * 8 + 3 * 8 + 8


# ---- rotary -----------------------------------------------------------------------------------

@pytest.mark.parametrize("kw", [dict(rot=16), dict(rot=128, base=500000.0),
                                dict(rot=64, scaling="linear", factor=8.0),
                                dict(rot=64, scaling="ntk", factor=4.0),
                                dict(rot=48, scaling="parts", factor=7.5, original=8192.0, fast=16.0,
                                     slow=0.0)])
def test_frequencies(lib, kw):
    want, m = G.frequencies(**kw)
    n = kw["rot"] // 2
    freq, scale = (ctypes.c_uint64 * n)(), ctypes.c_float(0)
    st = lib.diffrotary_frequencies(kw["rot"], kw.get("base", 10000.0),
                                    ops._SCALING[kw.get("scaling")], kw.get("factor", 1.0),
                                    kw.get("original", 0.0), kw.get("fast", 32.0),
                                    kw.get("slow", 1.0), freq, ctypes.byref(scale))
    assert st == ops.OK and abs(scale.value - m) <= m * 2.0 ** -24
    unit = 2 * math.pi / 2.0 ** 64  # fractions are cut to whole numbers of these
    for x, w in zip(freq, want.tolist()):
        assert abs(x * unit - w) <= w * 2.0 ** -48 + unit


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=8), dict(rot=24), dict(rot=-16),
                                dict(base=1.0), dict(base=math.nan), dict(base=math.inf),
                                dict(scaling=4), dict(scaling=-1), dict(scaling=1, factor=0.5),
                                dict(scaling=2, factor=math.nan), dict(scaling=3, factor=2.0),
                                dict(scaling=3, factor=2.0, original=10.0, slow=32.0),
                                dict(scaling=3, factor=2.0, original=10.0, slow=-1.0),
                                dict(freq=None), dict(scale=None)])
def test_frequencies_refused(lib, kw):
    a = dict(rot=64, base=10000.0, scaling=0, factor=1.0, original=0.0, fast=32.0, slow=1.0,
             freq=(ctypes.c_uint64 * 64)(), scale=ctypes.byref(ctypes.c_float(0)))
    a.update(kw)
    assert lib.diffrotary_frequencies(*a.values()) == I


def _table(**kw):
    t = ops.RotaryTableStruct(FAKE, 64, 0, 1.0, 0)
    for name, x in kw.items():
        setattr(t, name, x)
    return t


def _rotary(lib, desc=None, table=None, count=1, x=(FAKE,), y=(2 * FAKE,), heads=(2,), strides=None,
            positions=FAKE, step=0):
    desc = ops.make_desc(1, 2, 4, 64, ops.BF16, True, 0, 0.0, 0.0) if desc is None else desc
    n = len(x)
    return lib.diffrotary_apply(ctypes.byref(desc), ctypes.byref(_table() if table is None else table),
                                count, (ctypes.c_void_p * n)(*x), (ctypes.c_void_p * n)(*y),
                                (ctypes.c_int64 * n)(*heads), strides, positions, step, 0, 0, None)


def test_rotary_refused(lib):
    d = lambda **k: ops.make_desc(*[k.get(n, v) for n, v in dict(
        B=1, H=2, N=4, d=64, dtype=ops.BF16, causal=True, headnorm=0, eps=0.0, li=0.0).items()])
    assert lib.diffrotary_apply(None, None, 1, None, None, None, None, None, 0, 0, 0, None) == I
    assert _rotary(lib, d(d=32)) == U
    assert _rotary(lib, d(dtype=ops.E4M3_QK)) == U
    assert _rotary(lib, d(B=-1)) == I
    assert _rotary(lib, d(B=1 << 20, N=1 << 11)) == U
    for bad in (dict(rot=0), dict(rot=24), dict(rot=80), dict(freq=0), dict(freq=FAKE + 4),
                dict(neighbours=2), dict(reserved=1)):
        assert _rotary(lib, table=_table(**bad)) == I, bad
    assert _rotary(lib, count=0) == I
    assert _rotary(lib, count=5, x=(FAKE,) * 5, y=(2 * FAKE,) * 5, heads=(1,) * 5) == I
    assert _rotary(lib, x=(0,)) == I
    assert _rotary(lib, x=(FAKE + 8,)) == I
    assert _rotary(lib, y=(FAKE + 2,)) == I
    assert _rotary(lib, heads=(-1,)) == I
    assert _rotary(lib, positions=FAKE + 2) == I
    assert _rotary(lib, step=-1) == I
    for s in (ops.Strides(512, 256, 60), ops.Strides(512, 0, 64), ops.Strides(1 << 39, 256, 64)):
        both = (ops.Strides * 2)(s, ops.Strides(512, 256, 64))
        assert _rotary(lib, strides=both) == I
    uneven = (ops.Strides * 2)(ops.Strides(512, 256, 64), ops.Strides(1024, 256, 64))
    assert _rotary(lib, y=(FAKE,), strides=uneven) == I  # in place, other strides
    assert _rotary(lib, d(N=0)) == ops.OK
    assert _rotary(lib, x=(0,), y=(0,), heads=(0,)) == ops.OK


# ---- packed batches ---------------------------------------------------------------------------

def _book(**kw):
    b = ops.PageBookStruct(FAKE, FAKE, FAKE, FAKE, FAKE, 2, 4, 8, 16, 0)
    for name, x in kw.items():
        setattr(b, name, x)
    return b


def _step(lib, book, new=FAKE, n=8, q=FAKE, pos=FAKE, slots=FAKE, status=FAKE):
    return lib.diffragged_step(ctypes.byref(book) if book else None, new, n, q, pos, slots, status,
                               None)


def test_step_refused(lib):
    assert _step(lib, None) == I
    for bad in (dict(kv_len=0), dict(held=0), dict(page_table=0), dict(free_pages=0),
                dict(free_count=0), dict(kv_len=FAKE + 2), dict(page_table=FAKE + 1), dict(B=-1),
                dict(max_pages=0), dict(capacity=-1), dict(page_size=0), dict(reserved=1)):
        assert _step(lib, _book(**bad)) == I, bad
    for bad in (dict(new=0), dict(q=0), dict(q=FAKE + 2), dict(pos=FAKE + 2), dict(slots=FAKE + 4),
                dict(status=FAKE + 1), dict(n=-1)):
        assert _step(lib, _book(), **bad) == I, bad
    for bad in (dict(B=1 << 24), dict(max_pages=1 << 26), dict(capacity=(1 << 30) + 1)):
        assert _step(lib, _book(**bad)) == U, bad
    assert _step(lib, _book(), n=(1 << 30) + 1) == U


def _cache(heads=2, d=64, page=16, pages=8, max_pages=64, **kw):
    st = lambda w: ops.Strides(heads * page * w, page * w, w)
    c = ops.PagedCacheStruct(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, st(d), st(d), st(2 * d), pages,
                             heads, max_pages, page, 0)
    for name, x in kw.items():
        setattr(c, name, x)
    return c


def _desc(B=1, H=4, N=3, d=64, dtype=ops.BF16, headnorm=1, eps=1e-5):
    return ops.make_desc(B, H, N, d, dtype, True, headnorm, eps, 0.0)


def _append(lib, desc=None, cache=None, q=(FAKE, FAKE), kv=(FAKE,) * 3, out=(2 * FAKE, 3 * FAKE),
            strides=None, slots=FAKE, table=None, positions=FAKE):
    return lib.diffragged_append(ctypes.byref(desc or _desc()), ctypes.byref(cache or _cache()), *q,
                                 *kv, *out, strides, slots, table, positions, None)


def _fwd(lib, desc=None, cache=None, q_start=FAKE, ptrs=(FAKE,) * 5, strides=None, ws=FAKE,
         nbytes=1 << 40):
    return lib.diffragged_fwd(ctypes.byref(desc or _desc()), ctypes.byref(cache or _cache()), q_start,
                              *ptrs, strides, ws, nbytes, None)


@pytest.mark.parametrize("call", [_append, _fwd])
def test_descriptor_and_cache_refused(lib, call):
    assert lib.diffragged_fwd(None, None, None, None, None, None, None, None, None, None, 0,
                              None) == I
    assert lib.diffragged_append(None, None, *(None,) * 12) == I
    for bad in (dict(k1=0), dict(v=FAKE + 8), dict(page_size=-16), dict(kv_heads=3),
                dict(k2_strides=ops.Strides(2048, 1024, 60))):
        assert call(lib, cache=_cache(**bad)) == I, bad
    assert call(lib, _desc(H=3)) == I
    assert call(lib, _desc(N=-1)) == I
    assert call(lib, _desc(dtype=ops.F32)) == U
    assert call(lib, _desc(d=32)) == U
    assert call(lib, cache=_cache(page_size=24)) == U
    assert call(lib, _desc(N=0)) == ops.OK


def test_append_refused(lib):
    assert _append(lib, kv=(FAKE, 0, FAKE)) == I
    assert _append(lib, kv=(FAKE, FAKE, FAKE + 8)) == I
    assert _append(lib, q=(FAKE, 0)) == I
    assert _append(lib, q=(0, 0)) == I            # outputs without inputs
    assert _append(lib, out=(2 * FAKE, 0)) == I
    assert _append(lib, out=(2 * FAKE, 2 * FAKE + 8)) == I
    assert _append(lib, slots=0) == I
    assert _append(lib, slots=FAKE + 4) == I
    t = _table()
    assert _append(lib, table=ctypes.byref(t), positions=0) == I
    assert _append(lib, table=ctypes.byref(t), positions=FAKE + 2) == I
    assert _append(lib, table=ctypes.byref(_table(rot=128))) == I
    good = ops.Strides(0, 64, 256)
    for i in (0, 2, 4, 6):
        st = [good] * 7
        st[i] = ops.Strides(0, 60, 256)
        assert _append(lib, strides=(ops.Strides * 7)(*st)) == I
    apart = [good] * 5 + [ops.Strides(0, 64, 512), good]
    assert _append(lib, out=(FAKE, 3 * FAKE), strides=(ops.Strides * 7)(*apart)) == I  # in place
    e4m3 = _desc(dtype=ops.E4M3_QK)
    assert _append(lib, e4m3, _cache(k1_strides=ops.Strides(2048, 1024, 64),
                                     k2_strides=ops.Strides(2048, 1024, 64)), out=(FAKE, FAKE)) == I


def test_fwd_refused(lib):
    for k in range(5):
        if k == 3:
            continue  # norm_w may be NULL
        ptrs = [FAKE] * 5
        ptrs[k] = 0
        assert _fwd(lib, ptrs=ptrs) == I, k
    for k, x in ((0, FAKE + 8), (1, FAKE + 2), (2, FAKE + 2), (3, FAKE + 4), (4, FAKE + 8)):
        ptrs = [FAKE] * 5
        ptrs[k] = x
        assert _fwd(lib, ptrs=ptrs) == I, k
    assert _fwd(lib, q_start=0) == I
    assert _fwd(lib, q_start=FAKE + 2) == I
    assert _fwd(lib, _desc(H=2 * 65)) == U
    bad = (ops.Strides * 3)(ops.Strides(0, 64, 256), ops.Strides(0, 64, 256), ops.Strides(0, 4, 512))
    assert _fwd(lib, strides=bad) == I
    big = _cache(page=1 << 20, max_pages=1, heads=2)
    assert _fwd(lib, _desc(N=1 << 29), big) == U   # more steps than 31 bits
    n = ctypes.c_size_t(0)
    assert lib.diffragged_fwd_plan(ctypes.byref(_desc()), ctypes.byref(_cache()), None) == I
    st = lib.diffragged_fwd_plan(ctypes.byref(_desc()), ctypes.byref(_cache()), ctypes.byref(n))
    if st == ops.OK:  # a device to ask for its SMs
        assert n.value > 0
        assert _fwd(lib, ws=0) == I
        assert _fwd(lib, ws=FAKE + 16) == I
        assert _fwd(lib, nbytes=n.value - 1) == I
    else:
        assert st == ops.ERR_CUDA


def test_what_other_kernels_write_is_not_read_through_the_read_only_path():
    """Lengths, tables, positions, slots and rows may come from a kernel that is still running when
    these start (dependent launch): ld.global.nc, which __ldg is, must not read them."""
    files = glob.glob(os.path.join(libbuild.CSRC, "ragged*")) + \
        glob.glob(os.path.join(libbuild.CSRC, "rotary*"))
    assert len(files) >= 8
    for path in files:
        assert "__ldg(" not in open(path).read(), path


# ---- the binding's own checks -----------------------------------------------------------------

def _without_a_device(cls, **fields):
    """An object of the binding as far as its checks of arguments go: they come before any launch,
    and a tensor without a device has the index -1."""
    x = cls.__new__(cls)
    for name, value in dict(fields, index=-1, device=torch.device("cpu"), _calls={}, _ref=None).items():
        setattr(x, name, value)
    return x


def test_first_rotary_call_with_wrong_outputs_names_them():
    x = torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16)
    for outs in ([], [x], [x] * 3, [x[0], x[0]], [x[0, 0, 0], x], [x, x[..., None]]):
        table = _without_a_device(ops.RotaryTable)
        with pytest.raises(ValueError, match="outs must be as many tensors of the inputs' shapes"):
            ops.rotary(table, [x, x], outs=outs)
        assert not table._calls


def _cache_without_a_device():
    return _without_a_device(ops.PagedCache, dtype=torch.bfloat16, kv_heads=2, d=64, B=1,
                             code=ops.BF16)


def test_first_append_with_wrong_queries_or_outputs_names_them():
    k, v, q = (torch.zeros(3, h, w, dtype=torch.bfloat16) for h, w in ((2, 64), (2, 128), (4, 64)))
    slots = torch.zeros(3, dtype=torch.int64)
    for kw in (dict(q=(q,)), dict(q=(q, q, q)), dict(q=(q, q), q_out=(q,)),
               dict(q=(q, q), q_out=[q] * 3), dict(q=()), dict(q_out=(q, q))):
        with pytest.raises(ValueError, match="q_out"):
            ops.ragged_append(_cache_without_a_device(), k, k, v, slots, **kw)
    for kw in (dict(q=(q, q), q_out=(q, q[0])), dict(q=(q, q[0])), dict(q=(q[0], q[0]))):
        with pytest.raises(ValueError, match="must be"):
            ops.ragged_append(_cache_without_a_device(), k, k, v, slots, **kw)


def test_first_forward_with_an_output_of_other_axes_names_it():
    q, lam = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(4)
    for shape in ((3, 512), (1536,), (1, 3, 4, 128), (3, 4, 64), (4, 4, 128)):
        with pytest.raises(ValueError, match="out must be"):
            ops.ragged_fwd(_cache_without_a_device(), q, q, lam, torch.zeros(2, dtype=torch.int32),
                           out=torch.zeros(shape, dtype=torch.bfloat16))
