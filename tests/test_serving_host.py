"""Host checks of the paged-serving calls and the rotary table (CPU only).

Every refused call below is answered before the first CUDA call, so the
placeholder pointers are never used."""
import ctypes
import math
import re

import pytest
import torch

import sparse_head_latent_b200 as mla
from sparse_head_latent_b200 import build as cuda_build
from sparse_head_latent_b200.mla import MlaPages, MlaRopeTable
from test_abi import HEADER

OK, NULL, SHAPE, UNSUPPORTED, WORKSPACE, ALIGN = 0, 1, 2, 3, 4, 6


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return mla.load_library()


def _frequencies(base, scaling, factor=1.0, original_len=4096, fast=32.0, slow=1.0):
    out = []
    dim = lambda b: 64 * math.log(original_len / (2 * math.pi * b)) / (2 * math.log(base))  # noqa: E731
    for i in range(32):
        f = base ** (-2.0 * i / 64)
        if scaling == mla.MLA_ROPE_LINEAR:
            f /= factor
        elif scaling == mla.MLA_ROPE_YARN:
            lo, hi = max(math.floor(dim(fast)), 0), min(math.ceil(dim(slow)), 63)
            r = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
            f = f * (1 - r) + f / factor * r
        out.append(f)
    return out


@pytest.mark.parametrize("base,scaling,factor,original", [
    (10000.0, mla.MLA_ROPE_UNSCALED, 1.0, 4096), (1.5, mla.MLA_ROPE_UNSCALED, 1.0, 4096),
    (10000.0, mla.MLA_ROPE_LINEAR, 4.0, 4096), (10000.0, mla.MLA_ROPE_YARN, 40.0, 4096),
    (50000.0, mla.MLA_ROPE_YARN, 32.0, 4096), (10000.0, mla.MLA_ROPE_YARN, 1.0, 4096),
    (10000.0, mla.MLA_ROPE_YARN, 8.0, 3)])
def test_rope_table_holds_the_frequencies_as_turns(lib, base, scaling, factor, original):
    t = mla.make_rope(base=base, scaling=scaling, factor=factor, original_len=original)
    for turns, f in zip(t.turns, _frequencies(base, scaling, factor, original)):
        # f is a double (relative error 2^-53 in each of a few operations)
        assert abs(turns / 2.0 ** 64 * 2 * math.pi - f) <= 8 * 2.0 ** -53 * f + 2.0 ** -62
    assert t.magnitude == 1.0 and t.layout == mla.MLA_ROPE_INTERLEAVED


def test_rope_table_refusals(lib):
    t = MlaRopeTable()

    def init(layout=0, base=1e4, scaling=2, factor=4.0, original=4096.0, fast=32.0, slow=1.0, magnitude=1.0):
        return lib.mla_rope_init(ctypes.byref(t), layout, base, scaling, factor, original, fast, slow, magnitude)

    assert init() == OK
    assert lib.mla_rope_init(None, 0, 1e4, 0, 1.0, 1.0, 1.0, 1.0, 1.0) == NULL
    assert init(layout=2) == UNSUPPORTED and init(scaling=3) == UNSUPPORTED
    for bad in (dict(base=1.0), dict(base=0.0), dict(base=float("inf")), dict(base=float("nan")),
                dict(factor=0.5), dict(factor=float("nan")), dict(original=0.0), dict(slow=0.0),
                dict(fast=0.5), dict(magnitude=float("inf"))):
        assert init(**bad) == SHAPE, bad
    assert init(scaling=0, factor=0.0, original=0.0, fast=0.0, slow=0.0) == OK  # ignored when unscaled
    with pytest.raises(mla.MlaError):
        mla.make_rope(base=0.5)


def _rope(lib, table, **kw):
    a = dict(x=16, xr=768, xh=192, out=32, outr=768, outh=192, rows=2, heads=4, width=192, offset=128, pos=16, inv=0)
    a.update(kw)
    return lib.mla_rope(None if table is None else ctypes.byref(table), a["x"], a["xr"], a["xh"], a["out"], a["outr"],
                        a["outh"], a["rows"], a["heads"], a["width"], a["offset"], a["pos"], a["inv"], None)


def test_rope_refusals(lib):
    t = mla.make_rope()
    assert _rope(lib, None) == NULL
    for kw in (dict(x=None), dict(out=None), dict(pos=None)):
        assert _rope(lib, t, **kw) == NULL
    for kw in (dict(rows=-1), dict(heads=-1), dict(width=56), dict(width=196), dict(width=2056), dict(offset=-8),
               dict(offset=4), dict(offset=136), dict(inv=2), dict(xr=100), dict(outh=65)):
        assert _rope(lib, t, **kw) == SHAPE, kw
    for kw in (dict(x=24), dict(out=8), dict(pos=18)):
        assert _rope(lib, t, **kw) == ALIGN
    assert _rope(lib, t, rows=0, x=None, out=None, pos=None) == OK
    assert _rope(lib, t, heads=0) == OK
    bad = mla.make_rope()
    bad.layout = 5
    assert _rope(lib, bad) == UNSUPPORTED


def _append(lib, table, **kw):
    a = dict(kv=16, stride=576, w=16, f32=0, eps=1e-6, pos=16, slots=None, rows=3, cache=16, pe=16, n=64)
    a.update(kw)
    return lib.mla_cache_append(None if table is None else ctypes.byref(table), a["kv"], a["stride"], a["w"],
                                a["f32"], a["eps"], a["pos"], a["slots"], a["rows"], a["cache"], a["pe"], a["n"], None)


def test_append_refusals(lib):
    t = mla.make_rope()
    assert _append(lib, None) == NULL
    for k in ("kv", "w", "pos", "cache", "pe"):
        assert _append(lib, t, **{k: None}) == NULL
    for kw in (dict(rows=-1), dict(stride=568), dict(stride=577), dict(eps=-1.0), dict(eps=float("nan")),
               dict(f32=2), dict(n=-1)):
        assert _append(lib, t, **kw) == SHAPE, kw
    for kw in (dict(kv=8), dict(w=24), dict(cache=8), dict(pe=8), dict(pos=17), dict(slots=2)):
        assert _append(lib, t, **kw) == ALIGN
    assert _append(lib, t, rows=0, kv=None) == OK
    assert _append(lib, t, n=0, cache=None, pe=None) == OK


def _pages(**kw):
    p = dict(num_pages=8, page_size=64, table_width=4, layers=1)
    p.update(kw)
    return MlaPages(p["num_pages"], p["page_size"], p["table_width"], p["layers"])


BAD_PAGES = (dict(page_size=0), dict(page_size=8), dict(page_size=48), dict(page_size=-16), dict(num_pages=-1),
             dict(num_pages=1 << 30), dict(layers=0), dict(layers=70000))


def _tree(lib, dims=None, pages=None, **kw):
    a = dict(q=16, kv=16, pe=16, table=16, n0=16, nodes=None, parents=None, w=16, ws=None, o=16, os=None, scale=0.07,
             out=16, work=None, nbytes=0)
    a.update(kw)
    d = dims if dims is not None else mla.make_dims(2, 4, 3)
    p = pages if pages is not None else _pages()
    return lib.mla_tree_decode(ctypes.byref(d), ctypes.byref(p), a["q"], a["kv"], a["pe"], a["table"], a["n0"],
                               a["nodes"], a["parents"], a["w"], a["ws"], a["o"], a["os"],
                               ctypes.c_float(a["scale"]), a["out"], a["work"], a["nbytes"], None)


def test_tree_decode_refusals(lib):
    assert _tree(lib, mla.make_dims(2, 65, 3)) == SHAPE
    assert _tree(lib, mla.make_dims(2, -1, 3)) == SHAPE
    assert _tree(lib, mla.make_dims(2, 4, 0)) == SHAPE
    d = mla.make_dims(2, 4, 3)
    d.d_latent = 256
    assert _tree(lib, d) == UNSUPPORTED
    for bad in BAD_PAGES + (dict(table_width=0), dict(table_width=1 << 30), dict(layers=2), dict(num_pages=0)):
        assert _tree(lib, pages=_pages(**bad)) == SHAPE, bad
    for k in ("q", "kv", "pe", "table", "n0", "w", "o", "out"):
        assert _tree(lib, **{k: None}) == NULL, k
    d8 = mla.make_dims(2, 4, 3, 0, True)
    assert _tree(lib, d8) == NULL and _tree(lib, d8, ws=16) == NULL
    for k in ("q", "kv", "pe", "w", "o", "out"):
        assert _tree(lib, **{k: 24}) == ALIGN, k
    for k in ("table", "n0", "nodes", "parents"):
        assert _tree(lib, **{k: 18}) == ALIGN, k
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert _tree(lib, scale=s) == SHAPE
    act8 = mla.make_dims(2, 4, 3, 0, True, act=mla.MLA_ACT_E4M3_DYNAMIC)
    assert _tree(lib, act8, ws=16, os=16) == UNSUPPORTED
    need = mla.mla_workspace_bytes(mla.make_dims(2, 4, 3), mla.MLA_ENTRY_TREE_DECODE, False)
    assert need > 0
    assert _tree(lib) == WORKSPACE and _tree(lib, work=16, nbytes=need - 1) == WORKSPACE
    assert _tree(lib, work=24, nbytes=need) == ALIGN
    assert _tree(lib, mla.make_dims(0, 4, 3), q=None) == OK
    assert _tree(lib, mla.make_dims(2, 0, 3), q=None) == OK
    assert lib.mla_tree_decode(ctypes.byref(mla.make_dims(2, 4, 3)), None, 16, 16, 16, 16, 16, None, None, 16, None, 16,
                               None, ctypes.c_float(0.1), 16, None, 0, None) == NULL
    assert mla.mla_workspace_bytes(mla.make_dims(2, 65, 3), mla.MLA_ENTRY_TREE_DECODE, False) == 0
    assert mla.mla_workspace_bytes(act8, mla.MLA_ENTRY_TREE_DECODE, False) == 0


def _compact(lib, pages=None, **kw):
    a = dict(kv=16, pe=16, table=16, n0=16, acc=16, cnt=16, B=2, width=4)
    a.update(kw)
    return lib.mla_cache_compact(ctypes.byref(pages or _pages()), a["kv"], a["pe"], a["table"], a["n0"], a["acc"],
                                 a["cnt"], a["B"], a["width"], None)


def test_compact_refusals(lib):
    for bad in BAD_PAGES + (dict(table_width=0),):
        assert _compact(lib, _pages(**bad)) == SHAPE, bad
    for kw in (dict(B=-1), dict(width=-1), dict(width=65)):
        assert _compact(lib, **kw) == SHAPE
    for k in ("kv", "pe", "table", "n0", "acc", "cnt"):
        assert _compact(lib, **{k: None}) == NULL
    for kw in (dict(kv=8), dict(pe=8), dict(table=2), dict(n0=2), dict(acc=2), dict(cnt=2)):
        assert _compact(lib, **kw) == ALIGN
    assert _compact(lib, B=0, kv=None) == OK and _compact(lib, width=0, kv=None) == OK
    assert lib.mla_cache_compact(None, 16, 16, 16, 16, 16, 16, 1, 1, None) == NULL


def _copy(lib, src, dst, pages=None, kv=16, pe=16):
    n = len(src)
    return lib.mla_cache_copy_pages(ctypes.byref(pages or _pages(num_pages=300)), kv, pe, (ctypes.c_int32 * n)(*src),
                                    (ctypes.c_int32 * n)(*dst), n, None)


@pytest.mark.parametrize("more", [0, 100])
def test_copy_refusals(lib, more):
    # a few pairs and many are checked in different ways
    s, d = list(range(100, 100 + more)), list(range(200, 200 + more))
    assert _copy(lib, [1, 2] + s, [3, 3] + d) == SHAPE        # a destination twice
    assert _copy(lib, [1, 3] + s, [3, 4] + d) == SHAPE        # a destination that another pair reads
    assert _copy(lib, [1, 3] + s, [3, 3] + d) == SHAPE        # ... by the pair that copies onto itself
    assert _copy(lib, [1, 1] + s, [1, 2] + d) == SHAPE
    assert _copy(lib, [-1] + s, [3] + d) == SHAPE and _copy(lib, [1] + s, [300] + d) == SHAPE
    assert _copy(lib, [1] + s, [-1] + d) == SHAPE and _copy(lib, [300] + s, [1] + d) == SHAPE
    assert _copy(lib, [1] + s, [2] + d, kv=None) == NULL and _copy(lib, [1] + s, [2] + d, pe=8) == ALIGN
    for bad in BAD_PAGES:
        assert _copy(lib, [1], [2], _pages(**bad)) == SHAPE
    assert _copy(lib, [], []) == OK
    assert lib.mla_cache_copy_pages(ctypes.byref(_pages()), 16, 16, None, None, 1, None) == NULL
    assert lib.mla_cache_copy_pages(ctypes.byref(_pages()), 16, 16, None, None, -1, None) == SHAPE


def test_structs_match_the_header():
    src = open(HEADER).read()
    for name, struct in (("mla_pages", MlaPages), ("mla_rope_table", MlaRopeTable)):
        body = re.search(r"typedef struct \{([^}]*)\} %s;" % name, src).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        assert re.findall(r"\b([a-z_]+)(?:\[\d+\])?\s*;", body) == [f[0] for f in struct._fields_]
    assert ctypes.sizeof(MlaRopeTable) == 32 * 8 + 8 and ctypes.sizeof(MlaPages) == 16
    assert int(re.search(r"#define MLA_MAX_TREE (\d+)", src).group(1)) == mla.MLA_MAX_TREE


def test_binding_checks_shapes_types_and_devices(lib):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    rope = mla.make_rope()
    with pytest.raises(ValueError, match="CUDA"):
        mla.mla_rope(bf(2, 3, 192), i32(2), rope)
    with pytest.raises(ValueError, match="int32"):
        mla.mla_rope(bf(2, 3, 192), torch.zeros(2, dtype=torch.int64), rope)
    with pytest.raises(ValueError, match="bfloat16"):
        mla.mla_rope(torch.zeros(2, 3, 192), i32(2), rope)
    with pytest.raises(ValueError, match="positions"):
        mla.mla_rope(bf(2, 3, 192), i32(3), rope)
    with pytest.raises(ValueError, match="fold"):
        mla.mla_rope(bf(4, 2, 3, 192).transpose(0, 1), i32(2, 4), rope)
    with pytest.raises(ValueError, match="contiguous"):
        mla.mla_rope(bf(2, 192, 3).transpose(1, 2), i32(2), rope)
    with pytest.raises(ValueError, match="576"):
        mla.mla_cache_append(bf(2, 512), bf(512), i32(2), rope, bf(4, 512), bf(4, 64))
    with pytest.raises(ValueError, match="norm_weight"):
        mla.mla_cache_append(bf(2, 576), bf(500), i32(2), rope, bf(4, 512), bf(4, 64))
    with pytest.raises(ValueError, match="rows"):
        mla.mla_cache_append(bf(2, 576), bf(512), i32(2), rope, bf(4, 512), bf(5, 64))
    with pytest.raises(ValueError, match="fewer"):
        mla.mla_cache_append(bf(5, 576), bf(512), i32(5), rope, bf(4, 512), bf(4, 64))
    kv, pe = bf(4, 16, 512), bf(4, 16, 64)
    w, o = bf(2 * 256, 512), bf(2 * 128, 7168)
    ok = dict(q=bf(1, 3, 2, 192), kv_cache=kv, k_pe_cache=pe, block_table=i32(1, 4), cache_len=i32(1), W_kvb=w, W_o=o)
    for name, value in (("q", bf(1, 3, 2, 128)), ("q", bf(3, 2, 192)), ("kv_cache", bf(2, 4, 16, 512)),
                        ("k_pe_cache", bf(4, 8, 64)), ("block_table", i32(2, 4)), ("cache_len", i32(2)),
                        ("parents", i32(1, 2)), ("n_nodes", i32(3)), ("W_kvb", bf(256, 512)), ("W_o", bf(256, 7167)),
                        ("block_table", torch.zeros(1, 4, dtype=torch.int64)), ("out", bf(1, 3, 7167))):
        with pytest.raises(ValueError):
            mla.mla_tree_decode(**{**ok, name: value})
    with pytest.raises(ValueError, match="CUDA"):
        mla.mla_tree_decode(**ok)
    with pytest.raises(ValueError, match="length"):
        mla.mla_cache_copy_pages(kv, pe, [1, 2], [3])
    with pytest.raises(OverflowError):
        mla.mla_cache_copy_pages(kv, pe, [1 << 32], [3])
    with pytest.raises(ValueError):
        mla.mla_cache_compact(kv, pe, i32(1, 4), i32(1), i32(2, 3), i32(1))
