"""More refusals of the paged-serving calls (CPU only; answered before the first CUDA call)."""
import array
import ctypes
import random
import time

import pytest
import torch

import sparse_head_latent_b200 as mla
from sparse_head_latent_b200 import mla as binding
from test_serving_host import OK, SHAPE, UNSUPPORTED, WORKSPACE, _copy, _pages, _tree, lib  # noqa: F401


@pytest.mark.parametrize("topk", [1, 40, 2048, -1])
def test_tree_decode_refuses_a_selection_it_would_not_make(lib, topk):  # noqa: F811
    dims = mla.make_dims(2, 4, 3, topk)
    assert mla.mla_workspace_bytes(dims, mla.MLA_ENTRY_TREE_DECODE, False) == 0
    assert _tree(lib, dims) == UNSUPPORTED
    assert _tree(lib, mla.make_dims(0, 4, 3, topk)) == OK  # nothing to attend to
    assert _tree(lib, mla.make_dims(2, 4, 3, 0, path=mla.MLA_PATH_ABSORBED)) == WORKSPACE  # the path is ignored


def _arrays(src, dst):
    n = len(src)
    return (ctypes.c_int32 * n)(*src), (ctypes.c_int32 * n)(*dst), n


def test_copy_check_grows_with_the_list_and_not_with_the_pool(lib):  # noqa: F811
    src, dst = list(range(65)), list(range(100, 164)) + [100]  # a destination twice, found last
    args = (*_arrays(src, dst), None)
    pages = _pages(num_pages=1 << 26, page_size=16)
    took = []
    for _ in range(3):
        t0 = time.perf_counter()
        assert lib.mla_cache_copy_pages(ctypes.byref(pages), 16, 16, *args) == SHAPE
        took.append(time.perf_counter() - t0)
    assert min(took) < 5e-3  # one mark per page is 256 MB to fill


@pytest.mark.parametrize("n", [1, 2, 3, 33, 63, 64, 65, 66, 200, 1000])
def test_copy_refuses_lists_that_clash(lib, n):  # noqa: F811
    # only lists that clash are given to the call here: another would go on to the device
    rng = random.Random(n)
    for i in range(60):
        pool = rng.choice([2 * n + 2, 5 * n, 1 << 20])
        order = rng.sample(range(pool), 2 * n + 1)
        src, dst = order[:n], order[n:2 * n]
        kind = i % 6
        a, b = rng.randrange(n), rng.randrange(n)
        if kind == 1:  # a source several times
            src[a] = src[b]
        elif kind == 2:  # onto itself
            src[a] = dst[a]
        elif kind == 3:
            dst[a] = dst[b]
        elif kind == 4:
            src[a] = dst[b]
        elif kind == 5:  # onto itself, and read by another
            src[a] = dst[a]
            src[b] = dst[a]
        clash = len(set(dst)) < n or any(s == d for i, s in enumerate(src) for j, d in enumerate(dst) if i != j and s == d)
        if not clash:
            continue
        assert _copy(lib, src, dst, _pages(num_pages=pool, page_size=16)) == SHAPE
    if n > 1:  # more pairs than pages have a destination twice
        assert _copy(lib, [0] * n, [0] * n, _pages(num_pages=n - 1, page_size=16)) == SHAPE


def test_copy_reads_as_many_indexes_as_its_lists_hold(lib, monkeypatch):  # noqa: F811
    # the addresses and the length that reach the library, with no device: a list may be any sequence of ints
    seen = []

    def call(name, index, stream, args):
        n = args[5]
        seen.append([list((ctypes.c_int32 * n).from_address(a)) if n else [] for a in args[3:5]])

    monkeypatch.setattr(binding, "_call", call)
    monkeypatch.setattr(binding, "_cuda", lambda t: 0)
    monkeypatch.setattr(binding, "_data", lambda t, index: t.data_ptr())
    kv, pe = torch.zeros(4, 16, 512, dtype=torch.bfloat16), torch.zeros(4, 16, 64, dtype=torch.bfloat16)
    for src, dst in (([0, 1], [2, 3]), (range(2), (2, 3)), (torch.tensor([0, 1]), torch.tensor([2, 3], dtype=torch.int32)),
                     (array.array("i", [0, 1]), array.array("q", [2, 3])), (torch.arange(4)[::2] // 2, [2, 3])):
        mla.mla_cache_copy_pages(kv, pe, src, dst)
        assert seen.pop() == [[0, 1], [2, 3]]
    mla.mla_cache_copy_pages(kv, pe, [], [])
    assert seen.pop() == [[], []]
    for src, dst in ((bytes(8), [2, 3]), (bytes(8), bytes(8)), (bytearray(8), [1] * 8), ([0, 1], bytes(2)), ([0], [1, 2]),
                     (bytes(4), [2])):
        with pytest.raises(ValueError):
            mla.mla_cache_copy_pages(kv, pe, src, dst)
    assert not seen


def test_withhold_hook_takes_its_values_only(lib):  # noqa: F811
    for bad in (-1, 1 << 30):
        assert lib.mla_test_withhold_attention_loads(bad) == SHAPE
