"""Lists of mla_cache_copy_pages (needs a B200): what the check of the list lets through is copied."""
import random

import pytest
import torch

mla = pytest.importorskip("sparse_head_latent_b200")

from test_gpu_parity import _no_device_error  # noqa: E402
from test_gpu_tree import _caches  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 2, 3, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300])
def test_lists_without_a_clash_are_copied(n):
    rng = random.Random(n)
    for tight in (False, True):
        pages = 2 * n if tight else 3 * n + 50
        kv, pe = _caches(2, pages, 16, seed=n)
        order = rng.sample(range(pages), 2 * n)
        dst, src = order[:n], [rng.choice(order[n:]) for _ in range(n)]
        if n > 3:
            src[n // 2] = dst[n // 2]  # onto itself: nothing
        want = [c.clone() for c in (kv, pe)]
        for w, c in zip(want, (kv, pe)):
            w[:, dst] = c[:, src]
        mla.mla_cache_copy_pages(kv, pe, src, dst)
        _no_device_error()
        assert torch.equal(kv, want[0]) and torch.equal(pe, want[1])


def test_every_page_onto_itself():
    kv, pe = _caches(None, 200, 16)
    want = kv.clone(), pe.clone()
    mla.mla_cache_copy_pages(kv, pe, list(range(200)), list(range(200)))
    _no_device_error()
    assert torch.equal(kv, want[0]) and torch.equal(pe, want[1])
