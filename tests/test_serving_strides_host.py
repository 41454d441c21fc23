"""Strides that the binding passes on for the rotation's and the append's tensors (CPU only)."""
import itertools
import random

import pytest
import torch

from sparse_head_latent_b200.mla import _rows_and_heads


def _elements(t, lead):
    """Offsets of a tensor's elements as (row, head, e), by its own strides."""
    width = t.shape[-1]
    t = t.reshape(-1, 1, width) if t.dim() == lead + 1 else t.reshape(-1, t.shape[-2], width)
    return t


def _check(t, lead):
    storage = torch.arange(t.untyped_storage().nbytes() // 8, dtype=torch.int64)
    assert storage.data_ptr() != t.data_ptr()
    rows, row, heads, head = _rows_and_heads(t, t.shape, lead)
    want = _elements(t, lead)
    assert (rows, heads) == (want.shape[0], want.shape[1])
    base = t.storage_offset()
    for r, h in itertools.product(range(rows), range(heads)):
        at = base + r * row + h * head
        assert torch.equal(want[r, h], storage[at:at + t.shape[-1]])
    assert row % 8 == 0 and head % 8 == 0  # as the library wants them
    return rows, heads


def test_views_with_aligned_rows_are_taken_as_they_are():
    # values are their own offsets in the storage
    base = torch.arange(6 * 4 * 3 * 576, dtype=torch.int64)
    rng = random.Random(0)
    kv = base.view(72, 576)
    for t, lead in ((kv[:, 512:], 1), (kv[:, None, 512:], 1), (kv[:, 512:, None].transpose(1, 2), 1),
                    (kv[::2, 512:].unsqueeze(1), 1), (kv.view(6, 12, 576)[:, :, :64], 2), (kv[3, 512:], 0),
                    (kv[3:4, 512:, None].transpose(1, 2), 1), (kv.view(6, 12, 1, 576)[..., 64:128], 2),
                    (kv.view(72, 3, 192)[:, 1:2], 1), (kv.view(72, 3, 192)[:, :, 128:], 1),
                    (kv.view(72, 3, 192).transpose(0, 1)[1, :, 128:], 1), (kv.view(72, 3, 192)[::5, 1:], 1),
                    (kv.view(6, 12, 576)[:1, :, :64], 2), (kv.view(6, 12, 576)[:, :1, 64:], 2)):
        assert _check(t, lead)[0] == t.shape[:lead].numel()
    for _ in range(50):
        heads, width = rng.choice([1, 1, 2, 3]), rng.choice([64, 128, 192])
        t = kv.view(72, 3, 192)[rng.randrange(3)::rng.choice([1, 2, 7]), :heads, :width]
        _check(t, 1)


def test_leading_dimensions_that_do_not_fold_are_refused():
    kv = torch.arange(72 * 576).view(6, 12, 576)
    with pytest.raises(ValueError, match="fold"):
        _rows_and_heads(kv[:, ::5, :64], (6, 3, 64), 2)
    with pytest.raises(ValueError, match="contiguous"):
        _rows_and_heads(kv[..., ::2], (6, 12, 288), 2)
