"""More refusals of the paged-serving calls (CPU only; answered before the first CUDA call)."""
import pytest

import sparse_head_latent_b200 as mla
from test_serving_host import OK, UNSUPPORTED, WORKSPACE, _tree, lib  # noqa: F401


@pytest.mark.parametrize("topk", [1, 40, 2048, -1])
def test_tree_decode_refuses_a_selection_it_would_not_make(lib, topk):  # noqa: F811
    dims = mla.make_dims(2, 4, 3, topk)
    assert mla.mla_workspace_bytes(dims, mla.MLA_ENTRY_TREE_DECODE, False) == 0
    assert _tree(lib, dims) == UNSUPPORTED
    assert _tree(lib, mla.make_dims(0, 4, 3, topk)) == OK  # nothing to attend to
    assert _tree(lib, mla.make_dims(2, 4, 3, 0, path=mla.MLA_PATH_ABSORBED)) == WORKSPACE  # the path is ignored
