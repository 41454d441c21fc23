"""Waits that run out in the serving kernels, without a fault (needs a B200).

With the test hook on, a producer stops issuing loads after a first block or tile, so that products are under way in
some CTAs when the waits for the next ones reach the time limit, lowered to 2 ms. The call has to return, the error word to hold
a 1xx code, and the next call to give what it gave before, bit for bit."""
import time

import pytest
import torch

mla = pytest.importorskip("sparse_head_latent_b200")

from test_gpu_parity import _no_device_error  # noqa: E402
from test_gpu_tree import Problem  # noqa: E402

pytestmark = pytest.mark.gpu

TREE, FEW_ROWS = 2, 3
SHAPES = {
    "one_tile_of_many_blocks": dict(lens=[30000], N=2, H=4),
    "several_runs_a_pair": dict(lens=[700 + 61 * b for b in range(90)], N=2, H=128),
    "rows_above_64": dict(lens=[900 + 50 * b for b in range(20)], N=5, H=16, page=32),
}


def _gives_up(call, what):
    good = call()
    _no_device_error()
    mla.mla_set_wait_timeout_ns(2_000_000)
    mla.mla_test_withhold_attention_loads(what)
    try:
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        call()
        err = mla.mla_device_status()
        took = time.perf_counter() - t0
    finally:
        mla.mla_test_withhold_attention_loads(False)
        mla.mla_set_wait_timeout_ns(0)
    assert 100 < err < 200, err
    assert took < 5.0, took  # a few limits of 2 ms in a row
    for _ in range(3):
        assert torch.equal(call(), good)
    _no_device_error()


@pytest.mark.parametrize("shape", sorted(SHAPES))
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("what", [TREE, FEW_ROWS])
def test_withheld_loads_of_tree_decode_end_in_a_status(what, fp8, shape):
    p = Problem(fp8=fp8, **SHAPES[shape])
    args = dict(cache_len=p.i32(p.lens), n_nodes=p.i32(p.nodes))
    _gives_up(lambda: p.run(**args), what)


def test_withheld_loads_of_decode_end_in_a_status():
    p = Problem([383, 383, 383], 1, 16, tree=False, spare=0)
    kv, pe = p.kv.view(3, 384, 512), p.pe.view(3, 384, 64)
    q = p.q[:, 0].contiguous()
    _gives_up(lambda: mla.mla_decode(q, kv, pe, p.w, p.o), FEW_ROWS)


def test_withheld_loads_of_one_kernel_leave_the_others_alone():
    p = Problem([500, 90], 3, 8)
    good = p.run()
    mla.mla_test_withhold_attention_loads(True)  # of the block-dense attention
    try:
        assert torch.equal(p.run(), good)
    finally:
        mla.mla_test_withhold_attention_loads(False)
    _no_device_error()
