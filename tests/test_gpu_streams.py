"""Calls on two streams at once whose workspaces and results the binding makes itself (needs a B200).

Different problems in turn on the current and on a side stream: each has to give what it gives alone, bit for bit.
One call's blocks are free for the next as soon as it returns, while its kernels still run."""
import pytest
import torch

mla = pytest.importorskip("sparse_head_latent_b200")

from test_gpu_parity import _no_device_error  # noqa: E402
from test_gpu_tree import Problem  # noqa: E402

pytestmark = pytest.mark.gpu


def _in_turn(calls, times=8):
    """calls: four f(stream=None) of one workspace size; each alone, then in turn on two streams."""
    want = [f() for f in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for i in range(times):
        got += [(0, calls[0]()), (1, calls[1](stream=side)), (2, calls[2]()), (3, calls[3](stream=side))]
    torch.cuda.synchronize()
    _no_device_error()
    for i, out in got:
        assert torch.equal(out, want[i]), i


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_decode_of_different_problems_on_two_streams(fp8):
    problems = [Problem([3000 + 17 * s, 10 + s, 700], 5, 16, fp8=fp8, seed=s) for s in range(4)]
    args = [dict(cache_len=p.i32(p.lens), n_nodes=p.i32(p.nodes)) for p in problems]
    _in_turn([lambda p=p, a=a, **k: p.run(**a, **k) for p, a in zip(problems, args)])


def test_rope_of_different_rows_on_two_streams():
    rope = mla.make_rope()
    xs = [torch.randn(2048, 64, 192, device="cuda").to(torch.bfloat16) for _ in range(4)]
    at = torch.arange(2048, dtype=torch.int32, device="cuda")
    _in_turn([lambda x=x, **k: mla.mla_rope(x, at, rope, **k) for x in xs])


def test_prefill_and_decode_of_different_problems_on_two_streams():
    g = torch.Generator(device="cuda").manual_seed(5)
    bf = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    w, o = bf(8 * 256, 512) * 0.04, bf(8 * 128, 7168) * 0.03
    data = [(bf(2, 700, 8, 192), bf(2, 700, 512), bf(2, 700, 64)) for _ in range(4)]
    last = [d[0][:, 0].contiguous() for d in data]
    _in_turn([lambda d=d, **k: mla.mla_prefill(*d, w, o, **k) for d in data])
    _in_turn([lambda d=d, q=q, **k: mla.mla_decode(q, d[1], d[2], w, o, **k) for d, q in zip(data, last)])
    _in_turn([lambda d=d, **k: mla.mla_kv_upproject(d[1], w, **k) for d in data])
