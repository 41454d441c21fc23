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


def test_a_call_on_a_forked_stream_is_captured_with_the_memory_it_makes():
    p = Problem([500, 90, 3000], 3, 16)
    x = torch.randn(300, 16, 192, device="cuda").to(torch.bfloat16)
    at, rope = torch.arange(300, dtype=torch.int32, device="cuda"), mla.make_rope()
    args = dict(cache_len=p.i32(p.lens), n_nodes=p.i32(p.nodes))
    want = p.run(**args), mla.mla_rope(x, at, rope)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        first = p.run(stream=side, **args)
        turned = mla.mla_rope(x, at, rope, stream=side)
        second = p.run(stream=side, **args)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for out in (first, turned, second):
            out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, want[0]) and torch.equal(second, want[0]) and torch.equal(turned, want[1])
    _no_device_error()
    del graph


def test_results_of_a_side_stream_outlive_their_names_on_the_current_one():
    # a result dropped while the current stream still reads it is not handed to the next call on the side stream
    side, rope = torch.cuda.Stream(), mla.make_rope()
    at = torch.arange(4096, dtype=torch.int32, device="cuda")
    xs = [torch.randn(4096, 32, 192, device="cuda").to(torch.bfloat16) for _ in range(2)]
    want = [mla.mla_rope(x, at, rope) for x in xs]
    torch.cuda.synchronize()
    sums = []
    for i in range(12):
        out = mla.mla_rope(xs[i % 2], at, rope, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        big = out
        for _ in range(4):
            big = big * 1  # the current stream lags behind
        sums.append(big.clone())
        del out, big
    torch.cuda.synchronize()
    for i, s in enumerate(sums):
        assert torch.equal(s, want[i % 2])
    _no_device_error()
