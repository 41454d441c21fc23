"""mla_tree_decode against a plain form in 64 bits, and the cache upkeep calls
(needs a B200).

The oracle up-projects every key and value and knows nothing of pages or of
the absorbed form. Tolerance: between the inputs and the output stand five
roundings to bf16 (q_abs, softmax weights, latent output, head output, out),
with e4m3 weights three more (W_kvb twice, W_o). One rounding is off by at most
half a step, 2^-8 of the value, uniformly: 2^-8 / sqrt(3) rms relative to the
step's binade, 0.68 of that relative to the values (mantissas spread over the
binade), 1.54e-3. The scores have a spread of about one (that of the recipe),
so q_abs's rounding counts once. In quadrature: 3.4e-3 with five, 4.4e-3 with
eight; 5e-3 relative L2 is asserted. The largest of up to 10^6 errors of that
rms is within 8 of it: 4e-2 of the rms of their own output row, plus the last
half step. The row's, not the tensor's: every rounding above is relative to
values of the row itself, and rows differ. A node that sees n keys of unit
variance averages them to about n^-1/2, so next to rows over 500 keys (0.045)
stand rows over one (1.0) whose errors, 4.4e-3 rms, reach 5 x 4.4e-3 = 2.2e-2
among 7168 values: with 64 such sequences 0.13 of the tensor's rms of 0.17.
"""
import pytest
import torch

mla = pytest.importorskip("sparse_head_latent_b200")

from synth.inputs import SOFTMAX_SCALE, quantize_e4m3_block128  # noqa: E402
from test_gpu_parity import _no_device_error  # noqa: E402

pytestmark = pytest.mark.gpu

HALF_STEP = torch.finfo(torch.bfloat16).eps / 2


class Problem:
    def __init__(self, lens, N, H, page=64, fp8=False, tree=True, nodes=None, seed=0, spare=3):
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.B, self.N, self.H, self.page, self.fp8 = len(lens), N, H, page, fp8
        self.lens = list(lens)
        self.nodes = [N] * self.B if nodes is None else list(nodes)
        bf = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        width = max(1, max((n + k + page - 1) // page for n, k in zip(lens, self.nodes)))
        pages = self.B * width + spare
        self.q = bf(self.B, N, H, 192)
        self.kv, self.pe = bf(pages, page, 512), bf(pages, page, 64)
        self.table = torch.randperm(pages, generator=g, device="cuda")[:self.B * width].view(self.B, width).to(torch.int32)
        w = torch.randn(H * 256, 512, generator=g, device="cuda") * 512 ** -0.5
        o = torch.randn(H * 128, 7168, generator=g, device="cuda") * (H * 128) ** -0.5
        self.ws = self.os = None
        if fp8:
            cg = torch.Generator().manual_seed(seed)
            (self.w, self.ws), (self.o, self.os) = ([t.cuda() for t in quantize_e4m3_block128(x.cpu(), cg)] for x in (w, o))
        else:
            self.w, self.o = w.to(torch.bfloat16), o.to(torch.bfloat16)
        up = torch.randint(-1, 1 << 20, (self.B, N), generator=g, device="cuda")
        j = torch.arange(N, device="cuda")
        self.parents = None
        if tree:  # any earlier node, or none
            self.parents = (up % (j + 1) - 1).to(torch.int32)
        self.i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def run(self, **kw):
        a = {"parents": self.parents, "scale": SOFTMAX_SCALE, **kw}
        if "n_nodes" not in a:
            a["n_nodes"] = self.i32(self.nodes)
        q, kv, pe, table = (a.pop(k, getattr(self, k)) for k in ("q", "kv", "pe", "table"))
        n0 = a.pop("cache_len", None)
        return mla.mla_tree_decode(q, kv, pe, table, self.i32(self.lens) if n0 is None else n0, self.w, self.o,
                                   self.ws, self.os, **a)

    def weights(self):
        out = []
        for w, s in ((self.w, self.ws), (self.o, self.os)):
            if s is not None:
                w = w.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
            out.append(w.double())
        return out

    def sees(self, b):
        """bool [nodes, len + nodes]"""
        n0, n = self.lens[b], self.nodes[b]
        m = torch.zeros(n, n0 + n, dtype=torch.bool)
        m[:, :n0] = True
        for j in range(n):
            k = j
            while True:
                m[j, n0 + k] = True
                up = k - 1 if self.parents is None else int(self.parents[b, k])
                if not 0 <= up < k:
                    break
                k = up
        return m.cuda()

    def rows(self, b):
        flat = (self.table[b].long()[:, None] * self.page + torch.arange(self.page, device="cuda")).view(-1)
        flat = flat[:self.lens[b] + self.nodes[b]]
        return self.kv.view(-1, 512)[flat].double(), self.pe.view(-1, 64)[flat].double()

    def expect(self, sequences=None):
        w, o = self.weights()
        w = w.view(self.H, 256, 512)
        out = torch.zeros(self.B, self.N, 7168, dtype=torch.float64, device="cuda")
        for b in range(self.B) if sequences is None else sequences:
            n = self.nodes[b]
            if n == 0:
                continue
            c, pe = self.rows(b)
            k = torch.einsum("tl,hdl->htd", c, w)
            z = torch.einsum("nhd,htd->hnt", self.q[b, :n, :, :128].double(), k[..., :128])
            z += torch.einsum("nhd,td->hnt", self.q[b, :n, :, 128:].double(), pe)
            z = (z * SOFTMAX_SCALE).masked_fill(~self.sees(b)[None], float("-inf"))
            a = torch.einsum("hnt,htd->nhd", torch.softmax(z, -1), k[..., 128:])
            out[b, :n] = a.reshape(n, self.H * 128) @ o
        return out


def assert_near(got, want, rel=5e-3):
    got = got.double()
    assert torch.isfinite(got).all()
    err = (got - want)
    norm = want.norm()
    assert err.norm() <= rel * norm, float(err.norm() / norm)
    rms = want.square().mean(-1, keepdim=True).sqrt()
    assert (err.abs() <= 8 * rel * rms + HALF_STEP * want.abs()).all(), float((err.abs() / rms.clamp_min(1e-30)).max())


CASES = {
    "one_token_empty_cache": dict(lens=[0], N=1, H=2),
    "one_token_one_cached": dict(lens=[1], N=1, H=1, page=16),
    "around_a_key_block": dict(lens=[126, 127, 128, 129, 191, 192, 255, 256, 257], N=1, H=3, page=16),
    "nodes_across_a_key_block": dict(lens=[60, 64, 100, 120, 127, 128, 250], N=9, H=5, page=32),
    "page_128": dict(lens=[300, 127, 5], N=6, H=4, page=128),
    "page_256": dict(lens=[700, 255], N=3, H=4, page=256),
    "heads_128": dict(lens=[515, 40], N=3, H=128),
    "heads_64": dict(lens=[333, 200, 64], N=5, H=64, page=32),
    "heads_straddle_rows": dict(lens=[222, 30], N=13, H=20),
    "one_head_wide_tree": dict(lens=[400, 0, 63], N=64, H=1),
    "wide_tree": dict(lens=[190], N=64, H=8, page=16),
    "empty_and_tiny": dict(lens=[0, 0, 2, 1], N=4, H=6),
    "ragged_nodes": dict(lens=[100, 50, 700, 12, 90], N=8, H=16, nodes=[8, 0, 3, 1, 7]),
    "rows_above_64": dict(lens=[20 + b for b in range(100)], N=1, H=4, page=16),
    "rows_above_192": dict(lens=[70 + 5 * b for b in range(49)], N=4, H=3, page=32),
    "rows_above_256": dict(lens=[90 + 3 * b for b in range(70)], N=4, H=4),
    "e4m3_weights": dict(lens=[260, 33], N=4, H=4, fp8=True),
    "e4m3_rows_above_256": dict(lens=[50] * 70, N=4, H=2, fp8=True),
    "e4m3_rows_512": dict(lens=[9 * b for b in range(64)], N=8, H=3, page=16, fp8=True),
    "e4m3_rows_above_512": dict(lens=[40 + b for b in range(103)], N=5, H=2, fp8=True),
    "e4m3_rows_above_768": dict(lens=[b % 40 for b in range(130)], N=6, H=2, page=32, fp8=True),
    "long": dict(lens=[9000, 20000, 33], N=2, H=8),
    "one_long": dict(lens=[20000], N=1, H=128, tree=False),
    "one_long_few_rows": dict(lens=[9890], N=5, H=8, page=16),
    "two_long": dict(lens=[9000, 7000], N=3, H=16, page=32, nodes=[3, 1]),
    "two_long_e4m3": dict(lens=[3000, 7000], N=3, H=16, page=32, fp8=True),
    "eight_long": dict(lens=[2000 + 700 * b for b in range(8)], N=2, H=40),
    "long_many_rows": dict(lens=[5000], N=40, H=64),
    "chain": dict(lens=[130, 61], N=7, H=4, tree=False),
}


@pytest.mark.parametrize("case", sorted(CASES))
def test_tree_decode_matches_the_plain_form(case):
    p = Problem(seed=len(case), **CASES[case])
    out = p.run()
    _no_device_error()
    assert_near(out, p.expect())
    for b, n in enumerate(p.nodes):
        assert not out[b, n:].any()


def test_a_chain_is_the_tree_in_which_each_node_follows_the_last():
    p = Problem([75, 140, 3], 11, 6)
    chain = (torch.arange(11, device="cuda") - 1).to(torch.int32).expand(3, 11).contiguous()
    assert torch.equal(p.run(parents=None), p.run(parents=chain))
    _no_device_error()


def test_one_token_per_sequence_is_plain_decode():
    # a contiguous cache is a paged one with its pages in order
    p = Problem([191, 191], 1, 4, page=64, tree=False, spare=0)
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    got = p.run(table=table, n_nodes=None)
    want = mla.mla_decode(p.q[:, 0].contiguous(), p.kv.view(2, 192, 512), p.pe.view(2, 192, 64), p.w, p.o,
                          scale=SOFTMAX_SCALE)
    _no_device_error()
    # both are within the tolerance of the same exact value
    assert (got[:, 0].double() - want.double()).norm() <= 1e-2 * want.double().norm()


def test_parents_outside_the_earlier_nodes_mean_the_last_committed_position():
    p = Problem([70, 20], 6, 4)
    wild = p.parents.clone()
    wild[wild < 0] = torch.tensor([-7, -(2 ** 31), 2 ** 31 - 1, 6, 64, 99], dtype=torch.int32,
                                  device="cuda").repeat(4)[:int((wild < 0).sum())]
    wild[0, 3] = 3  # itself
    plain = p.parents.clone()
    plain[0, 3] = -1
    assert torch.equal(p.run(parents=wild), p.run(parents=plain))
    _no_device_error()


@pytest.mark.parametrize("stale", [float("nan"), float("inf"), -float("inf")])
def test_rows_behind_the_last_position_may_hold_anything(stale):
    p = Problem([100, 127, 5, 190], 3, 5, page=64, nodes=[3, 1, 2, 0])
    clean = p.run()
    live = torch.zeros(p.kv.shape[0] * p.page, dtype=torch.bool, device="cuda")
    for b in range(p.B):
        flat = (p.table[b].long()[:, None] * p.page + torch.arange(p.page, device="cuda")).view(-1)
        live[flat[:p.lens[b] + p.nodes[b]]] = True
    for c in (p.kv, p.pe):
        c.view(-1, c.shape[-1])[~live] = stale
    p.q[1, 1:] = stale  # queries of nodes that are not there
    assert torch.equal(p.run(), clean)
    _no_device_error()


def test_a_node_that_another_does_not_see_cannot_reach_it():
    # sibling branches: NaN in the rows of one leave the other as it was
    p = Problem([100, 126], 5, 4)
    p.parents[:] = torch.tensor([-1, 0, 0, 1, 2], dtype=torch.int32)
    clean = p.run()
    for b in range(2):
        t = p.lens[b] + 1
        page, r = int(p.table[b, t // p.page]), t % p.page
        p.kv[page, r], p.pe[page, r] = float("nan"), float("inf")
    got = p.run()
    for j in (0, 2, 4):
        assert torch.equal(got[:, j], clean[:, j]), j
    assert torch.isnan(got[:, 1]).all() and torch.isnan(got[:, 3]).all()
    _no_device_error()


def test_scores_that_keep_growing_are_rescaled():
    # keys ordered so that every block raises the running maximum by far more than the rescaling threshold
    p = Problem([1500], 2, 3, tree=False)
    ramp = torch.linspace(-12, 12, 1502, device="cuda")
    flat = (p.table[0].long()[:, None] * p.page + torch.arange(p.page, device="cuda")).view(-1)[:1502]
    p.q[..., :128] *= 0.1
    p.q[..., 128:] = 4.0
    p.pe.view(-1, 64)[flat] = (ramp[:, None] + 0.1 * torch.randn(1502, 64, device="cuda")).to(torch.bfloat16)
    out = p.run()
    _no_device_error()
    # the weight sits on few keys with scores of some hundreds: exact in q_pe . k_pe (no q_abs part to speak of)
    assert_near(out, p.expect())


def test_bad_pages_and_lengths_are_reported_and_stay_with_their_sequence():
    p = Problem([200, 90, 150, 40], 2, 4, page=16)
    clean = p.run()
    table = p.table.clone()
    table[1, 8:] = torch.tensor(-5, dtype=torch.int32)       # not needed: 92 positions are six pages
    table[3, 5:] = torch.tensor(2 ** 31 - 1, dtype=torch.int32)
    assert torch.equal(p.run(table=table), clean)
    _no_device_error()
    for bad in (-1, -(2 ** 31), p.kv.shape[0], 2 ** 31 - 1):
        table = p.table.clone()
        table[2, 3] = bad
        out = p.run(table=table)
        assert mla.mla_device_status() == 401
        assert mla.mla_device_status() == 0
        for b in (0, 1, 3):
            assert torch.equal(out[b], clean[b])
    for length in (-1, 2 ** 31 - 1, p.table.shape[1] * 16 - 1):
        n0 = p.i32(p.lens)
        n0[0] = length
        out = p.run(cache_len=n0)
        assert mla.mla_device_status() == 402
        assert not out[0].any() and torch.equal(out[1:], clean[1:])


def test_more_nodes_than_there_are_and_fewer_than_none_are_clamped():
    p = Problem([70, 20, 33], 4, 4, nodes=[4, 0, 4])
    assert torch.equal(p.run(n_nodes=p.i32([9, -3, 2 ** 31 - 1])), p.run())
    _no_device_error()


def test_sequences_may_share_pages():
    p = Problem([256, 256, 256], 3, 8)
    p.table[1, :3], p.table[2, :4] = p.table[0, :3], p.table[0, :4]
    p.nodes[2] = 2
    assert_near(p.run(), p.expect())
    _no_device_error()


def test_cache_larger_than_32_bit_offsets():
    p = Problem([130, 64], 2, 4)
    pages = 75_000  # 4.9 GB of latent rows
    kv = torch.empty(pages, 64, 512, dtype=torch.bfloat16, device="cuda")
    pe = torch.empty(pages, 64, 64, dtype=torch.bfloat16, device="cuda")
    far = p.table + (pages - p.kv.shape[0])
    kv[pages - p.kv.shape[0]:], pe[pages - p.kv.shape[0]:] = p.kv, p.pe
    assert torch.equal(p.run(kv=kv, pe=pe, table=far), p.run())
    _no_device_error()


def test_same_result_every_time_and_on_every_stream():
    p = Problem([3000, 10, 700], 5, 16)
    ws = torch.empty(mla.mla_workspace_bytes(mla.make_dims(3, 5, 16), mla.MLA_ENTRY_TREE_DECODE, False),
                     dtype=torch.uint8, device="cuda")
    ws.fill_(0xff)  # the workspace's contents do not matter
    first = p.run(workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [p.run(stream=side), p.run(), p.run(stream=side)]  # two streams at once, each call its own workspace
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, first)
    for _ in range(20):
        assert torch.equal(p.run(workspace=ws), first)
    _no_device_error()


@pytest.mark.parametrize("N,H,page", [(1, 128, 64), (5, 64, 16), (64, 8, 128)])
def test_many_runs_of_blocks_per_pair(N, H, page):
    # every pair works through several sequences and tiles, with one and two blocks of drafted keys at their ends,
    # many times over; tables too large to stay in the first-level cache
    lens = [37 * (b % 50) + 1000 * (b % 7) + 64 * (b % 3) for b in range(150)]
    p = Problem(lens, N, H, page=page)
    first = p.run()
    for _ in range(30):
        again = p.run()
    _no_device_error()
    assert torch.equal(again, first)
    some = [0, 1, 6, 49, 77, 149]
    assert_near(first[some], p.expect(some)[some])


@pytest.mark.parametrize("B,N,H", [(5, 1, 128), (8, 8, 64), (16, 8, 128), (50, 5, 128), (13, 5, 3)])
def test_e4m3_codes_read_as_stored_give_the_same_result_every_time(B, N, H):
    # rows of one, of 64 or fewer, of two tiles of 128: codes in flight for every head and all of W_o
    p = Problem([40 + 7 * b for b in range(B)], N, H, page=32, fp8=True)
    first = p.run()
    for _ in range(10):
        assert torch.equal(p.run(), first)
    _no_device_error()
    some = sorted({0, B // 2, B - 1})
    assert_near(first[some], p.expect(some)[some])


def test_captured_graph_follows_its_inputs():
    p = Problem([500, 900], 4, 8)
    n0, nodes, table = p.i32(p.lens), p.i32(p.nodes), p.table.clone()
    ws = torch.empty(mla.mla_workspace_bytes(mla.make_dims(2, 4, 8), mla.MLA_ENTRY_TREE_DECODE, False),
                     dtype=torch.uint8, device="cuda")
    out = torch.empty(2, 4, 7168, dtype=torch.bfloat16, device="cuda")
    call = lambda: p.run(cache_len=n0, n_nodes=nodes, table=table, out=out, workspace=ws)  # noqa: E731
    eager = call().clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    # the next step: other lengths, fewer nodes
    n0.copy_(torch.tensor([123, 877]))
    nodes.copy_(torch.tensor([2, 4]))
    graph.replay()
    torch.cuda.synchronize()
    p.lens, p.nodes = [123, 877], [2, 4]
    assert_near(out, p.expect())
    assert torch.equal(out, p.run())
    _no_device_error()
    del graph


# ------------------------------------------------------------------ upkeep


def test_more_sequences_than_a_block_has_threads():
    # several sequences per thread of the scan; some without nodes, some without a cache
    B = 1111
    p = Problem([(37 * b) % 150 if b % 9 else 0 for b in range(B)], 2, 2, page=16, nodes=[(b * 7) % 3 for b in range(B)])
    out = p.run()
    _no_device_error()
    for b, n in enumerate(p.nodes):
        assert not out[b, n:].any()
    some = list(range(0, 30)) + list(range(340, 372)) + list(range(700, 712)) + [1109, 1110]
    assert_near(out[some], p.expect(some)[some])


@pytest.mark.parametrize("fp8", [False, True])
def test_no_sequence_has_a_node(fp8):
    p = Problem([200, 0, 31], 3, 4, nodes=[0, 0, 0], fp8=fp8)
    out = torch.full((3, 3, 7168), 7.0, dtype=torch.bfloat16, device="cuda")
    p.run(out=out)
    assert not out.any()
    _no_device_error()


def test_a_table_filled_to_its_last_position():
    p = Problem([61, 30], 3, 4, page=64, spare=0)
    assert p.table.shape[1] == 1
    assert_near(p.run(), p.expect())
    _no_device_error()


@pytest.mark.parametrize("fp8", [False, True])
def test_two_graphs_share_a_workspace(fp8):
    # one step each of two models' batches, replayed in turn on one stream
    a, b = Problem([700, 90, 3000], 3, 16, fp8=fp8), Problem([64, 2000, 5], 3, 16, fp8=fp8, seed=9)
    ws = torch.empty(mla.mla_workspace_bytes(mla.make_dims(3, 3, 16, fp8=fp8), mla.MLA_ENTRY_TREE_DECODE, False),
                     dtype=torch.uint8, device="cuda")
    want = [p.run() for p in (a, b)]
    graphs, outs = [], []
    for p in (a, b):
        n0, nodes = p.i32(p.lens), p.i32(p.nodes)
        out = torch.empty(3, 3, 7168, dtype=torch.bfloat16, device="cuda")
        call = lambda: p.run(cache_len=n0, n_nodes=nodes, out=out, workspace=ws)  # noqa: B023, E731
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append((graph, n0, nodes))
        outs.append(out)
    for _ in range(3):
        for out in outs:
            out.zero_()
        for graph, _, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    _no_device_error()


def test_e4m3_calls_on_two_streams_at_once():
    problems = [Problem([300 + 50 * b for b in range(12)], 7, 128, fp8=True, seed=s) for s in (1, 2)]
    want = [p.run() for p in problems]
    streams = [torch.cuda.Stream() for _ in problems]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    args = [dict(cache_len=p.i32(p.lens), n_nodes=p.i32(p.nodes)) for p in problems]
    torch.cuda.synchronize()
    got = [[p.run(stream=st, **a) for _ in range(6)] for p, st, a in zip(problems, streams, args)]
    torch.cuda.synchronize()
    _no_device_error()
    for outs, w in zip(got, want):
        assert all(torch.equal(o, w) for o in outs)


def _caches(layers, pages, page, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (pages, page) if layers is None else (layers, pages, page)
    return [torch.randn(*shape, n, generator=g, device="cuda").to(torch.bfloat16) for n in (512, 64)]


@pytest.mark.parametrize("layers,page,width", [(None, 16, 3), (1, 16, 8), (3, 64, 9), (2, 32, 16), (2, 16, 64),
                                               (5, 16, 1), (4, 32, 17), (3, 16, 32), (2, 64, 33)])
def test_compact_moves_the_accepted_rows(layers, page, width):
    B, cols = 5, 12
    kv, pe = _caches(layers, B * cols + 2, page)
    g = torch.Generator().manual_seed(width)
    table = torch.randperm(B * cols + 2, generator=g)[:B * cols].view(B, cols).to(torch.int32)
    n0 = torch.randint(0, cols * page - 64, (B,), generator=g).to(torch.int32)
    acc = torch.stack([torch.randperm(64, generator=g)[:width] for _ in range(B)]).to(torch.int32)
    acc[0] = acc[0].sort().values
    if width > 4:
        acc[1, 2] = acc[1, 1]  # the same node twice
        acc[2] = torch.arange(width)  # nothing to move
    counts = torch.tensor([width, width, width, width // 2, 0], dtype=torch.int32)
    want = [c.clone() for c in (kv, pe)]
    for w, c in zip(want, (kv, pe)):
        w, c = (t if layers is not None else t[None] for t in (w, c))
        for b in range(B):
            for i in range(int(counts[b])):
                s, d = int(n0[b]) + int(acc[b, i]), int(n0[b]) + i
                w[:, int(table[b, d // page]), d % page] = c[:, int(table[b, s // page]), s % page]
    mla.mla_cache_compact(kv, pe, table.cuda(), n0.cuda(), acc.cuda(), counts.cuda())
    _no_device_error()
    assert torch.equal(kv, want[0]) and torch.equal(pe, want[1])


def test_compact_leaves_what_it_cannot_place():
    kv, pe = _caches(2, 8, 16)
    before = kv.clone(), pe.clone()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = i32([[0, 1, 2], [3, -1, 8], [4, 5, 6]])
    # beyond the table; on pages that are none; a negative node; a negative length
    for n0, acc in (([47, 0, 0], [[1, 2], [16, 33], [-1, -5]]), ([-1, 14, 2 ** 31 - 1], [[0, 1], [3, 18], [0, 1]])):
        mla.mla_cache_compact(kv, pe, table, i32(n0), i32(acc), i32([1, 2, 2]))
        assert mla.mla_device_status() == 401
        assert torch.equal(kv, before[0]) and torch.equal(pe, before[1])
    mla.mla_cache_compact(kv, pe, table, i32([0, 0, 0]), i32([[1], [1], [1]]), i32([-4, 0, 99]))  # counts are clamped
    assert mla.mla_device_status() == 0
    want = before[0].clone()
    want[:, 4, 0] = before[0][:, 4, 1]
    assert torch.equal(kv, want)


@pytest.mark.parametrize("layers,page,n", [(None, 16, 1), (3, 64, 5), (2, 16, 70), (1, 16, 600)])
def test_copy_pages(layers, page, n):
    pages = 2 * n + 10
    kv, pe = _caches(layers, pages, page)
    g = torch.Generator().manual_seed(n)
    order = torch.randperm(pages, generator=g).tolist()
    dst, free = order[:n], order[n:]
    src = [free[(3 * i) % 7 if i % 2 else i % len(free)] for i in range(n)]  # some pages several times
    src[0] = dst[0]  # onto itself: nothing
    want = [c.clone() for c in (kv, pe)]
    for w, c in zip(want, (kv, pe)):
        w, c = (t if layers is not None else t[None] for t in (w, c))
        w[:, dst] = c[:, src]
    mla.mla_cache_copy_pages(kv, pe, src, torch.tensor(dst, dtype=torch.int32))
    _no_device_error()
    assert torch.equal(kv, want[0]) and torch.equal(pe, want[1])
    with pytest.raises(mla.MlaError):
        mla.mla_cache_copy_pages(kv, pe, [free[0], free[1]], [dst[0], dst[0]])
    assert torch.equal(kv, want[0])


def test_upkeep_in_a_layer_beyond_32_bit_offsets():
    kv = torch.zeros(3, 27_000, 64, 512, dtype=torch.bfloat16, device="cuda")  # 5.3 GB
    pe = torch.zeros(3, 27_000, 64, 64, dtype=torch.bfloat16, device="cuda")
    kv[2, 26_998], pe[2, 26_998] = 3.0, 5.0
    mla.mla_cache_copy_pages(kv, pe, [26_998], [26_999])
    assert (kv[2, 26_999] == 3).all() and (pe[2, 26_999] == 5).all() and not kv[1, 26_999].any()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    kv[2, 26_999, 9], pe[2, 26_999, 9] = 7.0, 8.0
    mla.mla_cache_compact(kv, pe, i32([[26_999]]), i32([2]), i32([[7]]), i32([1]))
    assert (kv[2, 26_999, 2] == 7).all() and (pe[2, 26_999, 2] == 8).all() and (kv[2, 26_999, 3] == 3).all()
    _no_device_error()


# ------------------------------------------------------------------ a run of them together


@pytest.mark.parametrize("captured", [False, True])
def test_speculative_steps_equal_decoding_one_token_at_a_time(captured):
    """Three tokens decoded one by one, and the same three as the accepted path of one drafted tree, moved together
    afterwards and read by a forked sequence's next token: the same hidden states and the same cache."""
    B, H, page, width = 2, 8, 16, 6
    g = torch.Generator(device="cuda").manual_seed(3)
    bf = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    w = (torch.randn(H * 256, 512, generator=g, device="cuda") * 512 ** -0.5).to(torch.bfloat16)
    o = (torch.randn(H * 128, 7168, generator=g, device="cuda") * (H * 128) ** -0.5).to(torch.bfloat16)
    norm = (1 + 0.1 * torch.randn(512, generator=g, device="cuda")).to(torch.bfloat16)
    rope = mla.make_rope(scaling=mla.MLA_ROPE_YARN, factor=40.0)
    n0 = [45, 30]
    table = i32([[3, 7, 1, 12, 5, 9], [2, 4, 11, 0, 10, 8]])
    prompt = bf(B, 45, 576)
    # drafts: nodes 0..6, the accepted path is 1 -> 3 -> 6 in both sequences
    parents = [-1, -1, 0, 1, 1, 2, 3]
    depth = [0, 0, 1, 1, 1, 2, 2]
    path = [1, 3, 6]
    draft_kv, draft_q = bf(B, 7, 576), bf(B, 7, H, 192)
    next_kv, next_q = bf(B, 1, 576), bf(B, 1, H, 192)

    def fresh():
        kv = torch.full((14, page, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
        pe = torch.full((14, page, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
        for b in range(B):
            pos = torch.arange(n0[b], dtype=torch.int32, device="cuda")
            mla.mla_cache_append(prompt[b, :n0[b]], norm, pos, rope, kv, pe, slots=slots(b, pos))
        return kv, pe

    def slots(b, at):
        return (table[b].long()[(at // page).long()] * page + at % page).to(torch.int32)

    def step(kv, pe, q, new, at, positions, lens, up, tables):
        where = torch.stack([slots(b, at[b]) for b in range(B)])
        mla.mla_cache_append(new, norm, positions, rope, kv, pe, slots=where)
        return mla.mla_tree_decode(mla.mla_rope(q, positions, rope), kv, pe, tables, lens, w, o, parents=up)

    # one token at a time
    kv1, pe1 = fresh()
    one = []
    for i, node in enumerate(path):
        at = i32([[n0[0] + i], [n0[1] + i]])
        one.append(step(kv1, pe1, draft_q[:, node:node + 1].contiguous(), draft_kv[:, node:node + 1].contiguous(),
                        at, at, at[:, 0].contiguous(), None, table))
    at = i32([[n0[0] + 3], [n0[1] + 3]])
    one.append(step(kv1, pe1, next_q, next_kv, at, at, at[:, 0].contiguous(), None, table))

    # as a tree
    kv2, pe2 = fresh()
    lens = i32(n0)
    rank = i32([[n0[b] + j for j in range(7)] for b in range(B)])
    positions = i32([[n0[b] + depth[j] for j in range(7)] for b in range(B)])
    up = i32([parents] * B)
    accepted, counts = i32([path] * B), i32([3, 3])
    if captured:
        start = kv2.clone(), pe2.clone()
        where = torch.stack([slots(b, rank[b]) for b in range(B)])
        q = torch.empty_like(draft_q)
        tree = torch.empty(B, 7, 7168, dtype=torch.bfloat16, device="cuda")

        def whole():
            mla.mla_cache_append(draft_kv, norm, positions, rope, kv2, pe2, slots=where)
            mla.mla_rope(draft_q, positions, rope, out=q)
            mla.mla_tree_decode(q, kv2, pe2, table, lens, w, o, parents=up, out=tree)
            mla.mla_cache_compact(kv2, pe2, table, lens, accepted, counts)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            whole()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            whole()
        kv2.copy_(start[0]), pe2.copy_(start[1]), tree.zero_()
        graph.replay()
    else:
        tree = step(kv2, pe2, draft_q, draft_kv, rank, positions, lens, up, table)
        mla.mla_cache_compact(kv2, pe2, table, lens, accepted, counts)
    for i, node in enumerate(path):
        assert (tree[:, node].double() - one[i][:, 0].double()).norm() <= 1e-2 * one[i].double().norm()
    for b in range(B):
        rows = slots(b, torch.arange(n0[b] + 3, device="cuda")).long()
        assert torch.equal(kv2.view(-1, 512)[rows], kv1.view(-1, 512)[rows])
        assert torch.equal(pe2.view(-1, 64)[rows], pe1.view(-1, 64)[rows])

    # fork sequence 0: its full pages are shared, the last one copied; the fork decodes the next token
    last = (n0[0] + 3) // page
    mla.mla_cache_copy_pages(kv2, pe2, [int(table[0, last])], [13])
    fork = table.clone()
    fork[0, last] = 13
    kept = table
    table = fork
    at = i32([[n0[0] + 3], [n0[1] + 3]])
    got = step(kv2, pe2, next_q, next_kv, at, at, at[:, 0].contiguous(), None, fork)
    table = kept
    _no_device_error()
    # the same keys and the same kernel: bit for bit
    assert torch.equal(got, one[3])
