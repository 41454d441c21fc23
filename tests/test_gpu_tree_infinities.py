"""Infinities in a paged cache: mla_tree_decode against the plain form in 64 bits (needs a B200).

A key whose score is -inf has weight 0. With finite values it is then absent; 0 times a value that is not finite is NaN,
and a row that sees no key with a finite score is 0 / 0. A node that does not see the key is not touched by it."""
import pytest
import torch

mla = pytest.importorskip("sparse_head_latent_b200")

from synth.inputs import SOFTMAX_SCALE  # noqa: E402
from test_gpu_parity import _no_device_error  # noqa: E402
from test_gpu_tree import Problem, assert_near  # noqa: E402

pytestmark = pytest.mark.gpu
INF = float("inf")


def _at(p, b, t):
    return int(p.table[b, t // p.page]), t % p.page


def _q_abs(p, b, j):
    """q_nope W_UK in 64 bits: [H, 512]"""
    return torch.einsum("hd,hdl->hl", p.q[b, j, :, :128].double(), p.weights()[0].view(p.H, 256, 512)[:, :128])


def _expect(p):
    """The plain form with each node's own keys only, so that no other key's values are multiplied by 0."""
    w, o = p.weights()
    w = w.view(p.H, 256, 512)
    out = torch.zeros(p.B, p.N, 7168, dtype=torch.float64, device="cuda")
    for b in range(p.B):
        c, pe = p.rows(b)
        k = torch.einsum("tl,hdl->htd", c, w)
        for j, seen in enumerate(p.sees(b)):
            q = p.q[b, j].double()
            z = torch.einsum("hd,htd->ht", q[:, :128], k[:, seen, :128]) + q[:, 128:] @ pe[seen].T
            a = torch.einsum("ht,htd->hd", torch.softmax(z * SOFTMAX_SCALE, -1), k[:, seen, 128:])
            out[b, j] = a.reshape(-1) @ o
    return out


def _compare(p):
    got, want = p.run(), _expect(p)
    _no_device_error()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    good = ~torch.isnan(want).any(-1)
    if good.any():
        assert_near(got[good], want[good])
    return got


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("lens,H", [([100, 126], 1), ([640, 30], 3), ([9000], 1)])
def test_infinite_latent_of_a_drafted_key_reaches_every_node_that_sees_it(lens, H, sign, page):
    # sign: of the key's score in head 0. -inf and +inf both have to end as NaN, in the nodes below it only.
    p = Problem(lens, 5, H, page=page)
    p.parents[:] = torch.tensor([-1, 0, 0, 1, 2], dtype=torch.int32)
    clean = p.run()
    for b in range(p.B):
        # the largest product of both nodes that see the key, so that rounding leaves their signs; one sign for both
        a1, a3 = _q_abs(p, b, 1)[0], _q_abs(p, b, 3)[0]
        both = torch.where(a1 * a3 > 0, torch.minimum(a1.abs(), a3.abs()), torch.zeros_like(a1))
        l = int(both.argmax())
        page_, r = _at(p, b, p.lens[b] + 1)
        p.kv[page_, r, l] = INF * sign * float(a1[l].sign())
    got = _compare(p)
    for j in (0, 2, 4):
        assert torch.equal(got[:, j], clean[:, j]), j
    assert torch.isnan(got[:, 1]).all() and torch.isnan(got[:, 3]).all()


@pytest.mark.parametrize("lens", [[100, 126], [640, 30], [9000]])
def test_infinite_key_with_finite_values_is_absent_where_its_score_is_lowest(lens):
    p = Problem(lens, 5, 2)
    p.parents[:] = torch.tensor([-1, 0, 0, 1, 2], dtype=torch.int32)
    p.q[..., 128] = -p.q[..., 128].abs() - 0.1  # every score of the key is -inf
    for b in range(p.B):
        page, r = _at(p, b, p.lens[b] + 1)
        p.pe[page, r, 0] = INF
        page, r = _at(p, b, 3)  # and a committed one's
        p.pe[page, r, 0] = INF
    assert not torch.isnan(_compare(p)).any()


@pytest.mark.parametrize("lens,N", [([0], 1), ([0, 5], 3), ([130, 127], 1), ([9000], 2)])
def test_no_key_with_a_finite_score_is_not_a_number(lens, N):
    p = Problem(lens, N, 3, tree=False)
    p.q[..., 128] = -p.q[..., 128].abs() - 0.1
    p.pe[..., 0] = INF
    assert torch.isnan(_compare(p)).all()


def test_infinite_latent_of_a_committed_key_in_a_share_without_finite_scores():
    # one sequence over all pairs: the first blocks' scores are all -inf, and one of their values is not finite
    p = Problem([20000], 1, 1, tree=False)
    p.q[..., 128] = -p.q[..., 128].abs() - 0.1
    flat = (p.table[0].long()[:, None] * p.page + torch.arange(p.page, device="cuda")).view(-1)
    p.pe.view(-1, 64)[flat[:1280], 0] = INF
    assert not torch.isnan(_compare(p)).any()
    a = _q_abs(p, 0, 0)[0]
    l = int(a.abs().argmax())
    p.kv.view(-1, 512)[flat[700], l] = -INF * float(a[l].sign())
    assert torch.isnan(_compare(p)).all()


def test_stale_infinities_behind_the_last_node():
    # the table ends with the last node; rows of nodes that are not there would see positions behind it
    p = Problem([60, 61, 10], 8, 3, page=64, nodes=[4, 3, 2], spare=0)
    assert p.table.shape[1] == 1
    for b in range(p.B):
        page, r = _at(p, b, p.lens[b] + p.nodes[b] - 1)
        p.kv[page, r + 1:], p.pe[page, r + 1:] = -INF, INF
    p.q[..., 128] = -p.q[..., 128].abs()
    assert not torch.isnan(_compare(p)).any()
