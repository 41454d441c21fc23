"""mla_rope and mla_cache_append against 64-bit plain forms (needs a B200).

Tolerances, from the arithmetic. A result is one fp32 expression rounded once
to bf16: half a step, 2^-8 of its value, plus the fp32 part. Rotation: the
angle is off by at most 2^-24 of half a turn (2.0e-7) and the cosine and sine
by a few ulp, together under 2^-21, so each product u cos a is off by at most
2^-21 |u|, twice for the two products, with their own roundings (2^-24 each)
inside that: 2^-20 (|u| + |v|) |magnitude|. Norm: 512 squares summed in fp32
(any order: at most 512 * 2^-24 = 2^-15 of the sum, half of that after the
root), the division and two products a few 2^-24: 2^-15 of the value.
"""
import pytest
import torch

mla = pytest.importorskip("sparse_head_latent_b200")

from test_gpu_parity import _no_device_error  # noqa: E402
from test_serving_host import _frequencies  # noqa: E402

pytestmark = pytest.mark.gpu

HALF_STEP = torch.finfo(torch.bfloat16).eps / 2
SETTINGS = {
    "unscaled": dict(base=10000.0, scaling=0),
    "linear": dict(base=10000.0, scaling=1, factor=4.0),
    "yarn": dict(base=10000.0, scaling=2, factor=40.0, original_len=4096),
}


def rotated(x, positions, setting, layout, sign=1.0, magnitude=1.0):
    """fp64 rotation of [rows, heads, 64]."""
    f = torch.tensor(_frequencies(setting["base"], setting["scaling"], setting.get("factor", 1.0),
                                  setting.get("original_len", 4096)), dtype=torch.float64, device=x.device)
    a = positions.double()[:, None, None] * f
    c, s = magnitude * a.cos(), magnitude * sign * a.sin()
    x = x.double()
    out = torch.empty_like(x)
    u, v = (x[..., 0::2], x[..., 1::2]) if layout == 0 else (x[..., :32], x[..., 32:])
    p, q = u * c - v * s, u * s + v * c
    if layout == 0:
        out[..., 0::2], out[..., 1::2] = p, q
        size = (u.abs() + v.abs()).repeat_interleave(2, -1)
    else:
        out[..., :32], out[..., 32:] = p, q
        size = (u.abs() + v.abs()).repeat(1, 1, 2)
    return out, size * abs(magnitude)


def assert_rotated(got, x, positions, setting, layout, sign=1.0, magnitude=1.0):
    want, size = rotated(x, positions, setting, layout, sign, magnitude)
    err = (got.double() - want).abs()
    bound = HALF_STEP * (want.abs() + 2.0 ** -20 * size) + 2.0 ** -20 * size
    assert (err <= bound).all(), float((err - bound).max())


def _positions(rows, g, kind):
    if kind == "near":
        return torch.randint(0, 4096, (rows,), generator=g, device="cuda", dtype=torch.int32)
    p = torch.randint(-(2 ** 31), 2 ** 31 - 1, (rows,), generator=g, device="cuda", dtype=torch.int32)
    p[0] = 2 ** 31 - 1
    p[-1] = -(2 ** 31)
    return p


# the angle in fp64 is itself exact to 2^31 * 2^-53 radians: fine for both kinds
@pytest.mark.parametrize("kind", ["near", "any"])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("name", sorted(SETTINGS))
@pytest.mark.parametrize("rows,heads,width,offset", [
    (1, 1, 64, 0), (1, 64, 192, 128), (3, 5, 192, 128), (37, 1, 64, 0), (17, 3, 72, 8), (130, 128, 192, 128),
    (5, 7, 128, 0), (2, 2, 2048, 1984), (1000, 2, 192, 64)])
def test_rope_turns_its_part_and_copies_the_rest(rows, heads, width, offset, name, layout, kind):
    g = torch.Generator(device="cuda").manual_seed(rows * 1000 + heads)
    x = torch.randn(rows, heads, width, generator=g, device="cuda").to(torch.bfloat16)
    pos = _positions(rows, g, kind)
    setting = SETTINGS[name]
    rope = mla.make_rope(layout=layout, **setting)
    out = mla.mla_rope(x, pos, rope, offset=offset)
    part = slice(offset, offset + 64)
    assert_rotated(out[..., part], x[..., part], pos, setting, layout)
    rest = torch.ones(width, dtype=torch.bool, device="cuda")
    rest[part] = False
    assert torch.equal(out[..., rest], x[..., rest])
    back = mla.mla_rope(x, pos, rope, offset=offset, inverse=True)
    assert_rotated(back[..., part], x[..., part], pos, setting, layout, sign=-1.0)
    same = x.clone()
    mla.mla_rope(same, pos, rope, offset=offset, out=same)  # in place
    assert torch.equal(same, out)
    _no_device_error()


@pytest.mark.parametrize("layout", [0, 1])
def test_rope_inverse_is_the_gradient(layout):
    # <d, R x> has the gradient R^T d with respect to x: against the formula's derivative (autograd in fp64) and
    # against differences of the fp64 form, which is linear, so that one step of any size is exact.
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(9, 3, 64, generator=g, device="cuda").to(torch.bfloat16)
    d = torch.randn(9, 3, 64, generator=g, device="cuda").to(torch.bfloat16)
    pos = _positions(9, g, "near")
    setting = SETTINGS["yarn"]
    rope = mla.make_rope(layout=layout, magnitude=1.25, **setting)
    got = mla.mla_rope(d, pos, rope, inverse=True)
    assert_rotated(got, d, pos, setting, layout, sign=-1.0, magnitude=1.25)
    for i in (0, 1, 31, 32, 63):
        step = torch.zeros(9, 3, 64, dtype=torch.float64, device="cuda")
        step[..., i] = 1.0
        base = x.double()
        moved = (rotated(base + step, pos, setting, layout, magnitude=1.25)[0]
                 - rotated(base, pos, setting, layout, magnitude=1.25)[0])
        diff = (moved * d.double()).sum(-1)
        size = d.double().abs().sum(-1)
        assert ((got[..., i].double() - diff).abs() <= HALF_STEP * diff.abs() + 2.0 ** -19 * size).all()


def test_rope_takes_strides_and_leading_dimensions():
    g = torch.Generator(device="cuda").manual_seed(6)
    rope = mla.make_rope()
    kv_a = torch.randn(2, 7, 576, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.arange(14, device="cuda", dtype=torch.int32).view(2, 7)
    key = mla.mla_rope(kv_a[..., 512:], pos, rope)  # no head dimension, rows 576 apart
    assert key.shape == (2, 7, 64)
    assert torch.equal(key, mla.mla_rope(kv_a[..., 512:].contiguous(), pos, rope))
    before = kv_a.clone()
    mla.mla_rope(kv_a[..., 512:], pos, rope, out=kv_a[..., 512:])  # in place inside a wider row
    assert torch.equal(kv_a[..., 512:], key) and torch.equal(kv_a[..., :512], before[..., :512])
    q = torch.randn(2, 7, 5, 200, generator=g, device="cuda").to(torch.bfloat16)[..., :192]  # heads 200 apart
    assert torch.equal(mla.mla_rope(q, pos, rope), mla.mla_rope(q.contiguous(), pos, rope))
    one = torch.randn(1, 7, 1, 192, generator=g, device="cuda").to(torch.bfloat16).expand(1, 7, 3, 192)  # shared head
    assert torch.equal(mla.mla_rope(one, pos[:1], rope), mla.mla_rope(one.contiguous(), pos[:1], rope))
    assert mla.mla_rope(q[:0], pos[:0], rope).shape == (0, 7, 5, 192)
    x = q.contiguous()
    x[0, 0, 0, 128], x[0, 1, 0, 0] = float("inf"), float("nan")  # stay where they are
    out = mla.mla_rope(x, pos, rope)
    assert torch.isfinite(out[1]).all() and torch.isnan(out[0, 1, 0, 0]) and torch.isfinite(out[0, 2:]).all()


def normed(kv_a, weight, eps):
    x = kv_a[..., :512].double()
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("rows", [1, 3, 4, 5, 129, 1000])
def test_append_norms_rotates_and_places(rows, f32, layout):
    g = torch.Generator(device="cuda").manual_seed(rows)
    wide = torch.randn(rows, 640, generator=g, device="cuda").to(torch.bfloat16)
    kv_a = wide[:, :576]
    kv_a[:, :512] *= torch.logspace(-3, 3, rows, device="cuda")[:, None].to(torch.bfloat16)
    weight = (1 + 0.3 * torch.randn(512, generator=g, device="cuda")).to(torch.float32 if f32 else torch.bfloat16)
    pos = _positions(rows, g, "any")
    setting = SETTINGS["yarn"]
    rope = mla.make_rope(layout=layout, **setting)
    page, pages = 16, rows // 8 + 2
    kv = torch.randn(pages, page, 512, generator=g, device="cuda").to(torch.bfloat16)
    pe = torch.randn(pages, page, 64, generator=g, device="cuda").to(torch.bfloat16)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:rows].to(torch.int32)
    slots[::5] = torch.tensor([-1, -(2 ** 31), pages * page, 2 ** 31 - 1], device="cuda",
                              dtype=torch.int32).repeat(rows)[:slots[::5].numel()]
    kv0, pe0 = kv.clone(), pe.clone()
    mla.mla_cache_append(kv_a, weight, pos, rope, kv, pe, slots=slots, eps=1e-5)
    _no_device_error()
    live = (slots >= 0) & (slots < pages * page)
    at = slots[live].long()
    want = normed(kv_a, weight, 1e-5)[live]
    err = (kv.view(-1, 512)[at].double() - want).abs()
    assert (err <= (HALF_STEP + 2.0 ** -15) * want.abs() + 1e-38).all()
    assert_rotated(pe.view(-1, 64)[at][:, None], kv_a[live][:, None, 512:], pos[live], setting, layout)
    other = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    other[at] = False
    assert torch.equal(kv.view(-1, 512)[other], kv0.view(-1, 512)[other])  # rows of no token stay as they were
    assert torch.equal(pe.view(-1, 64)[other], pe0.view(-1, 64)[other])


def test_append_without_slots_makes_the_prefill_inputs():
    g = torch.Generator(device="cuda").manual_seed(8)
    kv_a = torch.randn(2, 9, 576, generator=g, device="cuda").to(torch.bfloat16)
    kv_a[0, 3] = 0  # a zero row is normalised to zero, without NaN (eps > 0)
    weight = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(9, device="cuda", dtype=torch.int32).expand(2, 9).contiguous()
    rope = mla.make_rope()
    lat = torch.empty(2, 9, 512, dtype=torch.bfloat16, device="cuda")
    pe = torch.empty(2, 9, 64, dtype=torch.bfloat16, device="cuda")
    got = mla.mla_cache_append(kv_a, weight, pos, rope, lat, pe)
    assert got[0] is lat and got[1] is pe
    want = normed(kv_a, weight, 1e-6)
    assert ((lat.double() - want).abs() <= (HALF_STEP + 2.0 ** -15) * want.abs()).all()
    assert torch.equal(pe, mla.mla_rope(kv_a[..., 512:], pos, rope))
    assert not lat[0, 3].any()


def test_append_far_into_a_large_cache():
    # byte offsets beyond 32 bits: the last row of a 4.6 GB layer
    rows = 4_500_000
    kv = torch.empty(rows, 512, dtype=torch.bfloat16, device="cuda")
    pe = torch.empty(rows, 64, dtype=torch.bfloat16, device="cuda")
    kv_a = torch.randn(2, 576, device="cuda").to(torch.bfloat16)
    weight = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor([5, 6], dtype=torch.int32, device="cuda")
    slots = torch.tensor([rows - 1, 4_194_304], dtype=torch.int32, device="cuda")
    mla.mla_cache_append(kv_a, weight, pos, mla.make_rope(), kv, pe, slots=slots)
    small = torch.empty(2, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 64, dtype=torch.bfloat16, device="cuda")
    mla.mla_cache_append(kv_a, weight, pos, mla.make_rope(), *small)
    assert torch.equal(kv[slots.long()], small[0]) and torch.equal(pe[slots.long()], small[1])


def test_rope_and_append_on_another_stream_and_in_a_graph():
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(40, 8, 192, generator=g, device="cuda").to(torch.bfloat16)
    kv_a = torch.randn(40, 576, generator=g, device="cuda").to(torch.bfloat16)
    weight = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(40, device="cuda", dtype=torch.int32)
    rope = mla.make_rope()
    kv, pe = (torch.zeros(40, n, dtype=torch.bfloat16, device="cuda") for n in (512, 64))
    want = mla.mla_rope(x, pos, rope)
    mla.mla_cache_append(kv_a, weight, pos, rope, kv, pe)
    want_kv, want_pe = kv.clone(), pe.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mla.mla_rope(x, pos, rope, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mla.mla_rope(x, pos, rope, out=out)
        mla.mla_cache_append(kv_a, weight, pos, rope, kv, pe)
    out.zero_(), kv.zero_(), pe.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(kv, want_kv) and torch.equal(pe, want_pe)
    pos.add_(3)  # a replay follows its inputs
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, mla.mla_rope(x, pos, rope))
    _no_device_error()
