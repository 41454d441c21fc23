"""Which stream's memory a call's own tensors come from, and a pipeline's (CPU only).

A call on `stream` writes its workspace, and a result it makes, on that stream.
The caching allocator hands a freed block out again at once, in the order of the
block's own stream, so a block of the current stream's pool can still be in use
there when `stream` writes it. Streams, tensors' devices and the library are
stand-ins here: what is checked is where each allocation is made."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

import sparse_head_latent_b200 as mla
from sparse_head_latent_b200 import mla as binding


class Tensor:
    """A CPU tensor that remembers the stream it was allocated on and its other users."""

    def __init__(self, t, stream):
        self.t, self.stream, self.users = t, stream, []

    def record_stream(self, s):
        self.users.append(s)

    def __getattr__(self, name):
        return getattr(self.t, name)


def _stream(name):
    return SimpleNamespace(name=name, device=SimpleNamespace(index=0), cuda_stream=hash(name) & 0xffff)


@pytest.fixture
def world(monkeypatch):
    w = SimpleNamespace(current=_stream("main"), made=[])
    empty = torch.empty

    def fake_empty(*shape, **kw):
        kw.pop("device", None)
        t = Tensor(empty(*shape, **kw), w.current)
        w.made.append(t)
        return t

    @contextlib.contextmanager
    def on(stream):
        before, w.current = w.current, stream
        yield
        w.current = before

    class Lib:
        mla_workspace_bytes = staticmethod(lambda *a: 4096)

        def __getattr__(self, name):
            return lambda *a: 0

    monkeypatch.setattr(torch, "empty", fake_empty)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: w.current)
    monkeypatch.setattr(binding, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    monkeypatch.setattr(binding, "_lib", Lib())
    monkeypatch.setattr(binding, "load_library", Lib)
    monkeypatch.setattr(binding, "_cuda", lambda t: 0)
    monkeypatch.setattr(binding, "_data", lambda t, index, strided=False: None if t is None else t.data_ptr())
    monkeypatch.setattr(binding, "_ptr", lambda t: None if t is None else t.data_ptr())
    return w


bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
W, O = (2 * 256, 512), (2 * 128, 7168)
CALLS = {
    # name: (call, tensors it makes, of which the caller gets)
    "kv_upproject": (lambda **k: mla.mla_kv_upproject(bf(3, 512), bf(*W), **k), 2, 1),
    "attend": (lambda **k: mla.mla_attend(bf(1, 3, 2, 192), bf(1, 3, 512), bf(1, 3, 64), bf(*W), **k), 2, 1),
    "attend_static": (lambda **k: mla.mla_attend_static(bf(1, 3, 2, 192), bf(1, 3, 512), bf(1, 3, 64), bf(*W), **k), 1, 1),
    "out_project": (lambda **k: mla.mla_out_project(bf(3, 256), bf(*O), **k), 2, 1),
    "prefill": (lambda **k: mla.mla_prefill(bf(1, 3, 2, 192), bf(1, 3, 512), bf(1, 3, 64), bf(*W), bf(*O), **k), 2, 1),
    "decode": (lambda **k: mla.mla_decode(bf(1, 2, 192), bf(1, 3, 512), bf(1, 3, 64), bf(*W), bf(*O), **k), 2, 1),
    "quantize_act": (lambda **k: mla.mla_quantize_act(bf(3, 256), **k), 2, 2),
    "rope": (lambda **k: mla.mla_rope(bf(3, 2, 192), i32(3), binding.MlaRopeTable(), **k), 1, 1),
    "tree_decode": (lambda **k: mla.mla_tree_decode(bf(1, 3, 2, 192), bf(4, 16, 512), bf(4, 16, 64), i32(1, 4), i32(1),
                                                    bf(*W), bf(*O), **k), 2, 1),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_call_on_a_stream_allocates_on_it(world, name):
    call, makes, gives = CALLS[name]
    main, side = world.current, _stream("side")
    got = call(stream=side)
    assert len(world.made) == makes and world.current is main
    assert all(t.stream is side for t in world.made), [t.stream.name for t in world.made]
    given = got if isinstance(got, tuple) else (got,)
    assert len(given) == gives
    # what the caller gets is used on the current stream, too, and not handed out again before that is done
    assert all(t.users == [main] for t in given)
    assert all(not t.users for t in world.made if not any(t is g for g in given))


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("named", [False, True])
def test_a_call_on_the_current_stream_needs_no_record(world, name, named):
    call, makes, _ = CALLS[name]
    call(**({"stream": world.current} if named else {}))
    assert len(world.made) == makes
    assert all(t.stream is world.current and not t.users for t in world.made)


def test_the_pipeline_orders_its_streams_with_the_memory_it_is_given(world, monkeypatch):
    class Side(SimpleNamespace):
        def wait_stream(self, other):
            self.after.append(other)

    streams = []
    monkeypatch.setattr(torch.cuda, "Stream", lambda dev: streams.append(Side(after=[])) or streams[-1])
    monkeypatch.setattr(torch.cuda, "Event", lambda: None)
    mla.PrefillPipeline(1, 3, 2, bf(*W), bf(*O), topk=2)
    assert len(streams) == 3 and all(s.after == [world.current] for s in streams)
    assert len(world.made) == 11  # two slots of four inputs and a result, and the workspace
    assert all(t.users == streams for t in world.made)
