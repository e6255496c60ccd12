"""Calls with `stream=`, without a GPU: everything that a call allocates comes from that stream's memory, and what it returns
is known to be used on the stream that was current."""
import contextlib
import inspect

import pytest

torch = pytest.importorskip("torch")
binding = pytest.importorskip("post_quantization_mean_amd.binding")
moe = pytest.importorskip("post_quantization_mean_amd.moe")


class _Stream:
    device = torch.device("cuda", 0)
    cuda_stream = 0x5000


class _Reached(Exception):
    pass


class _Tensor(torch.Tensor):
    """A host tensor that says it is on the device and notes the streams it is recorded on."""
    device = property(lambda self: torch.device("cuda", self.index if hasattr(self, "index") else 0))

    def record_stream(self, stream):
        self.recorded = getattr(self, "recorded", []) + [stream]


@pytest.fixture
def streams(monkeypatch):
    """(current stream, streams that were made current and not left yet)."""
    current, inside = _Stream(), []

    @contextlib.contextmanager
    def enter(stream):
        inside.append(stream)
        yield
        inside.pop()

    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current)
    return current, inside


def _functions(module):
    return [f for name, f in sorted(vars(module).items()) if name.startswith("awq_") and inspect.isfunction(f)
            and f.__module__ == module.__name__ and "stream" in inspect.signature(f).parameters]


def _library_asked_for(monkeypatch, module, loader, f, inside, positional):
    """The streams that are current where f starts its work, which is to ask for the library."""
    at = []

    def load(*_):
        at.append(list(inside))
        raise _Reached

    monkeypatch.setattr(module, loader, load)
    params = list(inspect.signature(f).parameters.values())
    args = [None if p.default is inspect.Parameter.empty else p.default for p in params if p.name != "stream"]
    s = _Stream()
    with pytest.raises(_Reached):
        if positional and params[-1].name == "stream":
            f(*args, s)
        else:
            f(*args, stream=s)
    return at, s


@pytest.mark.parametrize("positional", [False, True])
@pytest.mark.parametrize("f", _functions(moe), ids=lambda f: f.__name__)
def test_a_call_of_the_experts_block_allocates_on_its_stream(monkeypatch, streams, f, positional):
    at, s = _library_asked_for(monkeypatch, moe, "_load", f, streams[1], positional)
    assert at == [[s]]


@pytest.mark.parametrize("positional", [False, True])
@pytest.mark.parametrize("f", _functions(binding), ids=lambda f: f.__name__)
def test_a_call_of_the_search_allocates_on_its_stream(monkeypatch, streams, f, positional):
    at, s = _library_asked_for(monkeypatch, binding, "load_library", f, streams[1], positional)
    assert at == [[s]]


def test_outputs_are_recorded_on_the_stream_that_was_current(streams):
    current, inside = streams
    made = [torch.zeros(2).as_subclass(_Tensor) for _ in range(3)]
    s = _Stream()

    def f(*args):
        assert inside == [s] and args == (1, None)
        return {"a": made[0], "b": (made[1], [made[2]])}

    binding._on_stream(s, f, 1, None)
    assert [t.recorded for t in made] == [[current]] * 3 and inside == []
    own = torch.zeros(2).as_subclass(_Tensor)
    binding._on_stream(current, lambda: own)
    assert not hasattr(own, "recorded")


def test_a_stream_of_another_device_is_refused(streams):
    there = torch.zeros(2).as_subclass(_Tensor)
    there.index = 1
    for args in ((there,), ([there],), ({"h": there},)):
        with pytest.raises(ValueError, match="stream"):
            binding._on_stream(_Stream(), lambda *_: None, *args)
