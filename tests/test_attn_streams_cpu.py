"""Calls of attention over the 4-bit cache with `stream=`, without a GPU: everything that a call allocates comes from that
stream's memory."""
import pytest

pytest.importorskip("torch")
attn = pytest.importorskip("post_quantization_mean_amd.attn")

from test_streams_cpu import _functions, _library_asked_for, streams  # noqa: E402, F401


def test_every_call_takes_a_stream():
    assert {f.__name__ for f in _functions(attn)} == {n for n in attn.exported_symbols() if not n.endswith("_bytes")}


@pytest.mark.parametrize("positional", [False, True])
@pytest.mark.parametrize("f", _functions(attn), ids=lambda f: f.__name__)
def test_a_call_allocates_on_its_stream(monkeypatch, streams, f, positional):  # noqa: F811
    at, s = _library_asked_for(monkeypatch, attn, "_load", f, streams[1], positional)
    assert at == [[s]]
