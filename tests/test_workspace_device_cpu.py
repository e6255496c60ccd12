"""A caller's workspace on another device than the operands is refused (the library sees only a pointer)."""
import pytest

torch = pytest.importorskip("torch")
binding = pytest.importorskip("post_quantization_mean_amd.binding")


class _Tensor(torch.Tensor):
    """A host tensor that says where it is."""
    is_cuda = True
    device = property(lambda self: torch.device("cuda", self.at))


def test_a_workspace_on_another_device_is_refused():
    ws = torch.zeros(512, dtype=torch.uint8).as_subclass(_Tensor)
    ws.at = 1
    assert binding._workspace(512, torch.device("cuda", 1), ws) is ws
    with pytest.raises(ValueError, match="cuda:0"):
        binding._workspace(512, torch.device("cuda", 0), ws)
