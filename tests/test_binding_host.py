"""The binding's checks of workspaces, without a GPU."""
import pytest
import torch

from vision_transformer_encoder_dsv4v_b200 import dsv4v as A


class OnDevice:
    """What the binding asks of a workspace tensor."""

    def __init__(self, index, elements=100, size=1, contiguous=True):
        self.index, self.elements, self.size, self.contiguous = index, elements, size, contiguous
        self.is_cuda, self.device = True, f"cuda:{index}"

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.contiguous

    def numel(self):
        return self.elements

    def element_size(self):
        return self.size

    def data_ptr(self):
        return 4096


def test_host_workspace_is_refused():
    # the kernels would take its address for one of theirs
    with pytest.raises(ValueError, match="workspace is on cpu"):
        A._ws(torch.empty(1 << 20, dtype=torch.uint8))


def test_workspace_of_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(A, "_device_index", lambda: 0)
    with pytest.raises(ValueError, match="workspace is on cuda:1"):
        A._ws(OnDevice(1))
    with pytest.raises(ValueError, match="not contiguous"):
        A._ws(OnDevice(0, contiguous=False))


def test_workspace_is_measured_in_bytes(monkeypatch):
    monkeypatch.setattr(A, "_device_index", lambda: 0)
    assert A._ws(OnDevice(0, 100, 1)) == (4096, 100)
    assert A._ws(OnDevice(0, 100, 4)) == (4096, 400)
    assert A._ws(None) == (None, 0)


@pytest.mark.parametrize("call", ["linear_backward", "grad_norm"])
def test_calls_refuse_a_host_workspace(monkeypatch, call):
    host = torch.empty(1 << 20, dtype=torch.uint8)
    monkeypatch.setattr(A, "lib", lambda: type("L", (), {"dsv4v_linear_backward": lambda *a: pytest.fail("reached"),
                                                         "dsv4v_grad_norm": lambda *a: pytest.fail("reached")})())
    monkeypatch.setattr(A, "_device_index", lambda: 0)
    monkeypatch.setattr(A, "_raw_stream", lambda stream, device: 0)
    monkeypatch.setattr(A, "_matrix", lambda *a: 4096)
    monkeypatch.setattr(A, "_value", lambda *a: 4096)
    with pytest.raises(ValueError, match="workspace is on cpu"):
        if call == "linear_backward":
            A.dsv4v_linear_backward(A.make_linear(4, 64, 8), None, None, None, None, None, None, None, host)
        else:
            A.dsv4v_grad_norm(A.GradTable([]), None, host)
