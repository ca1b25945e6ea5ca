"""Host side of the dense experts: what is shown without a GPU."""
import pytest

torch = pytest.importorskip("torch")

from dynamic_any_precision_b200 import dpa  # noqa: E402
from dynamic_any_precision_b200.stack import DenseStack  # noqa: E402


def test_dense_stack_runs_on_the_device_of_its_stream_of_rows(monkeypatch):
    # every launch with the device of h current, whichever was current before
    current, seen = ["cuda:0"], []

    class Device:
        def __init__(self, device):
            self.device = str(device)

        def __enter__(self):
            self.before, current[0] = current[0], self.device

        def __exit__(self, *exc):
            current[0] = self.before

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(dpa, "residual_rmsnorm", lambda h, x, y=None, stream=None: seen.append(current[0]))
    monkeypatch.setattr(dpa, "dense_moe_forward", lambda *args, **kw: seen.append(current[0]))
    stack = DenseStack.__new__(DenseStack)
    stack.layers = [object(), object()]
    h = torch.zeros((2, 4), device="meta")
    stack.forward(h, {"x": None, "y": None})
    assert seen == ["meta"] * 5 and current[0] == "cuda:0"
