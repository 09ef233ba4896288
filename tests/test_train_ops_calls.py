"""The training operators' torch layer without a GPU: which device and stream a call takes."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

from mixed_precision_optimizer_bf16_gb300 import train_ops as ops  # noqa: E402


def test_host_tensors_by_name_are_refused():
    z = torch.zeros(2, 8)
    for call in (lambda: ops.distill_forward(logits=z, teacher_ids=z.int(), teacher_logits=z),
                 lambda: ops.distill_backward(logits=z, teacher_ids=z.int(), teacher_logits=z, lse=z),
                 lambda: ops.distill_loss_grad(logits=z, teacher_ids=z.int(), teacher_logits=z),
                 lambda: ops.norm_gate_forward(x=z, y=z), lambda: ops.norm_gate_backward(dr=None, dh=None, r=z, y=z, stats=z),
                 lambda: ops.balance_forward(logits=z, k=2), lambda: ops.balance_backward(logits=z, ids=z.int(), counts=z.int(), saved=z),
                 lambda: ops.norm_gate_backward(None, None, None, z, z), lambda: ops.norm_gate_backward(None, None, None, None, None)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


class Device:
    """Stands in for torch.cuda and for tensors on its devices; keeps the stream and device that a call ran on."""

    class Tensor:
        is_cuda = True

        def __init__(self, index, used):
            self.index, self.used = index, used

        def get_device(self):
            return self.index

        def record_stream(self, stream):
            self.used.append((self, stream))

    def __init__(self, monkeypatch):
        self.now, self.streams, self.used = 0, {0: "default 0", 1: "default 1"}, []
        monkeypatch.setattr(ops, "_Tensor", self.Tensor)
        monkeypatch.setattr(ops, "_current_device", lambda: self.now)
        monkeypatch.setattr(torch.cuda, "device", self.device)
        monkeypatch.setattr(torch.cuda, "stream", self.stream)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda index: self.streams[index])

    @contextlib.contextmanager
    def device(self, index):
        before, self.now = self.now, index
        yield
        self.now = before

    @contextlib.contextmanager
    def stream(self, stream):
        before, self.streams[self.now] = self.streams[self.now], stream
        yield
        self.streams[self.now] = before

    def tensor(self, index):
        return self.Tensor(index, self.used)


@pytest.mark.parametrize("place", [lambda t, u: ((t, u), {}), lambda t, u: ((None, t), {"y": u}), lambda t, u: ((None,), {"dh": t, "y": u}),
                                   lambda t, u: ((), {"k": 3, "logits": t, "mask": u}), lambda t, u: ((None, None), {"gate": None, "r": t, "y": u})])
@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("stream", [None, "side"])
def test_a_call_takes_the_device_and_the_stream_of_its_tensors(place, index, stream, monkeypatch):
    cuda = Device(monkeypatch)
    ran = ops._on_stream(lambda *args, **more: (cuda.now, cuda.streams[cuda.now]))
    t, u = cuda.tensor(index), cuda.tensor(index)
    args, more = place(t, u)
    assert ran(*args, stream=stream, **more) == (index, stream or f"default {index}")
    assert cuda.now == 0 and cuda.streams == {0: "default 0", 1: "default 1"}
    assert [x for x, _ in cuda.used] == ([t, u] if stream else []) and all(s == "side" for _, s in cuda.used)
