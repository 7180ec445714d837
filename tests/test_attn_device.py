"""The attention calls of the binding go to their tensors' device (no GPU: the library, the
tensors and the current device are stood in for), and refuse tensors that are on none."""
import contextlib

import pytest
import torch

from speculative_decode_gated_gb300 import binding


class Tensor:
    """What the binding asks of a contiguous tensor on a device."""

    def __init__(self, device, *shape, dtype=torch.bfloat16):
        self.device, self.dtype, self.shape = torch.device(device), dtype, torch.Size(shape)
        self.nbytes = 1 << 30

    def stride(self):
        out = [1]
        for n in self.shape[:0:-1]:
            out.insert(0, out[0] * n)
        return tuple(out)

    def data_ptr(self):
        return 1 << 40

    def is_contiguous(self):
        return True


class Machine:
    """Two devices, of which `now` is the current one; records the calls."""

    def __init__(self, monkeypatch, now):
        self.now, self.calls = now, []

        @contextlib.contextmanager
        def device(index):
            before, self.now = self.now, torch.device("cuda", index).index
            try:
                yield
            finally:
                self.now = before

        class Lib:
            gdn_status_string = gdn_last_error_string = staticmethod(lambda *a: b"")

        for name in ("gdn_rope_append", "gdn_paged_attn"):
            setattr(Lib, name, staticmethod(lambda *a, name=name: self.called(name, a)))
        monkeypatch.setattr(binding, "lib", lambda: Lib)
        monkeypatch.setattr(torch.cuda, "device", device)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: self.now, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 1000 + i, raising=False)
        self.status = 0

    def called(self, name, args):
        self.calls.append((name, self.now, args[-1]))
        return self.status


def step(device):
    c = binding.gdn_attn()
    c.n_tok, c.q_heads, c.kv_heads, c.head_dim = 6, 4, 2, 64
    attn = binding.Attn(c, (), torch.bfloat16, torch.device(device))
    rope = binding.Rope(binding.gdn_rope(), (Tensor(device, 32, dtype=torch.float32), None))
    q, kv, o = Tensor(device, 6, 4, 64), Tensor(device, 6, 2, 64), Tensor(device, 6, 4, 64)
    ws = Tensor(device, 1 << 30, dtype=torch.uint8)

    def both(stream=None):
        binding.gdn_rope_append(attn, rope, q, kv, kv, o, stream)
        binding.gdn_paged_attn(attn, q, o, workspace=ws, stream=stream)
    return both


@pytest.mark.parametrize("now", [0, 1])
@pytest.mark.parametrize("index", [0, 1])
def test_the_tensors_device_is_current(monkeypatch, now, index):
    m = Machine(monkeypatch, now)
    step(f"cuda:{index}")()
    assert m.calls == [("gdn_rope_append", index, 1000 + index), ("gdn_paged_attn", index, 1000 + index)]
    assert m.now == now


def test_a_given_stream_is_used(monkeypatch):
    m = Machine(monkeypatch, 0)

    class Stream:
        cuda_stream = 77
    step("cuda:1")(Stream())
    step("cuda:1")(55)
    assert [c[1:] for c in m.calls] == [(1, 77), (1, 77), (1, 55), (1, 55)]


def test_the_device_is_put_back_after_an_error(monkeypatch):
    m = Machine(monkeypatch, 0)
    m.status = 2
    with pytest.raises(binding.GdnError):
        step("cuda:1")()
    assert m.now == 0 and len(m.calls) == 1


def test_tensors_on_no_device_are_refused(monkeypatch):
    m = Machine(monkeypatch, 0)
    with pytest.raises(ValueError, match="expected a CUDA device"):
        step("cpu")()
    assert not m.calls
