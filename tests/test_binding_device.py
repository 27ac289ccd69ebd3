"""Which device and stream a call of the binding runs on: the operands', also
where another device is the current one."""
import inspect
import re

import pytest
import torch

import w8a8_quantized_linear_quant_amd as w8


class Devices:
    """Four devices as the binding sees them; `current` as torch.cuda.device moves it."""

    def __init__(self, monkeypatch):
        self.current, self.entered, outer = 0, [], self

        class Guard:
            def __init__(self, device):
                self.index = device.index if device.index is not None else outer.current

            def __enter__(self):
                self.before, outer.current = outer.current, self.index
                outer.entered.append(self.index)

            def __exit__(self, *_):
                outer.current = self.before

        monkeypatch.setattr(torch.cuda, "device", Guard)
        monkeypatch.setattr(w8, "_raw_device", lambda: self.current)
        monkeypatch.setattr(w8, "_raw_stream", lambda index: 100 + index)
        self.calls = []

    def entry(self, status=0):
        def call(*args):
            self.calls.append((self.current, args))
            return status
        return call


@pytest.fixture
def devices(monkeypatch):
    return Devices(monkeypatch)


@pytest.mark.parametrize("name,at", [("cuda:0", 0), ("cuda:1", 1), ("cuda:3", 3), ("cuda", 0)])
def test_the_operands_device_is_current_during_a_call(devices, name, at):
    w8._launch(devices.entry(), torch.device(name), 7, None, 2.5)
    assert devices.calls == [(at, (7, None, 2.5, 100 + at))] and devices.current == 0


def test_no_switch_where_it_is_current(devices):
    devices.current = 2
    w8._launch(devices.entry(), torch.device("cuda:2"))
    assert devices.calls == [(2, (102,))] and devices.entered == []


@pytest.mark.parametrize("name", ["cuda:0", "cuda:1"])
def test_the_current_device_comes_back_after_an_error(devices, name):
    with pytest.raises(w8.W8A8Error, match="SHAPE"):
        w8._launch(devices.entry(status=2), torch.device(name))
    assert devices.current == 0

    def broken(*_):
        raise TypeError("argument")
    with pytest.raises(TypeError):
        w8._launch(broken, torch.device(name))
    assert devices.current == 0


def test_every_call_with_a_stream_goes_this_way():
    """Entry points whose C declaration ends in a stream are called by _launch alone."""
    source = inspect.getsource(w8)
    streams = set()
    for header in (w8.HEADER, w8.BLOCK_HEADER, w8.EXPERTS_HEADER, w8.PROBE_HEADER):
        with open(header) as f:
            streams |= set(re.findall(r"(\w+)\([^()]*hipStream_t stream\)\s*;", f.read()))
    assert len(streams) > 25 and "mxfp4_linear_grouped" in streams and "lora_forward" in streams
    launched = set(re.findall(r"_launch\(_lib\.(\w+), ", source))
    called = set(re.findall(r"_lib\.(\w+)\(", source))
    assert launched <= streams and not called & streams


@pytest.mark.gpu
def test_results_where_another_device_is_current(monkeypatch):
    """The way through torch.cuda.device, with the binding told that device 1 is the current one."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn(5, 64, generator=g).bfloat16().cuda(), torch.randn(2, 40, 64, generator=g).bfloat16().cuda()
    offsets = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")

    def both():
        wq, _, ws = w8.w8a8_quant_weight_grouped(w)
        y = w8.w8a8_linear_grouped(*w8.w8a8_quant_act_rowwise(x), wq, ws, offsets)
        return y, w8.mxfp4_linear(*w8.mxfp4_quantize(x), *w8.mxfp4_quantize(w[0]))

    first = both()
    asked = []
    monkeypatch.setattr(w8, "_raw_device", lambda: asked.append(1) or 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = both()
    torch.cuda.current_stream().wait_stream(side)
    assert len(asked) == 7 and all(torch.equal(a, b) for a, b in zip(first, second))
