"""Which device the binding launches on, with a fake of torch's device calls (no GPU)."""
import pytest

from int2_kv_cache_rotate_b200 import okv

torch = pytest.importorskip("torch")


class _Tensor:
    def __init__(self, device):
        self.device = torch.device("cuda", device)

    def get_device(self):
        return self.device.index


class _Device:
    """torch.cuda.device of a machine with several GPUs."""
    current = 0

    def __init__(self, index):
        self.index = index if isinstance(index, int) else index.index

    def __enter__(self):
        self.before, _Device.current = _Device.current, self.index

    def __exit__(self, *exc):
        _Device.current = self.before


class _Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def two_devices(monkeypatch):
    monkeypatch.setattr(_Device, "current", 0)
    monkeypatch.setattr(torch.cuda, "device", _Device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: _Stream(100 + _Device.current))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: _Device.current, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 100 + dev, raising=False)


@pytest.mark.parametrize("device", [0, 1])
@pytest.mark.parametrize("stream,handle", [(None, None), (_Stream(7), 7)])
def test_a_prepared_step_runs_on_its_tensors_device(two_devices, device, stream, handle):
    seen = []
    step = object.__new__(okv.DecodeStepCall)
    step.out, step._stream, step._args, step._want_graph, step._graph = _Tensor(device), stream, (1, 2), False, None
    step._fn = lambda *a: seen.append((_Device.current, a)) or okv.OK
    assert step() is step.out and _Device.current == 0
    assert seen == [(device, (1, 2, handle or 100 + device))]


@pytest.mark.parametrize("device", [0, 1])
@pytest.mark.parametrize("stream,handle", [(None, None), (_Stream(7), 7)])
def test_without_torchs_private_short_cuts(two_devices, monkeypatch, device, stream, handle):
    monkeypatch.delattr(torch._C, "_cuda_getDevice", raising=False)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: _Device.current)
    seen = []
    okv._run(_Tensor(device), stream, lambda *a: seen.append((_Device.current, a)) or okv.OK, 5)
    assert seen == [(device, (5, handle or 100 + device))] and _Device.current == 0
