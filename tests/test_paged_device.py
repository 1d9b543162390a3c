"""The paged-cache functions called with another device current than the
tensors': the library is entered with theirs."""
import pytest
import torch

import exact_attention_58_gb300 as ea


class Machine:
    """Two devices, of which `current` is the current one, and a library that
    notes what it is called with."""

    def __init__(self, monkeypatch, current, status=0):
        self.current, self.calls, self.status = current, [], status
        machine = self

        class Guard:
            def __init__(self, device):
                self.device = device

            def __enter__(self):
                self.before, machine.current = machine.current, self.device

            def __exit__(self, *exc):
                machine.current = self.before

        monkeypatch.setattr(torch.cuda, "device", Guard)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: self.current, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x100 + device, raising=False)

    def entry(self, *args):
        self.calls.append((self.current, args))
        return self.status


@pytest.mark.parametrize("current,device", [(0, 0), (1, 0), (0, 1)])
@pytest.mark.parametrize("stream,handle", [(None, None), (0x77, 0x77), (0, 0)])
def test_library_runs_on_the_tensors_device(monkeypatch, current, device, stream, handle):
    m = Machine(monkeypatch, current)
    ea._call(m.entry, "entry", device, stream, 1, 2)
    assert m.calls == [(device, (1, 2, 0x100 + device if handle is None else handle))]
    assert m.current == current


def test_refusal_leaves_the_current_device(monkeypatch):
    m = Machine(monkeypatch, 1, status=2)
    with pytest.raises(ea.AttnError) as e:
        ea._call(m.entry, "entry", 0, None)
    assert e.value.status == 2 and m.current == 1 and m.calls == [(0, (0x100,))]


def test_functions_pass_the_tensors_device(monkeypatch):
    """All three functions, the extension leaving the call to them (as it does where
    the tensors are not on the current device)."""
    m = Machine(monkeypatch, 1)

    class Library:
        attn_page_table = attn_cache_append = attn_fwd_paged = staticmethod(m.entry)
        attn_fwd_paged_workspace_size = staticmethod(lambda *a: 256)

    class Extension:
        page_table = cache_append = fwd_paged = staticmethod(lambda *a: None)

    monkeypatch.setattr(ea, "_native_module", Extension)
    monkeypatch.setattr(ea, "library", lambda: Library)
    monkeypatch.setattr(ea, "_on_gpu", lambda t: None)

    class OnDevice(torch.Tensor):   # host memory that says it is on device 0
        def get_device(self):
            return 0

        @property
        def device(self):
            return torch.device("cuda", 0)

    def there(*shape, dtype=torch.int32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)

    made = []

    def empty(shape, dtype, device, stream):
        made.append((device.index, m.current))
        shape = (shape,) if isinstance(shape, int) else shape
        return there(*shape, dtype=dtype)

    monkeypatch.setattr(ea, "_empty", empty)
    half = torch.bfloat16
    cache, rows = there(3, 2, 16, 64, dtype=half), there(4, 2, 64, dtype=half)
    ea.attn_page_table(there(4), there(4), there(4, 2), there(9), there(1), 16, 8)
    ea.attn_cache_append(rows, rows, cache, cache, there(4, dtype=torch.int64))
    ea.attn_fwd_paged(rows, cache, cache, there(4, 2), there(4), there(5), 1)
    assert [current for current, _ in m.calls] == [0, 0, 0] and m.current == 1
    assert all(args[-1] == 0x100 for _, args in m.calls)   # device 0's stream
    assert {device for device, _ in made} == {0}
