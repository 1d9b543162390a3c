"""Rotation and the 8-bit cache's functions called with another device current than
the tensors': the library is entered with theirs, on their device's stream."""
import pytest
import torch

import exact_attention_58_gb300 as ea
from test_paged_device import Machine


@pytest.mark.parametrize("stream,handle", [(None, 0x100), (0x77, 0x77)])
def test_functions_pass_the_tensors_device(monkeypatch, stream, handle):
    m = Machine(monkeypatch, 1)

    class Library:
        attn_rope = attn_cache_append_rope = attn_cache_append_fp8 = attn_fwd_paged_fp8 = staticmethod(m.entry)
        attn_fwd_paged_workspace_size = staticmethod(lambda *a: 256)

    class Extension:   # leaves the call to the Python functions, as it does on another device
        rope = cache_append_rope = cache_append_fp8 = fwd_paged_fp8 = staticmethod(lambda *a: None)

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
        made.append(device.index)
        return there(*((shape,) if isinstance(shape, int) else shape), dtype=dtype)

    monkeypatch.setattr(ea, "_empty", empty)
    half, f32 = torch.bfloat16, torch.float32
    rows, dense, freq = there(4, 2, 64, dtype=half), there(1, 2, 4, 64, dtype=half), there(32, dtype=f32)
    cache, slots = there(3, 2, 16, 64, dtype=half), there(4, dtype=torch.int64)
    c8, scale = there(3, 2, 16, 64, dtype=torch.float8_e4m3fn), there(3, 2, dtype=f32)
    ea.attn_rope(dense, dense, freq, stream=stream)
    ea.attn_rope(rows, None, freq, there(4), stream=stream)
    ea.attn_cache_append_rope(rows, rows, rows, cache, cache, slots, freq, there(4), stream=stream)
    ea.attn_cache_append_fp8(rows, rows, c8, c8, scale, scale, slots, stream=stream)
    ea.attn_fwd_paged_fp8(rows, c8, c8, scale, scale, there(4, 2), there(4), there(5), 1, stream=stream)
    assert [current for current, _ in m.calls] == [0] * 5 and m.current == 1
    assert all(args[-1] == handle for _, args in m.calls)
    assert set(made) == {0}
