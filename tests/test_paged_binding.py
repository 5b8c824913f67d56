"""The serving calls' binding, on the host: what it checks before it launches."""
import sys

import pytest

torch = pytest.importorskip("torch")
from quantized_attention_smooth_gb300 import sage  # noqa: E402


class Rows:
    """Stands for a dense (3, 2, 64) tensor on a CUDA device."""
    is_cuda, dtype, shape = True, torch.bfloat16, (3, 2, 64)

    def __init__(self, index):
        self.index, self.device = index, f"cuda:{index}"

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x100000


def held(index):
    """A cache and a batch built on device `index`."""
    cache, batch = object.__new__(sage.PagedCache), object.__new__(sage.PagedBatch)
    cache.Hkv, cache.D, cache._dev, batch._dev = 2, 64, index, index
    return cache, batch


@pytest.mark.parametrize("cache_on,batch_on,name", [(0, 1, "cache"), (1, 0, "batch"), (0, 0, "cache")])
def test_cache_and_batch_of_another_device(monkeypatch, cache_on, batch_on, name):
    """The call's tensors are on the current device, the cache or the batch is not."""
    monkeypatch.setattr(sage, "_torch", torch)
    monkeypatch.setattr(sage, "_get_device", lambda: 1)
    monkeypatch.setattr(sage, "_get_stream", lambda d: 0)
    monkeypatch.setattr(sage, "_CODES", {torch.bfloat16: sage.BF16})
    monkeypatch.setattr(sage, "_empty_like", lambda t: t)
    cache, batch = held(cache_on)[0], held(batch_on)[1]
    x = Rows(1)
    with pytest.raises(ValueError, match=f"kv_append: the {name} is on cuda:0, the current device"):
        sage.kv_append(cache, batch, x, x)
    with pytest.raises(ValueError, match=f"attn_paged: the {name} is on cuda:0, the current device"):
        sage.attn_paged(cache, batch, x)


def test_first_calls_of_two_threads(monkeypatch):
    """A thread that sees _torch set finds everything set that goes with it: no
    line of the binding runs with _torch set and the rest not."""
    names = ("_torch", "_get_device", "_get_stream", "_empty_like")
    for n in names:
        monkeypatch.setattr(sage, n, None)
    monkeypatch.setattr(sage, "_CODES", {})
    early = []

    def trace(frame, event, arg):
        if frame.f_code is sage._bind_torch.__code__:
            if sage._torch is not None and not (sage._CODES and all(getattr(sage, n) for n in names)):
                early.append(frame.f_lineno)
            return trace
        return None

    before = sys.gettrace()
    sys.settrace(trace)
    try:
        sage._bind_torch()
    finally:
        sys.settrace(before)
    assert sage._torch is torch and not early


@pytest.mark.parametrize("name", ["max_q", "max_kv"])
@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32 + 5, -1, -2 ** 32])
def test_bounds_that_pass_32_bits(monkeypatch, name, value):
    """The batch's bounds are 32-bit: a larger one is refused, not cut."""
    monkeypatch.setattr(sage, "_on_device", lambda *a, **k: None)
    args = dict(max_q=3, max_kv=40)
    args[name] = value
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match=f"PagedBatch: {name} must be in 0..2147483647"):
        sage.PagedBatch(torch.zeros(2, **i32), torch.zeros(1, **i32), torch.zeros(1, 3, **i32), **args)
