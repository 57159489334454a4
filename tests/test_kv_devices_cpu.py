"""The cache's tensors have to be on the current device, where the library launches.  Tensors without memory stand in for a
second GPU's."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode


@pytest.fixture
def kv(monkeypatch):
    from w4a16_group_quantised_gb300 import kv

    class Never:
        def __getattr__(self, name):
            raise AssertionError(f"the library was asked for {name}")

    monkeypatch.setattr(kv, "load_library", lambda: Never())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    return kv


def tensors(where):
    k = torch.empty((4, 2, 16, 128), dtype=torch.int8, device=where)
    s = torch.empty((4, 2), device=where)
    table = torch.empty((2, 3), dtype=torch.int32, device=where)
    ints = torch.empty(2, dtype=torch.int32, device=where)
    return k, s, table, ints


def calls(kv, where):
    k, s, table, ints = tensors(where)
    cache = kv.KVCache(k, k, s, s)
    q = torch.empty((1, 4, 128), dtype=torch.float16, device=where)
    new = torch.empty((1, 2, 128), dtype=torch.float16, device=where)
    starts = torch.empty(3, dtype=torch.int32, device=where)
    ref = torch.empty(4, dtype=torch.int32, device=where)
    return {
        "append": lambda: kv.w4a16_kv_append(cache, new, new, table, ints, starts),
        "read": lambda: kv.w4a16_kv_read(cache, table, ints, starts, 1, torch.float16),
        "attention": lambda: kv.w4a16_kv_attention(q, cache, table, ints, starts, 1),
        "copy": lambda: kv.w4a16_kv_copy_pages(cache, ints, ints),
        "fork": lambda: kv.w4a16_kv_fork(cache, table, ints, ref, ints, ints),
        "free": lambda: kv.w4a16_kv_free(table, ints, ref, ints),
        "trim": lambda: kv.w4a16_kv_trim(table, ints, ref, 16, 4),
        "compact": lambda: kv.w4a16_kv_compact(cache, table, ref),
    }


NAMES = ["append", "read", "attention", "copy", "fork", "free", "trim", "compact"]


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_device_are_refused(kv, name):
    with FakeTensorMode():
        with pytest.raises(ValueError, match="cuda:1, the current device is cuda:0"):
            calls(kv, "cuda:1")[name]()


@pytest.mark.parametrize("name", NAMES)
def test_those_of_the_current_one_get_as_far_as_the_library(kv, name):
    # past every check of devices, to the first thing that needs memory or the library
    with FakeTensorMode():
        with pytest.raises(Exception) as e:
            calls(kv, "cuda:0")[name]()
        assert not isinstance(e.value, (ValueError, TypeError)), e.value
