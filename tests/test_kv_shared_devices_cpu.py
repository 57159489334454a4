"""The operators for batches that share what they have cached on tensors of a device that is not the current one."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from test_kv_devices_cpu import kv, tensors  # noqa: F401


def calls(kv, where):  # noqa: F811
    from w4a16_group_quantised_gb300 import beam
    k, s, table, ints = tensors(where)
    cache = kv.KVCache(k, k, s, s)
    q = torch.empty((1, 4, 128), dtype=torch.float16, device=where)
    starts = torch.empty(3, dtype=torch.int32, device=where)
    ref, one = torch.empty(4, dtype=torch.int32, device=where), torch.empty(1, dtype=torch.int32, device=where)
    return {
        "shared": lambda: kv.w4a16_kv_attention_shared(q, cache, table, ints, starts, 1, ints, one),
        "grow": lambda: kv.w4a16_kv_grow(cache, table, ints, ref, ints, 3),
        "reorder": lambda: kv.w4a16_kv_reorder(table, ints, ref, ints),
        "select": lambda: beam.w4a16_beam_select(torch.empty((4, 50), device=where), torch.empty(4, device=where), 2, 2),
    }


NAMES = ["shared", "grow", "reorder", "select"]


@pytest.fixture
def both(kv, monkeypatch):  # noqa: F811
    from w4a16_group_quantised_gb300 import beam
    monkeypatch.setattr(beam, "load_library", kv.load_library)
    return kv


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_device_are_refused(both, name):
    with FakeTensorMode():
        with pytest.raises(ValueError, match="cuda:1, the current device is cuda:0"):
            calls(both, "cuda:1")[name]()


@pytest.mark.parametrize("name", NAMES)
def test_those_of_the_current_one_get_as_far_as_the_library(both, name):
    with FakeTensorMode():
        with pytest.raises(Exception) as e:
            calls(both, "cuda:0")[name]()
        assert not isinstance(e.value, (ValueError, TypeError)), e.value


def test_shapes_and_types_are_refused(both):
    """What the binding looks at itself."""
    from w4a16_group_quantised_gb300 import beam
    with FakeTensorMode():
        k, s, table, ints = tensors("cuda:0")
        cache = both.KVCache(k, k, s, s)
        q = torch.empty((1, 4, 128), dtype=torch.float16, device="cuda:0")
        starts, ref = (torch.empty(n, dtype=torch.int32, device="cuda:0") for n in (3, 4))
        with pytest.raises(ValueError, match="group_starts"):
            both.w4a16_kv_attention_shared(q, cache, table, ints, starts, 1, ints, ints)
        with pytest.raises(TypeError, match="prefix_lens"):
            both.w4a16_kv_attention_shared(q, cache, table, ints, starts, 1, starts, ints.long())
        with pytest.raises(ValueError, match="new_lens"):
            both.w4a16_kv_grow(cache, table, ints, ref, starts, 3)
        with pytest.raises(ValueError, match="refcount"):
            both.w4a16_kv_grow(cache, table, ints, starts, ints, 3)
        with pytest.raises(ValueError, match="same length"):
            both.w4a16_kv_reorder(table, ints, ref, ints, starts)
        x, sc = torch.empty((4, 50), device="cuda:0"), torch.empty(4, device="cuda:0")
        with pytest.raises(ValueError, match="width"):
            beam.w4a16_beam_select(x, sc, 3, 2)
        with pytest.raises(TypeError, match="logits"):
            beam.w4a16_beam_select(x.double(), sc, 2, 2)
        with pytest.raises(ValueError, match="contiguous rows"):
            beam.w4a16_beam_select(x.t(), torch.empty(50, device="cuda:0"), 2, 2)
        with pytest.raises(TypeError, match="finished"):
            beam.w4a16_beam_select(x, sc, 2, 2, finished=torch.empty(4, dtype=torch.uint8, device="cuda:0"))
        with pytest.raises(ValueError, match="scores"):
            beam.w4a16_beam_select(x, sc[:3], 2, 2)
