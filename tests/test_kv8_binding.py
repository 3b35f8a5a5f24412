"""The 8-bit cache's binding refuses tensors of different devices, without a GPU: CPU tensors that say
that they are CUDA tensors of a device stand in, and the library's functions must not be reached."""

import pytest
import torch


class OnDevice(torch.Tensor):
    """A tensor that says it is on the CUDA device `index` (0 unless set)."""

    index = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.index


def on(index, *shape, dtype=torch.float32):
    t = torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)
    t.index = index
    return t


CODES, SCALES, I32 = (8, 2, 32, 64), (8, 2), torch.int32


def cache_on(q, index):
    return q.Kv8Cache(*(on(index, *CODES, dtype=torch.int8) for _ in range(2)), *(on(index, *SCALES) for _ in range(2)))


def calls(q):
    """Each operator's call as (function, its tensors by name, other arguments), of a cache of 2 sequences."""
    table, lens, row_start = on(0, 2, 4, dtype=I32), on(0, 2, dtype=I32), on(0, 3, dtype=I32)
    rows = dict(page_table=table, lens=lens, row_start=row_start)
    k_and_v = dict(k=on(0, 5, 128), v=on(0, 5, 128))
    evict = dict(page_table=table, lens=lens, weights=on(0, 2, 2, 128), fresh_pages=on(0, 2, 2, dtype=I32),
                 table_out=on(0, 2, 4, dtype=I32), lens_out=on(0, 2, dtype=I32), weights_out=on(0, 2, 2, 40),
                 kept=on(0, 2, 2, 40, dtype=I32))
    attend = dict(rows, q=on(0, 5, 256), out=on(0, 5, 256), weights=on(0, 2, 2, 128))
    return [(q.apr_kv8_append, dict(rows, **k_and_v), {}), (q.apr_kv8_read, dict(rows, **k_and_v), {}),
            (q.apr_kv8_attention, attend, dict(num_heads=4)), (q.apr_kv8_evict, evict, dict(budget=40, recent=8))]


class Unreached:
    def __getattr__(self, name):
        def call(*args):
            raise AssertionError(f"{name} was called")

        return call


@pytest.fixture
def kv8(q, monkeypatch):
    from quantized_weight_prefill_q4_gb300 import kv8

    monkeypatch.setattr(kv8, "_lib", Unreached())
    monkeypatch.setattr(kv8, "_current_device", lambda: 0)
    monkeypatch.setattr(kv8, "_raw_stream", lambda index: 0)
    return kv8


@pytest.mark.parametrize("which", range(4))
def test_tensors_of_another_device_are_refused(q, kv8, which):
    call, tensors, more = calls(q)[which]
    with pytest.raises(AssertionError, match="was called"):  # all on one device: the library is reached
        call(cache_on(q, 0), **tensors, **more)
    for name, t in tensors.items():
        other = on(1, *t.shape, dtype=t.dtype)
        with pytest.raises(ValueError, match=f"{name}: tensor is on device 1, the cache on 0"):
            call(cache_on(q, 0), **{**tensors, name: other}, **more)


@pytest.mark.parametrize("which", range(4))
def test_a_cache_of_another_device_than_the_current_one_is_refused(q, kv8, which, monkeypatch):
    call, tensors, more = calls(q)[which]
    monkeypatch.setattr(kv8, "_current_device", lambda: 2)
    for stream in (None, 1234):
        with pytest.raises(ValueError, match="device 0, the current device is 2"):
            call(cache_on(q, 0), **tensors, **more, stream=stream)


def test_a_cache_of_arrays_of_two_devices_is_refused(q):
    arrays = [on(0, *CODES, dtype=torch.int8), on(0, *CODES, dtype=torch.int8), on(0, *SCALES), on(0, *SCALES)]
    q.Kv8Cache(*arrays)
    for i, name in ((1, "V"), (2, "k_scale"), (3, "v_scale")):
        other = on(1, *arrays[i].shape, dtype=arrays[i].dtype)
        with pytest.raises(ValueError, match=f"{name}: tensor is on device 1"):
            q.Kv8Cache(*arrays[:i], other, *arrays[i + 1:])
