"""The binding of the K/V cache without a GPU: which tensors its calls take.
CPU tensors stand in for device ones, so calls that pass the checks are not made."""
import pytest
import torch


class OnGpu(torch.Tensor):
    is_cuda = True


def on_gpu(*shape, dtype=torch.float16):
    """Aligned as device memory is."""
    n = 1
    for d in shape:
        n *= d
    t = torch.zeros(n + 64, dtype=dtype)
    skip = -t.data_ptr() % 64 // t.element_size()
    return t[skip:skip + n].view(shape).as_subclass(OnGpu)


@pytest.fixture(scope="module")
def us():
    from bitmap_encoded_unstructured_ie_gb300 import binding, build
    build.build()
    binding.load()
    return binding


def cache(us, scale=torch.float16, k=torch.uint8, v=torch.uint8):
    return us.KVCache(us.US_I8, 64, on_gpu(3, 2, 16, 64, dtype=k), on_gpu(3, 2, 16, 64, dtype=v),
                      on_gpu(3, 2, 16, 2, dtype=scale), on_gpu(1, 3, dtype=torch.int32))


def ints(n):
    return on_gpu(n, dtype=torch.int32)


BITS = [torch.float16, torch.int16, torch.uint16]             # fp16, or its bit pattern


@pytest.mark.parametrize("dtype", BITS)
def test_fp16_and_its_bits_are_taken(us, dtype):
    C = cache(us, scale=dtype)
    T, ptr, ld = us._rows(on_gpu(5, 2, 64, dtype=dtype), 2, C)
    assert (T, ld) == (5, 128) and ptr


def test_other_16_bit_types_are_refused(us):
    C, off, pos = cache(us), ints(2), ints(1)
    x, y = on_gpu(3, 2, 64), on_gpu(3, 2, 64, dtype=torch.bfloat16)
    ws = on_gpu(64, dtype=torch.uint8)
    for k, v in ((x, y), (y, x)):
        with pytest.raises(AssertionError, match="fp16"):
            us.us_kv_write(C, k, v, off, pos, 3)
        with pytest.raises(AssertionError, match="fp16"):
            us.us_kv_read(C, off, pos, 3, k, v)
        with pytest.raises(AssertionError, match="fp16"):
            us.us_attn_kv(C, k, off, pos, None, 3, 0.1, v, ws)
    with pytest.raises(AssertionError, match="fp16"):
        cache(us, scale=torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.float64, torch.int32])
def test_masks_are_64_bit_words(us, dtype):
    x = on_gpu(3, 2, 64)
    with pytest.raises(AssertionError, match="64-bit"):
        us.us_attn_kv(cache(us), x, ints(2), ints(1), on_gpu(3, dtype=dtype), 3, 0.1, x, on_gpu(64, dtype=torch.uint8))


@pytest.mark.parametrize("kw", [dict(k=torch.float8_e4m3fn), dict(v=torch.bool)])
def test_codes_are_bytes(us, kw):
    with pytest.raises(AssertionError, match="bytes"):
        cache(us, **kw)


class OnOther(OnGpu):
    def get_device(self):
        return 1


def calls(us, C, k, off, pos, mask, ws, stream=None):
    yield lambda: us.us_kv_write(C, k, k, off, pos, 3, stream=stream)
    yield lambda: us.us_kv_read(C, off, pos, 3, k, k, stream=stream)
    yield lambda: us.us_kv_commit(C, off, ints(3), pos, 3, stream=stream)
    yield lambda: us.us_attn_kv(C, k, off, pos, mask, 3, 0.1, k, ws, stream=stream)


def test_one_device_for_the_call_its_stream_and_its_tensors(us, monkeypatch):
    """A stream's handle is of the current device, and so is the launch: the cache has to be there too."""
    monkeypatch.setattr(OnGpu, "get_device", lambda t: 0, raising=False)
    C, x, off, pos = cache(us), on_gpu(3, 2, 64), ints(2), ints(1)
    m, ws = on_gpu(3, dtype=torch.int64), on_gpu(64, dtype=torch.uint8)
    for device, stream in ((1, None), (1, 0), (0, 1)):
        monkeypatch.setattr(us, "_current_device", lambda: device)
        st = None if stream is None else type("Stream", (), {"device_index": stream, "cuda_stream": 0})()
        for call in calls(us, C, x, off, pos, m, ws, st):
            with pytest.raises(AssertionError, match="device"):
                call()
    monkeypatch.setattr(us, "_current_device", lambda: 0)
    other = [t.as_subclass(OnOther) for t in (x, off, pos, m, ws)]
    for i in range(5):
        args = [other[j] if j == i else t for j, t in enumerate((x, off, pos, m, ws))]
        made = list(calls(us, C, *args))
        for call in made if i < 3 else made[3:]:
            if i == 0 and call is made[2]:
                continue                                       # a commit has no rows
            with pytest.raises(AssertionError, match="device"):
                call()
    with pytest.raises(AssertionError, match="device"):
        us.KVCache(us.US_I8, 64, C.k, C.v.as_subclass(OnOther), C.scale, C.page_table)
