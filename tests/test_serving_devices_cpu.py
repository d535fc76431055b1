"""The binding refuses a call whose caches, prefixes or adapters lie on another device than the
current one: the kernels would follow their pointers.  Devices, tensors and the library are fakes."""
import math

import pytest
import torch

from intra_spatial_pipelining_gb300 import sgp


class Fake:
    """What the binding asks of a tensor, on a device that this machine does not have."""

    def __init__(self, dtype, *shape, dev=0):
        self.dtype, self.shape, self.dev = dtype, torch.Size(shape), dev

    def get_device(self):
        return self.dev

    @property
    def device(self):
        return torch.device("cuda", self.dev)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return math.prod(self.shape)

    def is_contiguous(self):
        return True

    def stride(self):
        return tuple(math.prod(self.shape[i + 1:]) for i in range(len(self.shape)))

    def data_ptr(self):
        return 4096


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def env(monkeypatch):
    sgp._dev()                                      # the first call loads torch's types
    lib, current = Library(), [0]
    monkeypatch.setattr(sgp, "_dev", lambda: current[0])
    monkeypatch.setattr(sgp, "_raw_stream", lambda dev: 0, raising=False)
    monkeypatch.setattr(sgp, "lib", lambda: lib)
    return lib, current


BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def calls(current, dev_cache, dev_prefix, dev_to, dev_lora):
    """The four operators on device 0, with the built structures on the devices given."""
    def on(dev, build):
        current[0] = dev                            # the builders check against the current device
        out = build(lambda dtype, *shape: Fake(dtype, *shape, dev=dev))
        current[0] = 0
        return out
    d = sgp.make_heads(8, 2)
    cache = on(dev_cache, lambda t: sgp.make_cache(t(BF, 3, 2, 10, 64), t(BF, 3, 2, 10, 64)))
    to = on(dev_to, lambda t: sgp.make_cache(t(BF, 3, 2, 9, 64), t(BF, 3, 2, 9, 64)))
    prefix = on(dev_prefix, lambda t: sgp.make_prefix(t(BF, 1, 2, 7, 64), t(BF, 1, 2, 7, 64), t(I32, 1), t(I32, 3)))
    lora = on(dev_lora, lambda t: sgp.make_lora(t(BF, 2, 16, 64), t(BF, 2, 96, 16), t(F32, 2), t(I32, 2)))
    n, q, o, lse, ws = Fake(I32, 3), Fake(BF, 3, 8, 64), Fake(BF, 3, 8, 64), Fake(F32, 3, 8), Fake(U8, 1 << 20)
    acc, acc2, x, y = Fake(F32, 3, 2, 10), Fake(F32, 3, 2, 9), Fake(BF, 3, 64), Fake(BF, 3, 96)
    return {
        "sgp_prefix_attention": lambda: sgp.sgp_prefix_attention(d, cache, prefix, n, q, o, lse, 3, ws),
        "sgp_attention_weights": lambda: sgp.sgp_attention_weights(d, cache, n, q, lse, acc, 3, ws),
        "sgp_kv_evict": lambda: sgp.sgp_kv_evict(d, cache, to, sgp.make_evict(8), n, n, acc, acc2, None, 3, ws),
        "sgp_lora_apply": lambda: sgp.sgp_lora_apply(lora, n, x, y, y, 3, ws)}


def test_everything_on_the_current_device_is_called(env):
    lib, current = env
    for name, call in calls(current, 0, 0, 0, 0).items():
        call()
        assert lib.calls[-1] == name


@pytest.mark.parametrize("name,devices", [
    ("sgp_prefix_attention", (1, 0, 0, 0)), ("sgp_prefix_attention", (0, 1, 0, 0)),
    ("sgp_attention_weights", (1, 0, 0, 0)), ("sgp_kv_evict", (1, 0, 0, 0)), ("sgp_kv_evict", (0, 0, 1, 0)),
    ("sgp_lora_apply", (0, 0, 0, 1))])
def test_structures_of_another_device_are_refused(env, name, devices):
    lib, current = env
    with pytest.raises(ValueError, match="device"):
        calls(current, *devices)[name]()
    assert not lib.calls
