"""What lies on another device than the current one never reaches the library: the decode step's calls with one argument
at a time on another device (stand-ins for CUDA tensors, no GPU)."""
import types

import pytest
import torch

import latent_moe_layer_fp32_gb300 as lm


class On(torch.Tensor):
    """A tensor that says it is on device `at`."""
    at = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.at


def on(t, at=0):
    t = t.as_subclass(On)
    t.at = at
    return t


class Called(Exception):
    pass


@pytest.fixture
def lib(monkeypatch):
    """The library as far as the descriptors need it; any of the calls raises Called."""
    def called(*_):
        raise Called

    fake = types.SimpleNamespace(lmoe_kv_maps_fp8_init=lambda *_: 0, lmoe_qk_norm_rope=called, lmoe_kv_write_fp8=called,
                                 lmoe_kv_read_fp8=called, lmoe_decode_attention_fp8=called)
    monkeypatch.setattr(lm, "load", lambda *_: fake)
    monkeypatch.setattr(lm, "_device", lambda: 0)
    monkeypatch.setattr(lm, "_raw_stream", lambda dev: 0)


def pages(at=0):
    shape = (4, 2, 16, 64)
    return [on(torch.zeros(shape, dtype=torch.uint8), at) for _ in range(2)] + \
        [on(torch.zeros(shape[:3], dtype=torch.uint8), at) for _ in range(2)]


def rows(n=3, heads=2):
    return on(torch.zeros(n, heads, 64, dtype=torch.bfloat16))


def ints(*shape):
    return on(torch.zeros(*shape, dtype=torch.int32))


def calls():
    """Each call's function and its tensors and cache, all on device 0."""
    cache, ws = lm.kv_cache_fp8_of(*pages()), on(torch.zeros(64, dtype=torch.uint8))
    return {
        "rope": (lm.lmoe_qk_norm_rope, dict(
            dims=lm.rope_dims_of(3, 4, 2, 64), q=rows(3, 4), k=rows(), q_gain=rows()[0, 0], k_gain=rows()[0, 0], pos=ints(1, 3),
            inv_freq=on(torch.zeros(32)), axis=ints(32), q_out=rows(3, 4), k_out=rows())),
        "write": (lm.lmoe_kv_write_fp8, dict(cache=cache, k_new=rows(), v_new=rows(), src=ints(3), slots=ints(3), ws=ws)),
        "read": (lm.lmoe_kv_read_fp8, dict(cache=cache, token_offsets=ints(2), first=ints(1), block_table=ints(1, 4),
                                           k_out=rows(), v_out=rows(), ws=ws)),
        "decode": (lm.lmoe_decode_attention_fp8, dict(
            dims=lm.decode_dims_of(3, 4, 4, 0.125), cache=cache, q=rows(3, 4), lens=ints(3), block_table=ints(3, 4),
            out=rows(3, 4), lse=on(torch.zeros(3, 4)), ws=ws)),
    }


@pytest.mark.parametrize("name", ["rope", "write", "read", "decode"])
def test_each_argument(lib, name):
    call, args = calls()[name]
    with pytest.raises(Called):
        call(**args)
    for what, x in args.items():
        if what == "cache":
            other = lm.kv_cache_fp8_of(*pages(1))
        elif what == "dims":
            continue
        else:
            other = on(x.clone(), 1)
        with pytest.raises(ValueError, match="current device"):
            call(**(args | {what: other}))
    if "ws" in args and name != "decode":
        with pytest.raises(Called):
            call(**(args | {"ws": None}))


def test_a_cache_is_on_one_device(lib):
    for i in range(4):
        p = pages()
        p[i].at = 1
        with pytest.raises(ValueError, match="cuda:1"):
            lm.kv_cache_fp8_of(*p)
