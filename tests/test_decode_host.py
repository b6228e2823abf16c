"""Refusals of the decode step's operators, which need no GPU: the C entries check their arguments before anything
else."""
import ctypes

import pytest

import fp8_ref
import latent_moe_layer_fp32_gb300 as lm

EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -6
P = 1 << 20  # a 256-byte aligned address that nothing reads
nan, inf = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    lm.build()
    return lm.load()


def cache(**kw):
    a = dict(k=P, v=P + (1 << 24), k_scale=P + (2 << 24), v_scale=P + (3 << 24), n_blocks=8, block_size=16, kv_heads=2,
             head_dim=64, block_stride=2048, head_stride=1024, slot_stride=64, maps=None)
    return lm.LmoeKvCacheFp8(**(a | kw))


def write(lib, c=None, **kw):
    a = dict(k=P, ks=128, v=P, vs=128, rows=4, src=P, slots=P, n=4, ws=None, ws_bytes=0)
    return lib.lmoe_kv_write_fp8(ctypes.byref(c or cache()), *(a | kw).values(), None)


def read(lib, c=None, **kw):
    a = dict(b=2, n=9, mb=4, off=P, first=P, table=P, k=P, ks=128, v=P + 64, vs=128, ws=None, ws_bytes=0)
    return lib.lmoe_kv_read_fp8(ctypes.byref(c or cache()), *(a | kw).values(), None)


def attend(lib, d=None, c=None, **kw):
    a = dict(q=P, qs=256, lens=P, table=P, out=P, lse=P, ws=P, ws_bytes=1 << 40)
    d = d or dims()
    return lib.lmoe_decode_attention_fp8(ctypes.byref(d), ctypes.byref(c or cache()), *(a | kw).values(), None)


def dims(**kw):
    return lm.LmoeDecodeDims(**(dict(n_requests=2, q_heads=4, max_blocks=4, window=0, scale=0.125) | kw))


def rope_dims(**kw):
    a = dict(n_tokens=5, q_heads=4, k_heads=2, head_dim=64, rot_dim=64, n_axes=1, interleaved=0, norm=1, eps=1e-6)
    return lm.LmoeRopeDims(**(a | kw))


def rope(lib, d=None, **kw):
    a = dict(q=P, qs=256, k=P + 4096, ks=128, qg=P, kg=P, pos=P, freq=P, axis=P, qo=P + 8192, qos=256, ko=P + 16384,
             kos=128)
    return lib.lmoe_qk_norm_rope(ctypes.byref(d or rope_dims()), *(a | kw).values(), None)


def test_cache_descriptors(lib):
    maps = lm.LmoeKvMapsFp8()
    for bad in (dict(k=0), dict(v=P + 8), dict(k_scale=0), dict(v_scale=P + 4), dict(n_blocks=0), dict(kv_heads=0),
                dict(kv_heads=257), dict(head_dim=0), dict(block_stride=2040), dict(head_stride=-1024),
                dict(slot_stride=72), dict(slot_stride=0), dict(slot_stride=48), dict(head_stride=0),
                dict(block_stride=0), dict(block_size=0)):
        for call in (write, read, attend):
            assert call(lib, c=cache(**bad)) == EINVAL, bad
        assert lib.lmoe_kv_maps_fp8_init(ctypes.byref(cache(**bad)), ctypes.byref(maps)) == EINVAL
    for bad in (dict(head_dim=96), dict(head_dim=256), dict(block_size=8), dict(block_size=24), dict(block_size=512),
                dict(n_blocks=1 << 27)):
        for call in (write, read, attend):
            assert call(lib, c=cache(**bad)) == EUNSUPPORTED, bad
    assert lib.lmoe_kv_maps_fp8_init(None, ctypes.byref(maps)) == EINVAL
    assert lib.lmoe_kv_maps_fp8_init(ctypes.byref(cache()), None) == EINVAL


def test_write_refuses(lib):
    for bad in (dict(k=0), dict(v=P + 4), dict(ks=120), dict(vs=129), dict(rows=0), dict(slots=0), dict(slots=P + 1),
                dict(src=P + 2), dict(n=0), dict(n=(1 << 20) + 1), dict(src=None, n=5)):
        assert write(lib, **bad) == EINVAL, bad


def test_write_refuses_rows_that_overlap(lib):
    # (an accepted layout ends at the workspace, of which there is nothing, or for want of a device)
    def at(**kw):
        return write(lib, c=cache(**kw), ws=P)

    for block, head, slot in ((2048, 64, 64), (64, 1024, 64), (2048, 1024, 1024), (1024, 1024, 64), (2032, 1024, 64),
                              (2048, 1008, 64), (2**62, 2**62, 64)):
        assert at(block_stride=block, head_stride=head, slot_stride=slot) == EINVAL, (block, head, slot)
    assert at(v=P) == EINVAL and at(v_scale=P + (2 << 24)) == EINVAL
    for kw in (dict(), dict(head_stride=64, slot_stride=128), dict(head_stride=80, slot_stride=160, block_stride=2560),
               dict(block_stride=1 << 40), dict(n_blocks=1, block_stride=0), dict(kv_heads=1, head_stride=0, block_stride=1024)):
        assert at(**kw) != EINVAL, kw


def test_read_refuses(lib):
    for bad in (dict(b=0), dict(b=8193), dict(n=0), dict(n=(1 << 20) + 1), dict(mb=0), dict(mb=(1 << 24) + 1), dict(off=0),
                dict(off=P + 2), dict(first=P + 1), dict(table=0), dict(k=0), dict(k=P + 8), dict(v=P), dict(ks=64),
                dict(vs=132)):
        assert read(lib, **bad) == EINVAL, bad


def test_decode_attention_refuses(lib):
    for bad in (dict(q=0), dict(q=P + 2), dict(qs=255), dict(qs=260), dict(qs=-256), dict(lens=0), dict(lens=P + 2),
                dict(table=0), dict(out=0), dict(out=P + 4), dict(lse=P + 2), dict(ws=0), dict(ws=P + 128)):
        assert attend(lib, **bad) == EINVAL, bad
    for bad in (dict(n_requests=0), dict(n_requests=8193), dict(q_heads=0), dict(q_heads=3), dict(q_heads=258),
                dict(max_blocks=0), dict(max_blocks=(1 << 24) + 1), dict(window=-1), dict(scale=0.0), dict(scale=nan),
                dict(scale=-1.0), dict(scale=inf), dict(scale=2.36e38)):
        assert attend(lib, d=dims(**bad)) == EINVAL, bad
        assert lm.lmoe_decode_attention_fp8_workspace_bytes(dims(**bad), cache()) == 0
    assert lib.lmoe_decode_attention_fp8(None, ctypes.byref(cache()), P, 256, *[P] * 5, 1 << 40, None) == EINVAL


def test_workspace_bytes(lib):
    n = lm.lmoe_decode_attention_fp8_workspace_bytes(dims(), cache())
    assert n > 256
    # only the heads and the width of the cache count, and not the lengths or the number of requests
    assert lm.lmoe_decode_attention_fp8_workspace_bytes(dims(n_requests=8192, max_blocks=1 << 24),
                                                        cache(k=0, v=0, n_blocks=0)) == n
    assert lm.lmoe_decode_attention_fp8_workspace_bytes(dims(), cache(head_dim=80)) == 0


def test_norm_rope_refuses(lib):
    for bad in (dict(q=0), dict(q=P + 8), dict(k=0), dict(qo=0), dict(ko=P + 2), dict(qs=255), dict(qs=252), dict(ks=64),
                dict(qos=128), dict(kos=132), dict(qg=P + 2), dict(kg=P + 4), dict(pos=0), dict(pos=P + 2),
                dict(freq=0), dict(freq=P + 1), dict(axis=P + 2), dict(qo=P, qos=512), dict(qo=P + 4096),
                dict(ko=P), dict(ko=P + 8192)):
        assert rope(lib, **bad) == EINVAL, bad
    for bad in (dict(n_tokens=0), dict(n_tokens=(1 << 20) + 1), dict(q_heads=-1), dict(k_heads=1025), dict(q_heads=1025),
                dict(q_heads=0, k_heads=0), dict(head_dim=0), dict(rot_dim=-8), dict(rot_dim=72), dict(n_axes=0),
                dict(n_axes=5), dict(interleaved=2), dict(norm=-1), dict(eps=-1.0), dict(eps=nan), dict(eps=inf)):
        assert rope(lib, d=rope_dims(**bad)) == EINVAL, bad
    for bad in (dict(head_dim=264), dict(head_dim=68, rot_dim=64), dict(rot_dim=20)):
        assert rope(lib, d=rope_dims(**bad)) == EUNSUPPORTED, bad
    assert lib.lmoe_qk_norm_rope(None, P, 256, P, 128, P, P, P, P, P, P, 256, P, 128, None) == EINVAL


def test_copy_descriptors_live_as_long_as_a_cache_descriptor_uses_them(lib):
    import gc
    import weakref

    first, maps = cache(), lm.LmoeKvMapsFp8()
    first.maps = ctypes.addressof(maps)
    alive = weakref.ref(maps)
    second = lm.LmoeKvCacheFp8(*[getattr(first, n) for n, _ in lm.LmoeKvCacheFp8._fields_])
    del first, maps
    gc.collect()
    assert alive() is not None and second.maps == ctypes.addressof(alive())
    second.maps = None
    gc.collect()
    assert alive() is None


def test_binding_refuses(lib):
    import torch
    t, s = torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.zeros(4, 2, 16, dtype=torch.uint8)
    with pytest.raises(ValueError):
        lm.kv_cache_fp8_of(t, t, s, s)  # not on a GPU
    with pytest.raises(TypeError):
        lm._rows_of(0, 4, t[0].float(), 2, 64, "q")
    with pytest.raises(ValueError):
        lm._rows_of(0, 4, t[0].bfloat16(), 2, 64, "q")


def test_the_reference_quantises_as_the_formats_say():
    """The tests' own reference against the E4M3 and E8M0 values of the formats' tables."""
    import os
    import numpy as np
    here = os.path.join(os.path.dirname(__file__), "golden", "e4m3_ocp_fp8.txt")
    rows = [line.split() for line in open(here) if not line.startswith("#") and line.strip()]
    assert len(rows) >= 14
    for code, value in rows:
        got, want = fp8_ref.E4M3[int(code, 16)], float(value)
        assert got == want or (np.isnan(got) and np.isnan(want)), code
    # 448 and what is above it, rows of zeros of both signs, ties to even
    codes, scale = fp8_ref.quantise(np.array([[448.0, 1.0, -3.25], [450.0, 17.0, 19.0], [0.0, -0.0, 0.0]]))
    assert scale.tolist() == [127, 128, 0]
    assert fp8_ref.values(codes, scale).tolist() == [[448.0, 1.0, -3.25], [448.0, 16.0, 20.0], [0.0, 0.0, 0.0]]
    assert codes[2].tolist() == [0, 128, 0]
