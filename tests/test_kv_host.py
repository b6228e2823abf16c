"""Refusals of the paged-cache operators, which need no GPU: the C entries check
their arguments before anything else."""
import ctypes

import pytest

import latent_moe_layer_fp32_gb300 as lm

EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -6
P = 1 << 20  # a 256-byte aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    lm.build()
    return lm.load()


def cache(**kw):
    a = dict(k=P, v=P, n_blocks=8, block_size=16, kv_heads=2, head_dim=64, block_stride=2048, head_stride=1024,
             slot_stride=64)
    return lm.LmoeKvCache(**(a | kw))


def dims(**kw):
    a = dict(n_requests=2, n_tokens=9, max_request_tokens=8, q_heads=4, max_blocks=4, mask_words=1, window=0,
             scale=0.125)
    return lm.LmoeAttnDims(**(a | kw))


def attend(lib, d=None, c=None, **kw):
    a = dict(q=P, qs=256, k=P, ks=128, v=P, vs=128, off=P, lens=P, table=P, mask=P, pos=P, out=P, lse=P, ws=P,
             ws_bytes=1 << 40)
    a |= kw
    d, c = d or dims(), c or cache()
    return lib.lmoe_tree_attention(ctypes.byref(d), ctypes.byref(c), *a.values(), None)


def test_tree_attention_refuses(lib):
    for bad in (dict(q=0), dict(q=P + 2), dict(k=0), dict(v=P + 8), dict(out=0), dict(out=P + 4), dict(off=0),
                dict(off=P + 2), dict(lens=0), dict(table=0), dict(mask=P + 4), dict(pos=P + 1), dict(lse=P + 2),
                dict(ws=0), dict(ws=P + 128), dict(qs=255), dict(qs=260), dict(ks=64), dict(ks=132), dict(vs=0),
                dict(vs=-128)):
        assert attend(lib, **bad) == EINVAL, bad
    for bad in (dict(n_requests=0), dict(n_requests=8193), dict(n_tokens=0), dict(n_tokens=(1 << 20) + 1),
                dict(max_request_tokens=0), dict(max_request_tokens=257), dict(max_request_tokens=65),
                dict(q_heads=0), dict(q_heads=3), dict(q_heads=258), dict(max_blocks=0), dict(mask_words=0),
                dict(mask_words=5), dict(window=-1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=-1.0),
                dict(scale=float("inf"))):
        assert attend(lib, d=dims(**bad)) == EINVAL, bad
    assert lib.lmoe_tree_attention(None, ctypes.byref(cache()), *[P] * 2, *[P] * 14, None) == EINVAL


def test_tree_attention_refuses_a_scale_that_has_no_base_2_form(lib):
    # scores are taken to base 2: scale * log2(e) has to be finite
    for scale in (2.36e38, 3e38, 3.4e38):
        assert attend(lib, d=dims(scale=scale), ws_bytes=0) == EINVAL
    for scale in (1e-45, 1e-30, 1.0, 2.35e38):  # (goes on to the workspace, of which there is nothing)
        assert attend(lib, d=dims(scale=scale), ws_bytes=0) != EINVAL


def test_cache_descriptors(lib):
    def write(c, **kw):
        a = dict(k=P, ks=128, v=P, vs=128, rows=4, src=P, slots=P, n=4, ws=None, ws_bytes=0)
        return lib.lmoe_kv_write(ctypes.byref(c), *(a | kw).values(), None)

    for bad in (dict(k=0), dict(v=P + 8), dict(n_blocks=0), dict(kv_heads=0), dict(kv_heads=257), dict(head_dim=0),
                dict(block_stride=2047), dict(head_stride=-1024), dict(slot_stride=60), dict(slot_stride=0),
                dict(head_stride=0), dict(block_stride=0)):
        assert attend(lib, c=cache(**bad)) == EINVAL, bad
        assert write(cache(**bad)) == EINVAL, bad
    for bad in (dict(head_dim=96), dict(head_dim=256), dict(block_size=8), dict(block_size=24),
                dict(block_size=512), dict(n_blocks=1 << 30)):
        assert attend(lib, c=cache(**bad)) == EUNSUPPORTED, bad
        assert write(cache(**bad)) == EUNSUPPORTED, bad
    for bad in (dict(k=0), dict(v=P + 4), dict(ks=120), dict(vs=129), dict(rows=0), dict(slots=0), dict(slots=P + 1),
                dict(src=P + 2), dict(n=0), dict(n=(1 << 20) + 1), dict(src=None, n=5)):
        assert write(cache(), **bad) == EINVAL, bad


def test_write_refuses_rows_that_overlap(lib):
    """cache(): 8 blocks of 2 heads of 16 slots of 64.  A refused call returns before it looks for a device; one
    whose layout is accepted ends at the workspace (no bytes of it), or for want of a device, and launches nothing."""
    def write(**kw):
        return lib.lmoe_kv_write(ctypes.byref(cache(**kw)), P, 128, P, 128, 4, P, P, 4, P, 0, None)

    # (block, head, slot) strides
    for block, head, slot in ((2048, 64, 64), (64, 1024, 64), (2048, 1024, 1024), (1024, 1024, 64), (2040, 1024, 64),
                              (2048, 1016, 64), (2048, 64, 120), (256, 64, 256), (4096, 2048, 136), (1984, 64, 128),
                              (2**62, 2**62, 64)):
        assert write(block_stride=block, head_stride=head, slot_stride=slot) == EINVAL, (block, head, slot)
    # either order, padded, one inside the other; dimensions of one do not count
    for kw in (dict(), dict(head_stride=64, slot_stride=128), dict(head_stride=72, slot_stride=136, block_stride=2176),
               dict(block_stride=1024, head_stride=8192), dict(block_stride=128, head_stride=64, slot_stride=1024),
               dict(block_stride=1 << 40), dict(head_stride=1024 + 8, block_stride=2056),
               dict(n_blocks=1, block_stride=0), dict(kv_heads=1, head_stride=0, block_stride=1024)):
        assert write(**kw) != EINVAL, kw


def test_copy_descriptors_refuse(lib):
    m = lm.LmoeKvMaps()
    assert lib.lmoe_kv_maps_init(ctypes.byref(cache(k=0)), ctypes.byref(m)) == EINVAL
    assert lib.lmoe_kv_maps_init(ctypes.byref(cache(head_dim=96)), ctypes.byref(m)) == EUNSUPPORTED
    assert lib.lmoe_kv_maps_init(ctypes.byref(cache()), None) == EINVAL
    assert lib.lmoe_kv_maps_init(None, ctypes.byref(m)) == EINVAL


def test_copy_descriptors_live_as_long_as_a_cache_descriptor_uses_them(lib):
    import copy
    import gc
    import weakref

    def fields(c):
        return [getattr(c, n) for n, _ in lm.LmoeKvCache._fields_]

    for take in (lambda c: lm.LmoeKvCache(*fields(c)), lambda c: lm.LmoeKvCache(**dict(zip("k v maps".split(),
                 (c.k, c.v, c.maps)))), lambda c: setattr(new := cache(), "maps", c.maps) or new):
        first, maps = cache(), lm.LmoeKvMaps()
        first.maps = ctypes.addressof(maps)
        alive = weakref.ref(maps)
        second = take(first)
        del first, maps
        gc.collect()
        assert alive() is not None and second.maps == ctypes.addressof(alive())
        second.maps = None
        gc.collect()
        assert alive() is None and second.maps is None
    with pytest.raises(ValueError):  # ctypes itself refuses to copy what holds addresses
        copy.copy(cache())


def test_workspace_bytes(lib):
    assert lm.lmoe_tree_attention_workspace_bytes(dims(), cache()) >= 8
    # only the heads and the width of the cache count
    assert lm.lmoe_tree_attention_workspace_bytes(dims(), cache(k=0, v=0, n_blocks=0)) > 0
    assert lm.lmoe_tree_attention_workspace_bytes(dims(q_heads=3), cache()) == 0
    assert lm.lmoe_tree_attention_workspace_bytes(dims(), cache(head_dim=80)) == 0


def test_tree_masks_refuses(lib):
    def call(**kw):
        a = dict(b=2, t=9, w=1, off=P, par=P, lens=P, mask=P, pos=P, ws=None, ws_bytes=0)
        return lib.lmoe_tree_masks(*(a | kw).values(), None)

    for bad in (dict(b=0), dict(b=8193), dict(t=0), dict(t=(1 << 20) + 1), dict(w=0), dict(w=5), dict(off=0),
                dict(par=P + 2), dict(lens=P + 1), dict(mask=0), dict(mask=P + 4), dict(pos=0)):
        assert call(**bad) == EINVAL, bad


def test_kv_plan_refuses(lib):
    def call(**kw):
        a = dict(b=2, bs=16, mb=4, slots_n=8, lens=P, new=P + 64, owned=P + 128, table=P + 192, ring=P + 256,
                 ring_n=64, state=P + 320, lens_out=P + 384, owned_out=P + 448, state_out=P + 512, off=P + 576,
                 slots=P + 640)
        return lib.lmoe_kv_plan(*(a | kw).values(), None)

    for bad in (dict(b=0), dict(b=8193), dict(bs=0), dict(mb=0), dict(mb=(1 << 24) + 1), dict(slots_n=0),
                dict(ring_n=0), dict(lens=0), dict(new=P + 2), dict(owned=0), dict(table=0), dict(ring=0),
                dict(state=0), dict(lens_out=0), dict(owned_out=0), dict(state_out=0), dict(off=0), dict(slots=0),
                dict(lens_out=P), dict(owned_out=P + 128), dict(state_out=P + 320), dict(off=P + 640),
                dict(slots=P + 256), dict(table=P + 256)):
        assert call(**bad) == EINVAL, bad


def test_binding_refuses(lib):
    import torch
    t = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lm.kv_cache_of(t, t)  # not on a GPU
    with pytest.raises(TypeError):
        lm._rows(t[0].float(), 2, 64)
    with pytest.raises(ValueError):
        lm._rows(t[0], 2, 64)
