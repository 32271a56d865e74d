"""Refusals of the latent cache's calls, rotary positions and page allocation: the library's status codes for bad
arguments, before any CUDA call, and the binding's errors."""
import ctypes

import pytest
import torch

import flash_attention_forward_gb300 as fa
from flash_attention_forward_gb300 import build as libbuild

FAKE, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10002)  # never dereferenced: every call below fails validation
F, SZ, I64 = ctypes.c_float, ctypes.c_size_t, ctypes.c_int64
INVALID, UNSUPPORTED = fa.SDPA_ERR_INVALID, fa.SDPA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return fa.library()


def caller(fn, **defaults):
    def call(**over):
        assert set(over) <= set(defaults), over
        return fn(*{**defaults, **over}.values())
    return call


def strides(*x):
    return (I64 * len(x))(*x)


def test_resize_codes(lib):
    call = caller(lib.sdpa_cache_resize, table=FAKE, kv=FAKE, change=FAKE, free=FAKE, n_free=FAKE, kv_out=FAKE, n_out=FAKE, cu=FAKE,
                  pos=FAKE, slots=FAKE, B=2000, total=5000, page=64, max_pages=64, n_pages=100, stride=64, ws=FAKE, wsb=1 << 20,
                  stream=None)
    for name in ("table", "kv", "change", "free", "n_free", "kv_out", "n_out", "cu", "pos", "slots"):
        assert call(**{name: None}) == INVALID
        assert call(**{name: ODD}) == INVALID
    assert call(slots=ctypes.c_void_p(0x10004)) == INVALID
    for over in (dict(B=0), dict(total=0), dict(page=0), dict(page=48), dict(max_pages=0), dict(n_pages=0), dict(stride=63), dict(ws=None),
                 dict(ws=ctypes.c_void_p(0x10008)), dict(wsb=2000 * 16)):
        assert call(**over) == INVALID, over
    assert call(page=8) == UNSUPPORTED
    assert call(page=1 << 20, max_pages=1 << 11, stride=1 << 11) == UNSUPPORTED
    assert fa.sdpa_cache_resize_workspace_size(2000, 5000, 64) == 2001 * 16
    assert fa.sdpa_cache_resize_workspace_size(64, 64, 256) == 0 == fa.sdpa_cache_resize_workspace_size(0, 1, 1)


def test_rope_codes(lib):
    call = caller(lib.sdpa_rope, q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, pos=FAKE, inv=FAKE, total=10, Hq=4, Hk=2, D=128, rot=64, inter=0,
                  factor=F(1.0), strides=None, dt=fa.SDPA_BF16, stream=None)
    for name in ("q", "k", "qo", "ko", "pos", "inv"):
        assert call(**{name: None}) == INVALID
    for over in (dict(total=0), dict(Hq=0), dict(Hk=-1), dict(D=0), dict(rot=0), dict(rot=144), dict(factor=F(float("nan"))),
                 dict(factor=F(float("inf"))), dict(pos=ODD), dict(inv=ODD)):
        assert call(**over) == INVALID, over
    for over in (dict(dt=fa.SDPA_E4M3), dict(rot=40), dict(rot=36, inter=1), dict(D=132), dict(q=ctypes.c_void_p(0x10008)),
                 dict(ko=ctypes.c_void_p(0x10008)), dict(strides=strides(516, 128, 256, 128, 512, 128, 256, 128)),
                 dict(strides=strides(512, 128, 256, 128, 512, -128, 256, 128)), dict(total=1 << 30)):
        assert call(**over) == UNSUPPORTED, over
    # an output whose rows coincide; in place with other strides
    assert call(qo=ctypes.c_void_p(0x20000), strides=strides(512, 128, 256, 128, 512, 0, 256, 128)) == INVALID
    assert call(ko=ctypes.c_void_p(0x20000), strides=strides(512, 128, 256, 128, 512, 128, 0, 128)) == INVALID
    assert call(strides=strides(512, 128, 256, 128, 1024, 128, 256, 128)) == INVALID
    assert call(strides=strides(512, 128, 256, 128, 512, 128, 256, 136)) == INVALID


def test_latent_write_codes(lib):
    call = caller(lib.sdpa_latent_write, c=FAKE, r=FAKE, pool=FAKE, slots=FAKE, pos=FAKE, inv=FAKE, total=10, page=64, n_pages=4,
                  latent=512, rot=64, inter=0, factor=F(1.0), strides=None, dt=fa.SDPA_BF16, stream=None)
    for over in (dict(c=None), dict(r=None), dict(pool=None), dict(slots=None), dict(pos=None), dict(inv=None), dict(total=0), dict(page=0),
                 dict(page=24), dict(n_pages=0), dict(latent=0), dict(slots=ctypes.c_void_p(0x10004)), dict(pos=ODD),
                 dict(factor=F(float("inf")))):
        assert call(**over) == INVALID, over
    for over in (dict(dt=fa.SDPA_I8), dict(latent=256), dict(rot=32), dict(page=8), dict(pool=ctypes.c_void_p(0x10008)),
                 dict(strides=strides(512, 64, 64 * 576, 580))):
        assert call(**over) == UNSUPPORTED, over


def test_absorbed_codes(lib):
    call = caller(lib.sdpa_fwd_latent_paged, q=FAKE, pool=FAKE, table=FAKE, kv=FAKE, cu=FAKE, o=FAKE, lse=None, B=2, Hq=16, total=10,
                  maxq=6, page=64, max_pages=8, n_pages=20, latent=512, rot=64, strides=None, scale=F(0.1), causal=1, ws=FAKE,
                  wsb=SZ(1 << 30), dt=fa.SDPA_BF16, stream=None)
    for name in ("q", "pool", "table", "kv", "cu", "o", "ws"):
        assert call(**{name: None}) == INVALID
    for over in (dict(B=0), dict(Hq=0), dict(total=0), dict(maxq=0), dict(maxq=11), dict(scale=F(0.0)), dict(scale=F(float("nan"))),
                 dict(page=96), dict(max_pages=0), dict(kv=ODD), dict(lse=ODD), dict(wsb=SZ(100)), dict(ws=ctypes.c_void_p(0x10008)),
                 dict(strides=strides(16 * 576, 576, 64 * 576, 576, 16 * 512, 512, 7))):
        assert call(**over) == INVALID, over
    for over in (dict(Hq=129), dict(latent=256), dict(rot=32), dict(dt=fa.SDPA_E4M3), dict(page=8), dict(o=ctypes.c_void_p(0x10008)),
                 dict(strides=strides(16 * 576, 580, 64 * 576, 576, 16 * 512, 512, 8))):
        assert call(**over) == UNSUPPORTED, over
    size = fa.sdpa_fwd_latent_paged_workspace_size
    assert size(2, 16, 10, 6, 512) > size(2, 16, 10, 6, 1) > 0   # room for partials, the plan alone
    for bad in ((0, 16, 10, 6, 512), (2, 129, 10, 6, 512), (2, 16, 10, 11, 512), (2, 16, 10, 0, 512), (2, 16, 10, 6, 0)):
        assert size(*bad) == 0


def test_expanded_codes(lib):
    call = caller(lib.sdpa_fwd_latent, q=FAKE, k=FAKE, r=FAKE, v=FAKE, cq=FAKE, ck=FAKE, o=FAKE, lse=None, B=2, Hq=16, Hkv=16, tq=10,
                  tk=20, maxq=6, nope=128, rot=64, Dv=128, strides=None, scale=F(0.1), causal=1, ws=FAKE, wsb=SZ(1 << 30),
                  dt=fa.SDPA_F16, stream=None)
    for name in ("q", "k", "r", "v", "cq", "ck", "o", "ws"):
        assert call(**{name: None}) == INVALID
    for over in (dict(B=0), dict(Hkv=3), dict(tq=0), dict(tk=0), dict(maxq=11), dict(scale=F(-1.0)), dict(ck=ODD), dict(wsb=SZ(64))):
        assert call(**over) == INVALID, over
    for over in (dict(nope=64), dict(rot=32), dict(Dv=64), dict(dt=fa.SDPA_E4M3), dict(Hq=129, Hkv=1), dict(r=ctypes.c_void_p(0x10008)),
                 dict(strides=strides(16 * 192, 192, 16 * 128, 128, 68, 16 * 128, 128, 16 * 128, 128))):
        assert call(**over) == UNSUPPORTED, over
    assert fa.sdpa_fwd_latent_workspace_size(2, 16, 16, 10, 6, 20) > 0 == fa.sdpa_fwd_latent_workspace_size(2, 16, 3, 10, 6, 20)


def test_binding_refuses_shapes_types_and_host_tensors():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    h = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    f = torch.ones(32)
    ok_resize = (i(2, 4), i(2), i(2), i(9), i(1), 16, 3)
    for at, bad in ((0, i(3, 4)), (0, i(2)), (1, i(2).long()), (2, i(3)), (3, i(3, 3)), (4, i(2))):
        args = list(ok_resize)
        args[at] = bad
        with pytest.raises(ValueError):
            fa.sdpa_cache_resize(*args)
    for kw in (dict(slots=i(3)), dict(positions=i(4)), dict(kv_len_out=i(3)), dict(cu_seqlens=i(2))):
        with pytest.raises(ValueError):
            fa.sdpa_cache_resize(*ok_resize, **kw)
    with pytest.raises(ValueError):
        fa.sdpa_cache_resize(*ok_resize)     # host tensors
    q, k = h(5, 4, 64), h(5, 2, 64)
    for args in ((h(5, 64), k, i(5), f), (q, h(4, 2, 64), i(5), f), (q, h(5, 2, 128), i(5), f), (q, k.half(), i(5), f), (q, k, i(4), f),
                 (q, k, i(5), f.double()), (q.float(), None, i(5), f), (q, k, i(5), f)):
        with pytest.raises(ValueError):
            fa.sdpa_rope(*args)
    with pytest.raises(ValueError):
        fa.sdpa_rope(q, None, i(5), f, k_out=k)
    with pytest.raises(ValueError):
        fa.sdpa_rope(q, k, i(5), f, q_out=h(5, 4, 32))
    pool, slots = h(3, 16, 576), torch.zeros(5, dtype=torch.int64)
    for args in ((h(5, 512), h(5, 64), h(3, 576), slots), (h(5, 512), h(4, 64), pool, slots), (h(5, 256), h(5, 64), pool, slots),
                 (h(5, 512).half(), h(5, 64), pool, slots), (h(5, 512), h(5, 64), pool, slots.int()), (h(5, 512), h(5, 64), pool, slots, i(5)),
                 (h(5, 512), h(5, 64), pool, slots, i(5), torch.ones(16)), (h(5, 512), h(5, 64), pool, slots, i(5), f)):
        with pytest.raises(ValueError):
            fa.sdpa_latent_write(*args)
    q = h(5, 4, 576)
    for args in ((h(5, 4, 64), h(3, 16, 64), i(2, 3), i(2), i(3)), (h(5, 576), pool, i(2, 3), i(2), i(3)), (q.half(), pool, i(2, 3), i(2), i(3)), (h(5, 4, 512), pool, i(2, 3), i(2), i(3)),
                 (q, pool, i(3, 3), i(2), i(3)), (q, pool, i(2, 3), i(2), i(2)), (q, pool, i(2, 3), i(2), i(3))):
        with pytest.raises(ValueError):
            fa.sdpa_fwd_latent_paged(*args, 5, scale=0.1)
    q, kn, r, v = h(5, 4, 192), h(7, 4, 128), h(7, 64), h(7, 4, 128)
    for args in ((h(5, 192), kn, r, v, i(2), i(2)), (q, kn, h(6, 64), v, i(2), i(2)), (q, kn, r, h(7, 2, 128), i(2), i(2)),
                 (q, kn, h(7, 32), v, i(2), i(2)), (q, kn, r, v.half(), i(2), i(2)), (q, kn, r, v, i(2), i(3)), (q, kn, r, v, i(2), i(2))):
        with pytest.raises(ValueError):
            fa.sdpa_fwd_latent(*args, 5)


def test_inputs_and_outputs_whose_rows_coincide(lib):
    """A broadcast view handed to an entry that cannot take it is refused before anything runs."""
    absorbed = caller(lib.sdpa_fwd_latent_paged, q=FAKE, pool=FAKE, table=FAKE, kv=FAKE, cu=FAKE, o=FAKE, lse=None, B=2, Hq=16, total=10,
                      maxq=6, page=64, max_pages=8, n_pages=20, latent=512, rot=64, strides=None, scale=F(0.1), causal=1, ws=FAKE,
                      wsb=SZ(1 << 30), dt=fa.SDPA_BF16, stream=None)
    expanded = caller(lib.sdpa_fwd_latent, q=FAKE, k=FAKE, r=FAKE, v=FAKE, cq=FAKE, ck=FAKE, o=FAKE, lse=None, B=2, Hq=16, Hkv=16, tq=10,
                      tk=20, maxq=6, nope=128, rot=64, Dv=128, strides=None, scale=F(0.1), causal=1, ws=FAKE, wsb=SZ(1 << 30),
                      dt=fa.SDPA_F16, stream=None)
    write = caller(lib.sdpa_latent_write, c=FAKE, r=FAKE, pool=FAKE, slots=FAKE, pos=FAKE, inv=FAKE, total=10, page=64, n_pages=4,
                   latent=512, rot=64, inter=0, factor=F(1.0), strides=None, dt=fa.SDPA_BF16, stream=None)
    for call, full, outputs in ((absorbed, (16 * 576, 576, 64 * 576, 576, 16 * 512, 512, 8), (4, 5)),
                                (expanded, (16 * 192, 192, 16 * 128, 128, 64, 16 * 128, 128, 16 * 128, 128), (7, 8))):
        for at in range(len(full) - (call is absorbed)):
            flat = [0 if i == at else x for i, x in enumerate(full)]
            assert call(strides=strides(*flat)) == (INVALID if at in outputs else UNSUPPORTED), (at, flat)
    for at in (2, 3):
        assert write(strides=strides(*(0 if i == at else x for i, x in enumerate((512, 64, 64 * 576, 576))))) == INVALID
