"""CPU-side checks of the quantised paged cache: argument codes of the C ABI, workspace sizes, the
binding's refusals, and the fp64 oracle's quantisation against torch's own cast."""
import ctypes

import numpy as np
import pytest
import torch

import flash_attention_forward_gb300 as fa
import oracle
from flash_attention_forward_gb300 import build as libbuild

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x10002)
OFF8 = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return fa.library()


def _write(lib, **over):
    a = dict(k=FAKE, v=FAKE, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, pt=FAKE, kv=FAKE, cu=FAKE, B=2, Hkv=2, total=10,
             page=16, maxp=4, np=8, D=128, Dv=128, strides=None, dt=fa.SDPA_BF16, stream=None)
    a.update(over)
    return lib.sdpa_cache_write_fp8(*a.values())


def _read(lib, **over):
    a = dict(kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, pt=FAKE, cu=FAKE, k=FAKE, v=FAKE, B=2, Hkv=2, total=10,
             page=16, maxp=4, np=8, D=128, Dv=128, strides=None, dt=fa.SDPA_BF16, stream=None)
    a.update(over)
    return lib.sdpa_cache_read_fp8(*a.values())


def _decode(lib, **over):
    a = dict(q=FAKE, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, pt=FAKE, kv=FAKE, o=FAKE, lse=None, B=2, Hq=8, Hkv=2,
             page=16, maxp=4, np=8, D=128, Dv=128, strides=None, scale=0.1, ws=FAKE, wsb=1 << 24,
             dt=fa.SDPA_BF16, stream=None)
    a.update(over)
    return lib.sdpa_decode_paged_fp8(*a.values())


@pytest.mark.parametrize("call", [_write, _read, _decode])
def test_page_and_pointer_codes(lib, call):
    for name in ("kp", "vp", "ks", "vs", "pt"):
        assert call(lib, **{name: None}) == fa.SDPA_ERR_INVALID, name
    assert call(lib, page=24) == fa.SDPA_ERR_INVALID        # not a power of two
    assert call(lib, page=0) == fa.SDPA_ERR_INVALID
    assert call(lib, page=8) == fa.SDPA_ERR_UNSUPPORTED
    assert call(lib, maxp=0) == fa.SDPA_ERR_INVALID
    assert call(lib, np=0) == fa.SDPA_ERR_INVALID
    assert call(lib, maxp=1 << 27, page=16) == fa.SDPA_ERR_UNSUPPORTED  # more than 2^30 rows a sequence
    assert call(lib, B=0) == fa.SDPA_ERR_INVALID
    assert call(lib, Hkv=0) == fa.SDPA_ERR_INVALID
    assert call(lib, pt=ODD) == fa.SDPA_ERR_INVALID
    for name in ("kp", "vp", "ks", "vs"):
        assert call(lib, **{name: OFF8}) == fa.SDPA_ERR_UNSUPPORTED, name
    assert call(lib, D=96) == fa.SDPA_ERR_UNSUPPORTED
    assert call(lib, D=128, Dv=64) == fa.SDPA_ERR_UNSUPPORTED
    assert call(lib, dt=fa.SDPA_E4M3) == fa.SDPA_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", [_write, _read])
def test_cache_codes(lib, call):
    assert call(lib, k=None) == fa.SDPA_ERR_INVALID
    assert call(lib, cu=None) == fa.SDPA_ERR_INVALID
    assert call(lib, cu=ODD) == fa.SDPA_ERR_INVALID
    assert call(lib, total=0) == fa.SDPA_ERR_INVALID
    assert call(lib, k=OFF8) == fa.SDPA_ERR_UNSUPPORTED
    assert call(lib, total=1 << 30, Hkv=2) == fa.SDPA_ERR_UNSUPPORTED
    good = [256, 128, 256, 128, 4096, 256, 128, 4096, 256, 128, 4]

    def strides(i, x):
        s = list(good)
        s[i] = x
        return (ctypes.c_int64 * 11)(*s)

    assert call(lib, strides=strides(0, 260)) == fa.SDPA_ERR_UNSUPPORTED   # 16-bit rows: multiples of 8
    assert call(lib, strides=strides(5, 264)) == fa.SDPA_ERR_UNSUPPORTED   # codes: multiples of 16
    assert call(lib, strides=strides(9, -128)) == fa.SDPA_ERR_UNSUPPORTED
    assert call(lib, strides=strides(10, 3)) == fa.SDPA_ERR_INVALID        # page-table rows shorter than max_pages


def test_decode_codes(lib):
    assert _write(lib, kv=None) == fa.SDPA_ERR_INVALID
    assert _decode(lib, q=None) == fa.SDPA_ERR_INVALID
    assert _decode(lib, kv=None) == fa.SDPA_ERR_INVALID
    assert _decode(lib, Hq=9) == fa.SDPA_ERR_INVALID
    assert _decode(lib, Hq=34) == fa.SDPA_ERR_UNSUPPORTED  # groups of at most 16
    assert _decode(lib, D=64, Dv=64) == fa.SDPA_ERR_UNSUPPORTED
    assert _decode(lib, scale=float("nan")) == fa.SDPA_ERR_INVALID
    assert _decode(lib, ws=None) == fa.SDPA_ERR_INVALID
    assert _decode(lib, wsb=16) == fa.SDPA_ERR_INVALID
    assert _decode(lib, lse=ODD) == fa.SDPA_ERR_INVALID
    s = (ctypes.c_int64 * 11)(1024, 128, 4096, 264, 128, 4096, 256, 128, 1024, 128, 4)
    assert _decode(lib, strides=s) == fa.SDPA_ERR_UNSUPPORTED


def test_decode_workspace(lib):
    # [B, Hq, splits, Dv + 2] fp32; splits of 2048 keys where they fill the card, shorter ones where not
    assert fa.sdpa_decode_paged_fp8_workspace_size(64, 32, 8, 16384, 128) == 64 * 32 * 8 * 130 * 4
    assert fa.sdpa_decode_paged_fp8_workspace_size(1, 8, 1, 16384, 128) == 8 * 64 * 130 * 4
    assert fa.sdpa_decode_paged_fp8_workspace_size(1, 8, 1, 10, 128) == 8 * 1 * 130 * 4
    for bad in ((0, 8, 1, 10, 128), (1, 8, 0, 10, 128), (1, 8, 1, 0, 128)):
        assert fa.sdpa_decode_paged_fp8_workspace_size(*bad) == 0


def test_binding_refuses_what_it_can_see():
    codes = torch.zeros((4, 16, 2, 128)).to(torch.float8_e4m3fn)
    scales = torch.ones((4, 2, 16))
    table, kv, cu = torch.zeros((2, 2), dtype=torch.int32), torch.ones(2, dtype=torch.int32), torch.arange(3, dtype=torch.int32)
    rows = torch.zeros((2, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.sdpa_cache_write_fp8(rows, rows, codes, codes, scales, scales, table, kv, cu)
    with pytest.raises(ValueError, match="float8"):
        fa.sdpa_cache_read_fp8(codes.float(), codes.float(), scales, scales, table, cu, 2)
    with pytest.raises(ValueError, match="k_scale"):
        fa.sdpa_cache_read_fp8(codes, codes, scales[:, :1], scales, table, cu, 2)
    with pytest.raises(ValueError, match="fp16 or bf16"):
        fa.sdpa_cache_write_fp8(rows.float(), rows.float(), codes, codes, scales, scales, table, kv, cu)


def test_oracle_quantisation_agrees_with_the_cast():
    g = torch.Generator().manual_seed(4)
    x = torch.randn((400, 128), generator=g) * torch.exp(4 * torch.randn((400, 1), generator=g))
    x[0] = 0.0
    x[1] = 0.0
    x[1, 3] = 448.0          # exactly the largest code: scale 1
    x[2] = 0.0
    x[2, 3] = 448.0001       # just above: scale 2
    codes, scales = oracle.quantise_e4m3_rows(x)
    assert torch.equal(codes.float(), (x / scales[:, None]).to(torch.float8_e4m3fn).float())
    assert scales[0] == 2.0 ** -80 and scales[1] == 1.0 and scales[2] == 2.0
    amax = x.abs().amax(-1)
    assert (amax <= 448 * scales).all() and (amax[1:] > 224 * scales[1:]).all()
    err = (codes.double() * scales[:, None].double() - x.double()).abs()
    assert (err <= torch.maximum(2.0 ** -4 * x.double().abs(), 2.0 ** -10 * scales[:, None].double())).all()


def test_oracle_paged_chunk_is_plain_attention():
    # one sequence, one head: against softmax written out, queries at the end of the cache
    g = torch.Generator().manual_seed(5)
    k = torch.randn((1, 64, 1, 8), generator=g, dtype=torch.float64)
    v = torch.randn((1, 64, 1, 8), generator=g, dtype=torch.float64)
    q = torch.randn((5, 1, 8), generator=g, dtype=torch.float64)
    kp, vp = k.view(4, 16, 1, 8)[[2, 0, 3, 1]], v.view(4, 16, 1, 8)[[2, 0, 3, 1]]
    table = torch.tensor([[1, 3, 0, 2]], dtype=torch.int32)
    o, lse = oracle.sdpa_fwd_paged(q, kp, vp, table, [50], [0, 5], scale=0.3, causal=True)
    s = 0.3 * q[:, 0] @ k[0, :50, 0].T
    s = s + torch.full_like(s, float("-inf")).triu(46)
    assert np.allclose(o[:, 0], (torch.softmax(s, -1) @ v[0, :50, 0]).numpy(), atol=1e-12)
    assert np.allclose(lse[0], torch.logsumexp(s, -1).numpy(), atol=1e-12)


def _fwd(lib, quant, **over):
    a = dict(q=FAKE, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, pt=FAKE, kv=FAKE, cu=FAKE, o=FAKE, lse=None, B=2, Hq=8, Hkv=2,
             total=20, maxq=12, page=16, maxp=4, np=8, D=128, Dv=128, strides=None, scale=0.1, causal=1, ws=FAKE,
             wsb=1 << 26, dt=fa.SDPA_BF16, stream=None)
    a.update(over)
    if not quant:
        del a["ks"], a["vs"]
    return (lib.sdpa_fwd_paged_fp8 if quant else lib.sdpa_fwd_paged)(*a.values())


@pytest.mark.parametrize("quant", [False, True])
def test_chunk_codes(lib, quant):
    for name in ("q", "kp", "vp", "pt", "kv", "cu", "o", "ws") + (("ks", "vs") if quant else ()):
        assert _fwd(lib, quant, **{name: None}) == fa.SDPA_ERR_INVALID, name
    for name in ("q", "kp", "vp", "o") + (("ks", "vs") if quant else ()):
        assert _fwd(lib, quant, **{name: OFF8}) == fa.SDPA_ERR_UNSUPPORTED, name
    for name in ("pt", "kv", "cu", "lse"):
        assert _fwd(lib, quant, **{name: ODD}) == fa.SDPA_ERR_INVALID, name
    for name in ("B", "Hq", "Hkv", "total", "maxq", "np", "maxp", "D"):
        assert _fwd(lib, quant, **{name: 0}) == fa.SDPA_ERR_INVALID, name
    assert _fwd(lib, quant, maxq=21) == fa.SDPA_ERR_INVALID       # longer than all the packed rows
    assert _fwd(lib, quant, Hkv=3) == fa.SDPA_ERR_INVALID
    assert _fwd(lib, quant, Hq=258) == fa.SDPA_ERR_UNSUPPORTED    # 129 heads per KV head
    assert _fwd(lib, quant, scale=0.0) == fa.SDPA_ERR_INVALID
    assert _fwd(lib, quant, page=48) == fa.SDPA_ERR_INVALID
    assert _fwd(lib, quant, page=8) == fa.SDPA_ERR_UNSUPPORTED
    assert _fwd(lib, quant, D=96, Dv=96) == fa.SDPA_ERR_UNSUPPORTED
    assert _fwd(lib, quant, D=64) == fa.SDPA_ERR_UNSUPPORTED
    assert _fwd(lib, quant, dt=fa.SDPA_E4M3) == fa.SDPA_ERR_UNSUPPORTED
    assert _fwd(lib, quant, wsb=32) == fa.SDPA_ERR_INVALID        # below the plan
    assert _fwd(lib, quant, ws=OFF8) == fa.SDPA_ERR_INVALID
    good = [1024, 128, 4096, 256, 128, 4096, 256, 128, 1024, 128, 4]

    def strides(i, x):
        s = list(good)
        s[i] = x
        return (ctypes.c_int64 * 11)(*s)

    assert _fwd(lib, quant, strides=strides(0, 1028)) == fa.SDPA_ERR_UNSUPPORTED
    assert _fwd(lib, quant, strides=strides(9, 130)) == fa.SDPA_ERR_UNSUPPORTED
    assert _fwd(lib, quant, strides=strides(10, 3)) == fa.SDPA_ERR_INVALID
    if quant:
        assert _fwd(lib, quant, strides=strides(3, 264)) == fa.SDPA_ERR_UNSUPPORTED


def test_chunk_workspace(lib):
    size = fa.sdpa_fwd_paged_workspace_size

    def plan(B, tiles):  # header, cuts and groups of 160 CTAs, tiles, sequences
        return (16 + 161 * 16 + 160 * 32 + tiles * 16 + 8 + (B + 1) * 4 + 15) // 16 * 16

    # fewer than six blocks of keys: nothing to cut
    assert size(3, 8, 2, 30, 12, 640, 128) == plan(3, 3)
    # 5 tokens x 4 heads = 20 rows a slot, two slots for each of 160 CTAs
    assert size(2, 8, 2, 10, 5, 1 << 20, 128) == plan(2, 2) + 320 * 20 * 130 * 4
    # long chunks take slots of both tiles' 256 rows; tiles of 64 tokens
    assert size(4, 32, 8, 8192, 2048, 16384, 128) == plan(4, 128) + 320 * 256 * 130 * 4
    for bad in ((0, 8, 2, 10, 5, 64, 128), (2, 8, 3, 10, 5, 64, 128), (2, 8, 2, 10, 11, 64, 128), (2, 8, 2, 10, 5, 0, 128)):
        assert size(*bad) == 0
