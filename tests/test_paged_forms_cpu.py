"""Host replay of the chunk attention's choice of kernel and plan, over batches on both sides of every border between them: a
list is only planned for the kernel that takes one, and what the chosen kernel walks covers every unit once."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from flash_attention_forward_gb300 import build as libbuild

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def replay(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("paged_forms") / "paged_forms.so")
    subprocess.run([libbuild.nvcc(), *libbuild.ARCH, *libbuild.NVCC_FLAGS, "-I" + libbuild.CSRC, "-shared", "-o", out,
                    os.path.join(HERE, "paged_forms.cu")], check=True)
    fn = ctypes.CDLL(out).paged_form_replay

    def run(new, lens, Hq, Hkv, packed=True, quant=False, D=192, sms=152, causal=True, cut=True, max_new=None):
        p = ctypes.POINTER(ctypes.c_int)
        cu_q, cu_k = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (new, lens))
        kv = np.asarray(lens, dtype=np.int32)
        form, msg = (ctypes.c_int * 3)(), ctypes.create_string_buffer(200)
        total_k = max(1, int(cu_k[-1]))
        rc = fn(len(new), Hq, Hkv, cu_q.ctypes.data_as(p), cu_k.ctypes.data_as(p) if packed else None,
                None if packed else kv.ctypes.data_as(p), max_new or int(max(new)), int(quant), D,
                ctypes.c_longlong(total_k * 256 * 2 if packed else 0), total_k if packed else 1 << 20, int(causal), sms, int(cut),
                form, msg)
        assert rc == 0, (msg.value.decode(), len(new), max(new), Hq, Hkv, packed)
        return tuple(bool(x) for x in form)

    return run


@pytest.mark.parametrize("B", [1, 256, 257, 300, 1200])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (3, 3), (16, 16), (16, 4), (64, 8), (128, 128)])
def test_one_tile_sequences_never_get_a_list(replay, B, Hq, Hkv):
    rng = np.random.default_rng(B + Hq)
    tile = 128 // (Hq // Hkv)
    for most in (1, tile):
        new = rng.integers(0, most + 1, B)
        new[0] = most
        lens = new + rng.integers(0, 700, B)
        assert replay(new, lens, Hq, Hkv) == (True, B <= 256, False)


def test_more_tiles_get_a_list_where_keys_are_packed_and_units_many(replay):
    new = [129] + [1, 3] * 600
    assert replay(new, [200] * 1201, 2, 2) == (False, False, True)
    assert replay(new, [200] * 1201, 2, 2, packed=False) == (False, False, False)
    assert replay([300, 1, 0, 129], [300, 7, 5, 900], 8, 8) == (False, False, False)
    # a tile's tokens at most, but announced as more
    assert replay([1] * 300, [37] * 300, 16, 16, max_new=129) == (False, False, True)


@pytest.mark.parametrize("packed,quant,D", [(True, False, 192), (False, False, 128), (False, True, 128), (False, True, 192)])
def test_random_batches(replay, packed, quant, D):
    rng = np.random.default_rng(D + quant)
    seen = set()
    for _ in range(300):
        Hkv, group = int(rng.choice([1, 2, 5, 16])), int(rng.choice([1, 4, 7]))
        tile = 128 // group
        B = int(np.exp(rng.uniform(0, np.log(700))))
        new = rng.integers(0, int(rng.choice([2, tile + 1, 3 * tile])), B) * (rng.random(B) < 0.8)
        if new.sum() == 0:
            new[0] = 1
        lens = rng.integers(0, int(rng.choice([50, 3000])), B)
        seen.add(replay(new, lens, Hkv * group, Hkv, packed, quant, D, int(rng.choice([76, 148, 152])), bool(rng.random() < 0.7),
                        bool(rng.random() < 0.8)))
    assert len(seen) == (1 if quant and D == 192 else 4 if packed else 3)
