"""Host replay of the latent attention's work plan: the kernels' own functions, compiled for the host.  The pieces must cover
every unit once, and the merge must read the slots written."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from flash_attention_forward_gb300 import build as libbuild

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def replay(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("latent_line") / "latent_line.so")
    subprocess.run([libbuild.nvcc(), *libbuild.ARCH, *libbuild.NVCC_FLAGS, "-I" + libbuild.CSRC, "-shared", "-o", out,
                    os.path.join(HERE, "latent_line.cu")], check=True)
    fn = ctypes.CDLL(out).latent_line_replay

    def run(new, kv, tok_tile, sms=152, inline=True, causal=True, max_kv=1 << 20, cut=True):
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        kv = np.asarray(kv, dtype=np.int32)
        msg = ctypes.create_string_buffer(200)
        p = ctypes.POINTER(ctypes.c_int)
        rc = fn(len(new), tok_tile, cu.ctypes.data_as(p), kv.ctypes.data_as(p), max_kv, int(causal), sms, int(inline), int(cut), msg)
        assert rc == 0, (msg.value.decode(), list(new), kv.tolist(), tok_tile, sms)

    return run


@pytest.mark.parametrize("inline", [True, False])
@pytest.mark.parametrize("sms", [1, 76, 152])
def test_batches(replay, sms, inline):
    rng = np.random.default_rng(sms)
    for _ in range(300):
        B = int(rng.integers(1, 40))
        tok_tile = int(rng.choice([1, 2, 4, 16, 64]))
        new = rng.integers(0, 8 * tok_tile + 1, B) * rng.integers(0, 2, B) if rng.random() < 0.5 else rng.integers(0, 4, B) % (8 * tok_tile + 1)
        kv = new + rng.integers(-3, int(rng.choice([4, 300, 20000])), B)
        if new.sum() == 0:
            new[0] = 1
        replay(new, kv, tok_tile, sms, inline, causal=bool(rng.random() < 0.7), cut=bool(rng.random() < 0.8))


@pytest.mark.parametrize("inline", [True, False])
def test_lines_past_32_bits_and_clamped_lengths(replay, inline):
    replay([1] * 256, [1 << 30] * 256, 1, inline=inline, max_kv=1 << 30)
    replay([8, 0, 3], [-5, 9, 1 << 30], 1, inline=inline, max_kv=1000)
    replay([1], [1], 16, inline=inline)
