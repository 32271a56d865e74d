"""Host replay of the chunk attention's work plan: the kernels' own functions, compiled for the host, over batches whose
equal stretches cut units anywhere.  The pieces must cover every unit once, and the merge must read the slots written."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from flash_attention_forward_gb300 import build as libbuild

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def replay(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("paged_line") / "paged_line.so")
    subprocess.run([libbuild.nvcc(), *libbuild.ARCH, *libbuild.NVCC_FLAGS, "-I" + libbuild.CSRC, "-shared", "-o", out,
                    os.path.join(HERE, "paged_line.cu")], check=True)
    fn = ctypes.CDLL(out).paged_line_replay

    def run(new, kv, Hq, Hkv, sms=152, one=True, causal=True, max_kv=1 << 20, cut=True):
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        kv = np.asarray(kv, dtype=np.int32)
        msg = ctypes.create_string_buffer(200)
        p = ctypes.POINTER(ctypes.c_int)
        rc = fn(len(new), Hq, Hkv, cu.ctypes.data_as(p), kv.ctypes.data_as(p), max_kv, int(causal), sms, int(one), int(cut), msg)
        assert rc == 0, (msg.value.decode(), list(new), kv.tolist(), Hq, Hkv, sms)

    return run


@pytest.mark.parametrize("sms", [148, 152, 160])
@pytest.mark.parametrize("new,kv,Hq,Hkv", [([4, 0, 2], [8600, 6600, 1200], 8, 2), ([1, 0, 1], [550, 5, 3000], 1, 1),
                                           ([1, 0, 0, 1, 0], [550, 5, 900, 8000, 70], 4, 1)])
def test_a_cut_next_to_a_sequence_without_tokens(replay, sms, new, kv, Hq, Hkv):
    replay(new, kv, Hq, Hkv, sms)


@pytest.mark.parametrize("one", [True, False])
@pytest.mark.parametrize("idle", [0.0, 0.2, 0.6])
def test_random_batches(replay, one, idle):
    g = np.random.default_rng(int(idle * 10) + one)
    for _ in range(2000):
        B, Hkv = int(g.integers(1, 65)), int(g.choice([1, 2, 4, 8]))
        group = int(g.choice([1, 4, 7, 8]))
        new = g.integers(1, 9 if one else 700, B) * (g.random(B) >= idle)
        kv = np.exp(g.uniform(0, np.log(16384), B)).astype(int)
        kv[g.random(B) < 0.05] = 0
        replay(new, kv, Hkv * group, Hkv, int(g.integers(1, 161)), one, bool(g.integers(2)), cut=bool(g.random() < 0.9))


@pytest.mark.parametrize("one", [True, False])
def test_a_sequence_whose_units_pass_32_bits(replay, one):
    # 300 KV heads of 2^23 key blocks each: the line of one sequence is longer than 2^31
    for kv in ([1 << 30], [1 << 30, 700, 1 << 30]):
        replay([1] * len(kv), kv, 300, 300, one=one, max_kv=1 << 30)
