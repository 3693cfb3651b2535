"""Host-side checks of the adapter call (no kernel is launched) and its oracle."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available to build the library")
    from gspo_logprob_gb300 import build
    build()
    from gspo_logprob_gb300 import _abi
    return _abi.load()


def test_struct_layout(lib, tmp_path):
    gcc = shutil.which("gcc") or shutil.which("cc")
    if gcc is None:
        pytest.skip("no C compiler")
    from gspo_logprob_gb300._abi import GhAdapter
    names = [f[0] for f in GhAdapter._fields_]
    prog = tmp_path / "layout.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "grpo_head.h"\nint main(void){printf("%zu",'
                    "sizeof(gh_adapter));" + "".join(f'printf(" %zu", offsetof(gh_adapter, {n}));' for n in names) +
                    "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run([gcc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(GhAdapter)] + [getattr(GhAdapter, n).offset for n in names]


def _p(**kw):
    from gspo_logprob_gb300._abi import GhAdapter
    base = dict(N=64, D=256, V=5000, dtype=0, out_dtype=0, rank=16, num_adapters=4, H=0x100, W=0x100, A=0x100, B=0x100,
                scale=0x100, adapter_id=0x100, logits=0x100, ld=5000)
    return GhAdapter(**{**base, **kw})


def _call(lib, status=0x100, ws=0x100, ws_bytes=1 << 30, **kw):
    code = lib.grpo_adapter_logits(ctypes.byref(_p(**kw)), status, ws, ws_bytes, None)
    return code, lib.gh_last_error()


def test_workspace_size(lib):
    al = lambda x: (x + 255) // 256 * 256  # noqa: E731
    # one 128-row tile, 4 adapters of one 16-wide chunk, two terms of 32 bytes; the list
    assert lib.grpo_adapter_logits_workspace_size(ctypes.byref(_p())) == al(4 * 2 * 128 * 32) + al(5 * 4)
    # two 256-row tiles, rank 24 takes two chunks
    assert lib.grpo_adapter_logits_workspace_size(ctypes.byref(_p(N=300, rank=24))) == \
        al(2 * 8 * 2 * 256 * 32) + al(2 * 5 * 4)
    # fp32 logits: three terms
    assert lib.grpo_adapter_logits_workspace_size(ctypes.byref(_p(out_dtype=1))) == al(4 * 3 * 128 * 32) + al(5 * 4)
    assert lib.grpo_adapter_logits_workspace_size(ctypes.byref(_p(dtype=1, out_dtype=1, rank=3))) == al(64 * 3 * 4)
    assert lib.grpo_adapter_logits_workspace_size(ctypes.byref(_p(rank=0))) == 0


@pytest.mark.parametrize("kw,msg", [
    (dict(N=-1), b"N="), (dict(N=(1 << 24) + 1), b"N="), (dict(D=0), b"D="), (dict(V=0), b"V="),
    (dict(dtype=3), b"dtype"), (dict(out_dtype=3), b"out_dtype"), (dict(dtype=1, out_dtype=0), b"fp32 heads"),
    (dict(rank=0), b"rank"), (dict(rank=257), b"rank"), (dict(rank=12), b"rank % 8"), (dict(D=100), b"D % 8"),
    (dict(num_adapters=0), b"num_adapters"), (dict(num_adapters=70000), b"num_adapters"),
    (dict(N=1 << 24, num_adapters=1000, rank=256), b"split the rows"),
    (dict(N=1 << 23, dtype=1, out_dtype=1), b"split the rows"),
    (dict(N=1 << 24, V=1 << 28), b"split the rows"),
    (dict(ld=4999), b"stride"), (dict(H=0x108), b"aligned"), (dict(B=0x108), b"aligned"), (dict(W=None), b"NULL"),
    (dict(logits=None), b"NULL"), (dict(logits=0x101), b"element-aligned"), (dict(status=None), b"status"),
    (dict(ws=0x108), b"ws must be"),
])
def test_refusals(lib, kw, msg):
    code, err = _call(lib, **kw)
    assert code == 1 and msg in err, err


def test_workspace_refusal(lib):
    assert _call(lib, ws_bytes=16)[0] == 3 and _call(lib, ws=None)[0] == 3


def test_oracle_reduces_to_a_merged_head():
    from oracle.adapter_oracle import adapter_logits
    rng = np.random.default_rng(0)
    H, W = rng.standard_normal((6, 5)), rng.standard_normal((7, 5))
    A, B = rng.standard_normal((2, 3, 5)), rng.standard_normal((2, 7, 3))
    ids = np.array([0, 1, -1, 1, 5, -3])
    z, _, bad = adapter_logits(H, W, A, B, [0.5, -2.0], ids)
    merged = [W + 0.5 * B[0] @ A[0], W - 2.0 * B[1] @ A[1], W]
    for i, a in enumerate([0, 1, 2, 1, 2, 2]):
        assert np.allclose(z[i], merged[a] @ H[i], atol=1e-12)
    assert np.array_equal(bad, [0, 0, 0, 0, 1, 1])
