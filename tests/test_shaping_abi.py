"""Host-side checks of the shaping calls (no kernel is launched): struct layout,
workspace sizes, refusals."""
import ctypes
import os
import shutil
import subprocess

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
    from gspo_logprob_gb300._abi import GhShaping
    names = [f[0] for f in GhShaping._fields_]
    prog = tmp_path / "layout.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "grpo_head.h"\nint main(void){printf("%zu",'
                    "sizeof(gh_shaping));" + "".join(f'printf(" %zu", offsetof(gh_shaping, {n}));' for n in names) +
                    "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run([gcc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(GhShaping)] + [getattr(GhShaping, n).offset for n in names]


def _s(**kw):
    from gspo_logprob_gb300._abi import GhShaping
    return GhShaping(**{**dict(rows=10, V=3000), **kw})


def test_workspace_size(lib):
    # a (max, sum) pair per row and 512 columns, and a target logit per row
    al = lambda x: (x + 255) // 256 * 256  # noqa: E731
    assert lib.grpo_shaped_logp_workspace_size(ctypes.byref(_s())) == al(10 * 6 * 8) + al(10 * 4)
    assert lib.grpo_shaped_logp_workspace_size(ctypes.byref(_s(V=0))) == 0


@pytest.mark.parametrize("kw,msg", [
    (dict(rows=-1), b"rows="),
    (dict(V=0), b"V="),
    (dict(V=(1 << 28) + 1), b"V="),
    (dict(rows=1 << 30, V=3000), b"split the rows"),
    (dict(reserved=1), b"reserved"),
    (dict(num_tokens=-1), b"negative"),
    (dict(hist_len=0x100), b"hist_begin"),
    (dict(hist_len=0x100, hist_begin=0x100, num_tokens=4), b"tokens"),
    (dict(bias_set=0x100), b"bias_offsets"),
    (dict(allow_row=0x100, num_allow=2), b"allow_bits"),
])
def test_shaping_refusals(lib, kw, msg):
    s = ctypes.byref(_s(**kw))
    assert lib.grpo_shape_logits(s, 0x100, 0, 3000, 0x100, 0, 3000, 0x100, None) == 1
    assert msg in lib.gh_last_error()
    assert lib.grpo_shaped_logp(s, 0x100, 0, 3000, 0x100, 0x100, 0x100, 0x100, 0x100, 0x100, 1 << 30, None) == 1
    assert lib.grpo_shaped_logp_backward(s, 0x100, 0, 3000, 0x100, 0x100, 0x100, 0x100, None, 0x100, 3000, 0x100,
                                         None) == 1


def test_logits_refusals(lib):
    s = ctypes.byref(_s())

    def shape(p=0x1000, dt=0, ld=3000, out=0x100000, odt=0, old=3000, st=0x100):
        return lib.grpo_shape_logits(s, p, dt, ld, out, odt, old, st, None), lib.gh_last_error()

    assert shape(p=None)[0] == 1 and shape(out=None)[0] == 1
    for bad, msg in ((dict(dt=5), b"dtype"), (dict(odt=9), b"dtype"), (dict(ld=2999), b"stride"),
                     (dict(old=2999), b"stride"), (dict(p=0x1001), b"element-aligned"), (dict(st=None), b"status"),
                     (dict(dt=1, odt=1, out=0x100002), b"element-aligned"), (dict(out=0x1010), b"overlaps"),
                     (dict(out=0x1000, old=3008), b"overlaps"), (dict(out=0x1000, odt=1), b"overlaps")):
        code, err = shape(**bad)
        assert code == 1 and msg in err, (bad, err)
    # logp: missing outputs, workspace too small or misaligned
    call = lambda *a: lib.grpo_shaped_logp(s, 0x1000, 0, 3000, *a, None)  # noqa: E731
    assert call(None, 0x100, 0x100, 0x100, 0x100, 0x100, 1 << 20) == 1
    assert call(0x100, 0x100, 0x100, 0x100, 0x100, 0x100, 16) == 3
    assert call(0x100, 0x100, 0x100, 0x100, 0x100, 0x108, 1 << 20) == 1 and b"aligned" in lib.gh_last_error()
    assert lib.grpo_shaped_logp_backward(s, 0x1000, 0, 3000, 0x100, 0x100, None, 0x100, None, 0x100000, 3000, 0x100,
                                         None) == 1
    assert lib.grpo_shaped_logp_backward(s, 0x1000, 0, 3000, 0x100, 0x100, 0x100, 0x100, None, 0x1002, 3000, 0x100,
                                         None) == 1 and b"overlaps" in lib.gh_last_error()


def test_shaping_object_refusals():
    import gspo_logprob_gb300 as g
    with pytest.raises(AttributeError):
        g.no_such_entry
    with pytest.raises(TypeError, match="torch.Tensor"):
        g.make_shaping(2, 10, temperature=[1.0, 1.0])
