"""The parameter structs of the operators around the recurrences have the layout in C that the Python binding declares."""
import ctypes
import os
import shutil
import subprocess

import pytest

from chunkwise_gated_linear_gla_gb300 import binding as bnd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = ("gla_conv_params", "gla_conv_grads", "gla_ssm_params", "gla_ssm_grads", "gla_norm_gate_params", "gla_norm_gate_grads",
           "gla_residual_params", "gla_residual_grads")


def test_plain_c_sees_the_same_offsets(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines = []
    for s in STRUCTS:
        lines.append(f'printf("{s} %zu\\n", sizeof({s}));')
        lines += [f'printf("{s}.{f} %zu\\n", offsetof({s}, {f}));' for f, *_ in getattr(bnd, s)._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "gla.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = str(tmp_path / "layout")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    r = subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), "-I", cuda, str(src), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    got = dict(line.split() for line in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines())
    for s in STRUCTS:
        t = getattr(bnd, s)
        assert int(got[s]) == ctypes.sizeof(t), s
        for f, *_ in t._fields_:
            assert int(got[f"{s}.{f}"]) == getattr(t, f).offset, f"{s}.{f}"
