"""An output that the header lets be an input itself is not told to the compiler as memory of its own: in the kernels'
intermediate code its pointer carries no `noalias`, as a __restrict__ one does.  CPU only (hipcc cross-compiles)."""
import os
import re
import subprocess

import pytest

from mamba_selective_scan_03_amd import build

CSRC = os.path.join(build.HERE, "csrc")

# kernel: the include, the instance, the positions of the arguments that may be one tensor
KERNELS = {
    "residual is out": ("int8_kernels.h", "matmul_i8_tiled_kernel<BF16, 16, 16, 1, 1, 8, 3, Finish::Residual>", [5]),
    "residual is out, large tile": ("int8_kernels.h", "matmul_i8_tiled_kernel<F32, 256, 256, 4, 4, 1, 2, Finish::Residual>", [5]),
    "state is state_out": ("causal_conv_kernels.h", "causal_conv_kernel<BF16, 4, 4, Act::Silu, false>", [1, 6]),
}


def arguments(include, kernel, tmp_path):
    """The argument list of the instance, in LLVM's notation."""
    src = tmp_path / "one.hip"
    src.write_text(f'#include <hip/hip_runtime.h>\n#include "{os.path.join(CSRC, include)}"\nusing namespace jscan;\n'
                   f"const void *kernel() {{ return reinterpret_cast<const void *>(&{kernel}); }}\n")
    out = tmp_path / "one.ll"
    flags = [f for f in build.FLAGS if f != "-O3"]
    res = subprocess.run([build.HIPCC, *flags, "-O1", "--cuda-device-only", "-emit-llvm", "-S", "-o", str(out), str(src)],
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
    lines = [ln for ln in out.read_text().splitlines() if re.match(r"define .*amdgpu_kernel void @_ZN5jscan", ln)]
    assert len(lines) == 1
    args, depth, word = [], 0, ""
    for c in lines[0][lines[0].index("(") + 1:]:
        if c == "," and depth == 0:
            args.append(word)
            word = ""
            continue
        depth += (c == "(") - (c == ")")
        if depth < 0:
            break
        word += c
    return args + [word]


@pytest.mark.parametrize("name", KERNELS)
def test_in_place_arguments_may_alias(name, tmp_path):
    include, kernel, places = KERNELS[name]
    args = arguments(include, kernel, tmp_path)
    assert any("noalias" in a for a in args)   # other arguments of the kernel have it
    for i in places:
        assert "ptr" in args[i] and "noalias" not in args[i], args[i]
