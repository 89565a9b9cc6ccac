"""The grouped layer's compiled kernels, from the built library and its objects; needs no GPU."""
import os
import re
import shutil
import subprocess

import pytest

from equivariant_interatomic_potentials_amd import build

LLVM = "/opt/rocm/llvm/bin"


def test_products_of_a_kept_d_form_no_input_gradient(tmp_path):
    """Where d is kept, grad_x is a product of its own: the panels from d compile without theirs (half the matrix
    instructions, and the registers of W's fragments)."""
    obj = os.path.join(build.BUILD, "etp_grouped_vjp.o")
    tools = [shutil.which("objcopy"), os.path.join(LLVM, "clang-offload-bundler"), os.path.join(LLVM, "llvm-readelf")]
    if not all(t and os.path.exists(t) for t in (obj, *tools)):
        pytest.skip("needs the objects of the build and the toolchain")
    bundle, code = str(tmp_path / "bundle"), str(tmp_path / "code")
    subprocess.run([tools[0], "-O", "binary", "--only-section=.hip_fatbin", obj, bundle], check=True)
    subprocess.run([tools[1], "--type=o", f"--targets=hipv4-amdgcn-amd-amdhsa--{build.ARCH}", "--unbundle",
                    f"--input={bundle}", f"--output={code}"], check=True)
    text = subprocess.run([tools[2], "-s", "--wide", "--demangle", code], check=True, capture_output=True, text=True).stdout
    size = {m[1]: int(m[0]) for m in re.findall(r" (\d+) FUNC .*grouped_panel_kernel<([^>]*)>\(", text)}
    for typ in ("float", "unsigned short"):
        assert size[f"{typ}, 4, 4, false, true"] < 0.75 * size[f"{typ}, 4, 4, false, false"]
