"""The grouped layer's compiled kernels, from the built library and its objects; needs no GPU."""
import os
import re
import shutil
import subprocess

import pytest

import grouped_shapes as shapes
from equivariant_interatomic_potentials_amd import build, etp

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


def compiled():
    """Every instantiation in the library, as grouped_shapes names them."""
    text = subprocess.run(["nm", "-C", etp._LIB_PATH], capture_output=True, text=True).stdout
    out = set()
    for name, args in re.findall(r" etp::grouped_(\w+)_kernel<([^>]*)>\(", text):
        a = [re.sub(r"\(etp::Dense\)", "", v.strip()) for v in args.split(",")]
        if name != "slope":
            out.add((name, a[0], *(v == "true" if v in ("true", "false") else int(v) for v in a[1:])))
    return out


def test_every_kernel_is_taken_by_some_call():
    """No kernel without a call, and every one is run against float64 (tests/test_gpu_grouped_forms.py)."""
    have, taken = compiled(), shapes.all_forms()
    assert have - taken == set()
    assert taken - have == set()


def test_the_rules_are_the_sources():
    """The thresholds that grouped_shapes repeats stand in the dispatch as they do there."""
    text = open(os.path.join(os.path.dirname(etp.__file__), "csrc", "etp_grouped.hip")).read()
    assert "if (tiles * nc <= (lies ? 2048 : 128) || rows < (lies ? (is_float ? 64 : 32) : (is_float ? 48 : 0)))" in text
    assert "lies = a.p.KD <= 128" in text and "if (rows >= 4096)" in text
