"""The dense operators' compiled kernels and their launches, from the built
library's symbols and the sources; needs no GPU."""
import os
import re
import subprocess

from equivariant_interatomic_potentials_amd import etp

CSRC = os.path.join(os.path.dirname(os.path.abspath(etp.__file__)), "csrc")


def kernels(name):
    """Template arguments of every instantiation of a kernel in the library."""
    text = subprocess.run(["nm", "-C", etp._LIB_PATH], capture_output=True, text=True).stdout
    return {tuple(a.strip() for a in m.split(",")) for m in re.findall(r" etp::%s<([^>]*)>\(" % name, text)}


def test_products_of_a_kept_d_are_wide_ones_only():
    """d is kept where both widths pass 128: neither a resident matrix nor narrow results take it."""
    resident = kernels("product_resident_kernel")
    assert resident and not [k for k in resident if k[1] == "(etp::Dense)2"]
    stream = kernels("product_stream_kernel")
    assert stream and not [k for k in stream if k[1] == "(etp::Dense)2" and k[3] != "128"]


def test_every_layer_norm_kernel_is_taken_by_some_row():
    def shape(vecs, most):  # lanes of a row, vectors of a lane
        lpr = ni = 1
        while lpr < 16 and lpr < vecs:
            lpr *= 2
        while ni < most and lpr * ni < vecs:
            ni *= 2
        while lpr < 64 and lpr * ni < vecs:
            lpr *= 2
        while lpr * ni < vecs:
            ni *= 2
        return str(lpr), str(ni)

    for name, vjp in (("layer_norm_kernel", False), ("layer_norm_vjp_kernel", True)):
        for typ, vec in (("float", 4), ("unsigned short", 8)):
            want = {shape(-(-c // vec), 2 if vjp and vec == 8 else 4) for c in range(1, 2049)}
            assert {k[1:3] for k in kernels(name) if k[0] == typ} == want


def test_every_launch_is_checked():
    """A refused launch is reported by the call that made it, not by a later one: hipGetLastError follows each launch
    before the next launch or runtime call."""
    files = [f for f in sorted(os.listdir(CSRC)) if f in ("etp_linear.hip", "etp_layer_norm.hip", "etp_orth.hip")]
    assert len(files) == 3
    for f in files:
        text = open(os.path.join(CSRC, f)).read()
        launches = [m.end() for m in re.finditer(r"hipLaunchKernelGGL\(", text)]
        assert launches
        for i, at in enumerate(launches):
            rest = text[at:]
            check, other = rest.find("hipGetLastError"), re.search(r"hipFuncSetAttribute|\n}\n", rest)
            stop = other.start() if other else len(rest)
            assert 0 <= check < stop, (f, text[:at].count("\n") + 1)
