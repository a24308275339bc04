"""Reads of what an earlier kernel may have written: kernels run under programmatic launch, so they start while their
predecessor still writes. Non-coherent loads are for memory that nothing writes while the kernel runs; the weights
alone are such."""
import glob
import os
import re

from quantized_activation_q4_gb300 import build


def sources():
    out = {}
    for p in sorted(glob.glob(os.path.join(build.CSRC, "*.cu*"))):
        with open(p) as f:
            text = f.read()
        out[os.path.basename(p)] = re.sub(r"//.*", "", text)
    return out


def test_no_read_goes_through_the_read_only_path_but_the_weights():
    for name, text in sources().items():
        assert not re.search(r"\b__ldg\b", text), name
        for use in re.finditer(r"ld\.global\.nc", text):   # inside the weight stream's loader
            assert "ldg_stream16" in text[max(0, use.start() - 200):use.start()], name


def test_no_kernel_takes_a_const_restrict_pointer():
    """The compiler may turn any read through one into a non-coherent load. The weight packers do not start early."""
    for name, text in sources().items():
        text = re.sub(r"__launch_bounds__\([^)]*\)", "", text)
        for k in re.finditer(r"__global__[^{;(]*?(\w+)\(([^{;]*?)\)\s*\{", text, flags=re.S):
            if k.group(1) not in ("pack_kernel", "pack_g_kernel"):
                assert not re.search(r"const \w+ \*__restrict__", k.group(2)), (name, k.group(1))
