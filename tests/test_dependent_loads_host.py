"""The kernels that are launched as programmatic dependents can be resident while the
kernel before them still writes their inputs.  A non-coherent load (ld.global.nc,
__ldg) promises data that nobody writes during the whole kernel, wherever in the kernel
it stands, so those kernels have none.  Checked on the source text."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_quantized_linear_gb300", "csrc")
NON_COHERENT = re.compile(r"__ldg\b|\bld_stream_v4\b|\bload16\b|ld\.global\.nc|__restrict__")


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def function(text, name):
    """The definition of __global__ function `name`: its text up to the closing brace in column 0."""
    m = re.search(r"__global__[^;{]*?\b" + name + r"\([^;]*?\)\s*\n\{.*?\n\}", text, re.S)
    assert m, name
    return m.group(0)


@pytest.mark.parametrize("name", ["gemm.cu", "gemm_pair.cu", "gemm_common.cuh", "epilogue.cuh", "norm_quant.cu", "moe.cu"])
def test_files_of_dependents_have_no_non_coherent_load(name):
    assert NON_COHERENT.findall(source(name)) == []


def test_the_quantizer_has_no_non_coherent_load():
    assert NON_COHERENT.findall(function(source("quant.cu"), "quant_kernel")) == []


def test_kernels_with_non_coherent_loads_are_launched_in_stream_order():
    """Those of quant.cu go out by <<<>>>, which has no programmatic edge to the kernel before."""
    text = source("quant.cu")
    for name in ("quant_mx_kernel", "act_amax_kernel", "quant_transform_kernel"):
        assert NON_COHERENT.search(function(text, name))
        assert re.search(name + r"(<\w+>)?\s*<<<", text) and not re.search(r"cudaLaunchKernelEx\([^;]*" + name, text)
