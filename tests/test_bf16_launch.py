"""A call of the bf16 products does not rest on what the compiler made of its kernels (no GPU needed)."""
import os
import re

import fp8_moe_expert_gb300 as fme

SOURCE = os.path.join(os.path.dirname(os.path.abspath(fme.__file__)), "csrc", "gemm_bf16.cu")


def test_no_launch_depends_on_the_number_of_registers():
    """A kernel whose warps ask for more registers than its launch has would wait for ever, and a launch that looks first and
    refuses would lose the call to another compiler: the kernels take what they are given."""
    code = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    assert not re.findall(r"setmaxnreg|cudaFuncGetAttributes|numRegs", code)
