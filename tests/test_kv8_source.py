"""What the sources of the 8-bit cache's kernels must keep to and no call can show without risking the GPU."""
import os
import re

import sparse_attention_block_qsa_b200 as qsa

CSRC = os.path.join(os.path.dirname(qsa.__file__), "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_each_warpgroup_has_one_register_instruction():
    """setmaxnreg must be one and the same instruction for all four warps of a warpgroup: with a copy in each warp's
    own branch its effect is undefined, and the growing warpgroup may wait for ever."""
    kernel = source("attention_fp8.cuh").split("attn_fp8_kernel(const Params p) {")[1]
    calls = re.findall(r"regs_(?:shrink|grow)<(\w+)>\(\)", kernel)
    assert sorted(calls) == ["REGS_PROD", "REGS_REST", "REGS_SOFT"], calls
    # and the branch in front of each is taken by whole warpgroups
    branch = re.findall(r"(?:if \(([^{}]*)\)|else) \{\s*if constexpr \(C::RESIDENT > 1\) regs_(?:shrink|grow)<(\w+)>", kernel)
    assert branch == [("warp >= 4 && warp < 8", "REGS_PROD"), ("warp >= 8", "REGS_REST"), ("", "REGS_SOFT")], branch


def test_a_build_detail_of_one_kernel_refuses_its_own_call_only():
    """How many registers the 8-bit attention was built with is checked by that call, not by what every call shares."""
    lib = source("qsa_lib.cu")
    body = re.search(r"qsa_status_t device_info\(int\* sms\) \{\n(.*?)\n\}\n", lib, re.S).group(1)
    assert "cudaFuncSetAttribute" in body            # (this is the function meant)
    assert "numRegs" not in body and "attn8_registers" not in body
    check = re.search(r"qsa_status_t attn8_registers\(\) \{\n(.*?)\n\}\n", lib, re.S).group(1)
    assert "numRegs" in check and "REGS_LAUNCH" in check
    assert len(re.findall(r"= attn8_registers\(\);", lib.split("static qsa_status_t attention_fp8_common(")[1])) == 1
