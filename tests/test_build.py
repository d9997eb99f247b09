"""The build refuses a kernel whose registers at the launch are not what its setmaxnreg split counts on (CPU only)."""

import os

import pytest

from weight_only_bit_qgemv_b200 import build


def log_of(*regs):
    return "".join(
        f"ptxas info    : Compiling entry function '_ZN3woq18attn_prompt_kernelILi64ELi{i}EEE' for 'sm_100a'\n"
        "    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads\n"
        f"ptxas info    : Used {n} registers, used 1 barriers\n" for i, n in enumerate(regs))


def test_registers_at_the_launch():
    source = open(os.path.join(build.CSRC, "attn_prompt.cu")).read()
    other = log_of(64).replace("attn_prompt_kernel", "attn_split_kernel")
    build.check_registers("attn_prompt.cu", source, log_of(168, 168) + other)
    build.check_registers("kv4.cu", "", log_of(32))  # no split, no demand
    for log in (log_of(168, 160), log_of(170), other, ""):
        with pytest.raises(RuntimeError):
            build.check_registers("attn_prompt.cu", source, log)


def test_the_built_library_passed_it():
    log = os.path.join(build.BUILD, "attn_prompt.cu.log")
    if not os.path.exists(log):
        pytest.skip("the library was not built here")
    build.check_registers("attn_prompt.cu", open(os.path.join(build.CSRC, "attn_prompt.cu")).read(), open(log).read())
