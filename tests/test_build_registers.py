"""The build's check on the registers of a kernel whose warps pass them on (CPU)."""
import pytest

from paged_kv_decode_25_gb300 import build

LINE = """ptxas info    : Compiling entry function '_ZN2mi%s' for 'sm_103a'
ptxas info    : Function properties for _ZN2mi%s
    8 bytes stack frame, 16 bytes spill stores, 20 bytes spill loads
ptxas info    : Used %d registers, used 1 barriers, 8 bytes cumulative stack size, 6144 bytes smem
"""


def report(**kernels):
    return "".join(LINE % (name, name, n) for name, n in kernels.items())


def test_numbers_are_read():
    text = report(prefill_tc2_kernelILi64EE=128, slide_tc2_kernelILi128EE=96, slide_tc2_kernelILi64EE=88)
    assert build.launch_registers(text, "slide_tc2_kernel") == [96, 88]
    assert build.launch_registers(text, "prefill_tc2_kernel") == [128]
    assert build.launch_registers("", "slide_tc2_kernel") == []


def test_other_numbers_are_refused():
    build.check_registers(report(other=40, slide_tc2_kernelILi128EE=96, slide_tc2_kernelILi64EE=96))
    build.check_registers("")
    for kernels in (dict(slide_tc2_kernelILi128EE=96, slide_tc2_kernelILi64EE=88), dict(slide_tc2_kernelILi64EE=104)):
        with pytest.raises(RuntimeError, match="kSlideRegs"):
            build.check_registers(report(**kernels))
