"""The build's look at the register counts that a launch depends on (no GPU needed)."""
import os

import pytest

from rotated_int2_kv_kvq_gb300 import build

SRC = os.path.join(build.CSRC, "kvq_prefill.cu")


def _log(*entries):
    return "".join(
        f"ptxas info    : Compiling entry function '{name}' for 'sm_103a'\n"
        f"ptxas info    : Function properties for {name}\n"
        f"    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads\n"
        f"ptxas info    : Used {regs} registers, used 2 barriers\n" for name, regs in entries)


INT2, BF16 = "_ZN3kvq1x14prefill_kernelILb1EEEvv", "_ZN3kvq1x14prefill_kernelILb0EEEvv"
OTHER = ("_ZN3kvq1x22prefill_combine_kernelEv", 90)


def test_exact_count_passes():
    build.check_registers(SRC, _log(OTHER, (INT2, 128), (BF16, 128)))


@pytest.mark.parametrize("entries", [
    [(INT2, 128), (BF16, 127)], [(INT2, 120), (BF16, 128)], [(INT2, 128)], [OTHER],
    [(INT2, 128), (BF16, 128), (BF16, 128)], []])
def test_other_counts_stop_the_build(entries):
    with pytest.raises(RuntimeError, match="prefill_kernel needs 128 registers"):
        build.check_registers(SRC, _log(*entries))


def test_the_sources_constant():
    """REGISTERS repeats the source's own number."""
    with open(SRC) as f:
        assert "constexpr int kRegLaunch = 128;" in f.read()
    assert build.REGISTERS["kvq_prefill.cu"][1] == 128
