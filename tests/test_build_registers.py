"""The build holds the attention kernels' registers, as the compiler reports
them, against those that their warpgroups share out (no GPU needed)."""
import pytest

from speculative_verification_gb300 import build as ss_build

ENTRY = """ptxas info    : Compiling entry function '_ZN3ssa11attn_kernelILi%dELb%dELi%dELi%dEEEv14CUtensorMap_stS1_S1_NS_8AttnArgsE' \
for 'sm_103a'
ptxas info    : Function properties for _ZN3ssa11attn_kernel
    48 bytes stack frame, 96 bytes spill stores, 148 bytes spill loads
ptxas info    : Used %d registers, used 16 barriers, 48 bytes cumulative stack size, 16432 bytes smem
"""


def test_the_reported_registers_are_those_shared_out():
    good = [(64, 1, 2, 96, 96), (8, 1, 1, 80, 80), (16, 0, 2, 0, 180), (128, 0, 1, 96, 96)]
    ss_build.check_registers("".join(ENTRY % e for e in good))
    for i, e in enumerate(good):
        for used in (e[4] - 8, e[4] + 8):
            bad = list(good)
            bad[i] = (*e[:4], used)
            log = "".join(ENTRY % x for x in bad)
            if e[3] == 0:  # nothing is shared out: any number will do
                ss_build.check_registers(log)
            else:
                with pytest.raises(RuntimeError, match="%d rows.*used %d registers" % (e[0], used)):
                    ss_build.check_registers(log)


def test_a_report_without_the_kernels_is_no_pass():
    with pytest.raises(RuntimeError):
        ss_build.check_registers("ptxas info    : Used 96 registers\n")


def test_the_build_checks_both_formats(monkeypatch):
    seen = []
    check = ss_build.check_registers
    monkeypatch.setattr(ss_build, "check_registers", lambda log: (seen.append(log), check(log)))
    ss_build.build(force=True)
    assert len(seen) == len(ss_build.SHARED_REGISTERS) == 2
    assert seen[0].count("attn_kernel") >= 10 and seen[1].count("attn_kernel") >= 8
