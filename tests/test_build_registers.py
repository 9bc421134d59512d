"""The build looks at the registers of the kernels that share them out: another count
than the shares' sum does not become a library."""

import pytest

from q4_quantized_linear_gb300 import build

SRC, (KERNEL, COUNT) = next(iter(build.SHARED_REGISTERS.items()))


def report(*kernels):
    """What ptxas -v says of kernels (name, registers)."""
    return "".join(f"ptxas info    : Compiling entry function '_ZN2q4{name}EE' for 'sm_103a'\n"
                   f"ptxas info    : Function properties for _ZN2q4{name}EE\n"
                   "    48 bytes stack frame, 16 bytes spill stores, 16 bytes spill loads\n"
                   f"ptxas info    : Used {n} registers, used 1 barriers\n" for name, n in kernels)


def test_the_count_of_the_shares():
    build.check_registers(SRC, "ptxas info    : 0 bytes gmem\n" + report((KERNEL + "Li64", COUNT), ("other", 40), (KERNEL + "Li128", COUNT)))


@pytest.mark.parametrize("n", [COUNT - 8, COUNT + 40])
def test_another_count(n):
    with pytest.raises(RuntimeError, match=str(n)):
        build.check_registers(SRC, report((KERNEL + "Li64", COUNT), (KERNEL + "Li128", n)))


def test_a_report_without_the_kernels():
    for log in ("", report(("other", COUNT))):
        with pytest.raises(RuntimeError):
            build.check_registers(SRC, log)


def test_other_sources_are_not_asked():
    build.check_registers("q4mm_pack.cu", "")


def test_the_build_asks(monkeypatch, tmp_path):
    """A compiler that gives other registers fails the build of that source."""

    class Done:
        returncode, stdout, stderr = 0, "", report((KERNEL + "Li64", COUNT - 8))

    def run(cmd, **kw):
        assert "-v" in cmd
        open(cmd[cmd.index("-o") + 1], "w").close()
        return Done()

    monkeypatch.setattr(build.subprocess, "run", run)
    with pytest.raises(RuntimeError, match="shares"):
        build._compile(SRC, False, str(tmp_path))
    assert not (tmp_path / SRC.replace(".cu", ".o")).exists()
