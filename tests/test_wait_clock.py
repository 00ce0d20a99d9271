"""CPU: where the time limit of a wait starts to count.  The difference, 64 polls
of about 80 ns, is too small to be timed from the host; the sources say it."""
import os
import re

import mixed_precision_matmul_gb300._build as _build


def source(name):
    with open(os.path.join(_build.CSRC, name)) as f:
        return f.read()


def test_the_limit_counts_from_the_start_of_a_wait():
    ptx = source("ptx.cuh")
    assert re.search(r"bool late_clock = false;", ptx)
    wait = ptx[ptx.index("bool mbar_wait("):]
    wait = wait[:wait.index("\n}\n")]
    assert "t0 = c.late_clock ? 0 : global_timer_ns();" in wait
    # only the operators whose header says so count from the 64th poll
    late = {s for s in _build.SOURCES + _build.HEADERS if s != "ptx.cuh" and "late_clock" in source(s)}
    assert late == {"fp8_gemm.cu", "fp8_pair.cu", "ortho.cu"}
    with open(os.path.join(_build.INCLUDE, "mpgemm.h")) as f:
        assert "product and the orthogonalised update count from the 64th poll" in f.read()
