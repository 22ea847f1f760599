"""The build's own checks: kernels that may not spill registers."""
import os

import pytest

from precision_grouped_gemm_gb300 import build

LOG = """ptxas info    : 0 bytes gmem
ptxas info    : Compiling entry function '_Z6first_v' for 'sm_103a'
ptxas info    : Function properties for _Z6first_v
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used 64 registers, used 1 barriers
ptxas info    : Compiling entry function '_Z6second_v' for 'sm_103a'
ptxas info    : Function properties for _Z6second_v
    8 bytes stack frame, {0} bytes spill stores, {1} bytes spill loads
ptxas info    : Used 254 registers, used 1 barriers
"""


def test_spills_are_read_from_the_log():
    assert build.spilled(LOG.format(0, 0)) == []
    assert build.spilled(LOG.format(12, 28)) == [("_Z6second_v", 12)]
    assert build.spilled(LOG.format(0, 4)) == [("_Z6second_v", 0)]


def test_kernels_beside_tensor_memory_spill_nothing():
    build.build()
    assert "linear.cu" in build.NO_SPILLS
    for src in build.NO_SPILLS:
        assert src in build.SOURCES
        with open(os.path.join(build.BUILD, src.replace(".cu", ".o.log"))) as f:
            log = f.read()
        assert "spill stores" in log and build.spilled(log) == [], src


def test_a_spill_fails_the_build(tmp_path, monkeypatch):
    """A compiler whose log tells of a spill: the build raises, and leaves no object that a later one would take."""
    fake = tmp_path / "nvcc"
    fake.write_text("#!/bin/sh\nwhile [ $# -gt 0 ]; do [ \"$1\" = -o ] && : > \"$2\"; shift; done\n"
                    "cat <<'END' >&2\n" + LOG.format(12, 28) + "END\n")
    fake.chmod(0o755)
    monkeypatch.setattr(build, "nvcc", lambda: str(fake))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "out"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "SOURCES", ["join.cu", "linear.cu"])
    with pytest.raises(RuntimeError, match="spill"):
        build.build()
    assert os.path.exists(tmp_path / "out" / "join.o") and not os.path.exists(tmp_path / "out" / "linear.o")
    monkeypatch.setattr(build, "SOURCES", ["join.cu"])
    build.build()
