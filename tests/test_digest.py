"""The digests that tie recorded measurements to the code they were taken of."""
import os
import re
import shutil

import bench
from speculative_decoding_verification_80_gb300 import build


def _recorded():
    with open(bench.PROFILE_TRAFFIC) as f:
        return re.search(r"^source_digest:\s*(\w+)", f.read(), flags=re.M).group(1)


def test_recorded_traffic_is_of_this_verify_kernel():
    assert build.verify_digest() == _recorded()
    assert all(bench.read_traffic(i, build.verify_digest()) is not None for i in "2345")


def test_verify_digest_has_what_the_verify_kernel_includes(tmp_path, monkeypatch):
    """A file of another operator does not move it, and one of its own does."""
    src, inc = str(tmp_path / "csrc"), str(tmp_path / "include")
    shutil.copytree(build.CSRC, src)
    shutil.copytree(build.INCLUDE, inc)
    monkeypatch.setattr(build, "CSRC", src)
    monkeypatch.setattr(build, "INCLUDE", inc)
    before, whole = build.verify_digest(), build.source_digest()
    assert before == _recorded()
    with open(os.path.join(src, "another_kernel.cuh"), "w") as f:
        f.write("int x;\n")
    assert build.verify_digest() == before and build.source_digest() != whole
    for name in ("api.cu", "verify_persistent.cuh", "philox.cuh", "ptx.cuh"):
        path = os.path.join(src, name)
        with open(path) as f:
            text = f.read()
        with open(path, "w") as f:
            f.write(re.sub(r"// ", "// and ", text))
        assert build.verify_digest() == before
        with open(path, "w") as f:
            f.write(text + "\nint x;\n")
        assert build.verify_digest() != before
        with open(path, "w") as f:
            f.write(text)
