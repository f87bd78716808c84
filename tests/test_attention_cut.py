"""The cut of spec_attention's list of tiles (csrc/attention_cut.cuh), replayed on
the CPU: every tile is one CTA's, and the CTA that joins an item's parts waits for
exactly those CTAs that have one."""
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "speculative_decoding_verification_80_gb300", "csrc")


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("cut") / "cut.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-x", "c++", f"-I{CSRC}",
                    os.path.join(HERE, "cuda", "attention_cut.cpp"), "-o", out], check=True)
    lib = ctypes.CDLL(out)
    lib.cut_of_all.restype = ctypes.c_longlong
    return lib


@pytest.mark.parametrize("first,rows,tiles,chunk", [
    (399, 64, 3, 10),   # 14 tokens of 64 query and 8 key heads over 300 positions: two CTAs without a tile at its start
    (159, 64, 3, 10),   # the third request of 6, 6 and 8 tokens of 8 heads over 16, 3231 and 260 positions
    (9, 64, 40, 10), (0, 64, 3, 10), (5, 40, 7, 11), (9, 16, 1, 10), (0, 16, 1, 1000)])
def test_join_expects_the_ctas_that_have_tiles(cut, first, rows, tiles, chunk):
    assert cut.cut_of_item(first, rows, tiles, chunk) == 0


def test_cut_from_every_unit(cut):
    where = (ctypes.c_int * 5)()
    assert cut.cut_of_all(60, 80, where) == 0, list(where)
