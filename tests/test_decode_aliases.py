"""Outputs of the cache's forks and moves, and of sampling, that lie on inputs or on
one another: refused on the host (CPU only; every call here is refused, so that none
launches a kernel)."""
import ctypes

import pytest

import speculative_decoding_verification_80_gb300 as sd

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_80_gb300 import build

    build.build()
    return sd.load_library()


FORK = ["block_table", "kv_len", "accepted_len", "held", "parent", "keep", "shares", "free_ring", "ring_state", "table_out", "kv_len_out",
        "held_out", "shares_out", "ring_state_out", "copies", "count", "workspace", "error_word"]


def _fork(lib, **at):
    """kv_fork of 4 old and 6 new requests, 8 blocks a row, 100 blocks; arrays 64 KB apart but for those in `at`."""
    p = {name: 0x100000 + 0x10000 * i for i, name in enumerate(FORK[:-2])}
    p["workspace"], p["error_word"] = 0x10000000, 0x20000000
    p.update(at)
    a = [P(p[name]) for name in FORK]
    return lib.kv_fork(4, 6, 16, 8, 100, *a[:-1], sd.page_workspace_bytes(100), a[-1], None)


AT = {name: 0x100000 + 0x10000 * i for i, name in enumerate(FORK[:-2])}


@pytest.mark.parametrize("out", ["table_out", "kv_len_out", "held_out", "copies", "count", "free_ring", "workspace", "error_word"])
@pytest.mark.parametrize("on", ["block_table", "kv_len", "accepted_len", "held", "parent", "keep", "shares", "ring_state"])
def test_fork_refuses_outputs_on_inputs(lib, out, on):
    assert _fork(lib, **{out: AT[on]}) == 1


@pytest.mark.parametrize("out,on,by", [("shares_out", "shares", 4), ("shares_out", "shares", -4), ("ring_state_out", "ring_state", 4),
                                       ("shares_out", "ring_state", 0), ("ring_state_out", "shares", 0), ("kv_len_out", "parent", 20),
                                       ("kv_len_out", "parent", -20), ("held_out", "block_table", 124), ("table_out", "held", -188)])
def test_fork_refuses_parts_on_parts(lib, out, on, by):
    assert _fork(lib, **{out: AT[on] + by}) == 1


@pytest.mark.parametrize("a,b", [("table_out", "kv_len_out"), ("kv_len_out", "held_out"), ("copies", "table_out"), ("count", "copies"),
                                 ("shares_out", "free_ring"), ("ring_state_out", "count"), ("workspace", "free_ring"),
                                 ("workspace", "shares_out")])
def test_fork_refuses_outputs_on_one_another(lib, a, b):
    assert _fork(lib, **{a: AT[b]}) == 1


COMPACT = ["block_table", "held", "shares", "free_ring", "ring_state", "table_out", "shares_out", "ring_out", "ring_state_out", "renamed",
           "copies", "count", "workspace", "error_word"]
MOVED = {name: 0x100000 + 0x10000 * i for i, name in enumerate(COMPACT[:-2])}


def _compact(lib, **at):
    """kv_compact of 4 requests, 8 blocks a row, 100 blocks."""
    p = {**MOVED, "workspace": 0x10000000, "error_word": 0x20000000, **at}
    a = [P(p[name]) for name in COMPACT]
    return lib.kv_compact(4, 8, 100, *a[:-1], sd.page_workspace_bytes(100), a[-1], None)


@pytest.mark.parametrize("out,on,by", [("table_out", "block_table", 4), ("table_out", "block_table", -124), ("shares_out", "shares", 396),
                                       ("ring_out", "free_ring", -4), ("ring_state_out", "ring_state", 4), ("shares_out", "free_ring", 0),
                                       ("ring_out", "shares", 0), ("table_out", "held", 0), ("renamed", "shares", 0), ("renamed", "block_table", 0),
                                       ("copies", "free_ring", 0), ("count", "ring_state", 0), ("workspace", "shares", 0),
                                       ("error_word", "held", 12)])
def test_compact_refuses_outputs_on_other_inputs(lib, out, on, by):
    assert _compact(lib, **{out: MOVED[on] + by}) == 1


@pytest.mark.parametrize("a,b", [("table_out", "renamed"), ("shares_out", "ring_out"), ("copies", "renamed"), ("count", "copies"),
                                 ("ring_state_out", "count"), ("renamed", "workspace")])
def test_compact_refuses_outputs_on_one_another(lib, a, b):
    at = {**MOVED, "workspace": 0x10000000}[b]
    assert _compact(lib, **{a: at}) == 1


SAMPLE = ["logits", "out", "draft_len", "temperature", "top_k", "top_p", "min_p", "uniform", "tokens", "error_word"]
ROWS = {name: 0x1000000 * (i + 1) for i, name in enumerate(SAMPLE)}


def _sample(lib, dtype=1, **at):
    """spec_sample of 3 requests of 2 rows of 1000 logits."""
    a = [P({**ROWS, **at}[name]) for name in SAMPLE]
    return lib.spec_sample(*a[:2], dtype, 3, 1, 1000, *a[2:], None)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("by", [4, -4, 2000, -2000, 11996, -11996])
def test_sample_refuses_rows_that_overlap(lib, by, dtype):
    assert _sample(lib, dtype, out=ROWS["logits"] + by) == 1


@pytest.mark.parametrize("out,on,by", [("tokens", "logits", 11996), ("tokens", "out", 0), ("tokens", "uniform", 0), ("tokens", "top_k", -20),
                                       ("out", "uniform", -11996), ("error_word", "tokens", 20), ("error_word", "temperature", 8)])
def test_sample_refuses_other_overlaps(lib, out, on, by):
    assert _sample(lib, **{out: ROWS[on] + by}) == 1
