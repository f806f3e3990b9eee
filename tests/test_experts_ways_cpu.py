"""Which kernels the GPU tests of the 8-bit products run, decided by the host's
rules as they are compiled: a rule that changes may not empty a test."""
import shutil

import pytest

from tests import waykit

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")


def test_every_way_has_a_test_of_wrong_offsets():
    gpu = pytest.importorskip("tests.test_gpu_experts_offsets")
    assert set(gpu.CASES) == set(waykit.NAMES.values())
    for way, (counts, k, n, spare) in gpu.CASES.items():
        for planes in (1, 2):
            assert waykit.way_of_counts(planes, counts, k, n, spare) == way


def test_tile_tests_reach_tiles():
    gpu = pytest.importorskip("tests.test_gpu_experts_tiles")
    for planes in (1, 2):
        for rows, n in gpu.DENSE:
            for k in gpu.INPUTS + [199]:
                assert gpu.dense_way(planes, rows, k, n) == "together", (planes, rows, k, n)
        for k in gpu.INPUTS + [1019]:
            assert waykit.way_of_counts(planes, gpu.COUNTS, k, 4801 if planes == 1 else 2401, 7) == "together", k
    for rows, k, n in gpu.LONG:
        assert waykit.way(1, rows, k, n) == "together", (rows, k, n)


def test_tile_tests_reach_every_body():
    gpu = pytest.importorskip("tests.test_gpu_experts_tiles")
    alone = set().union(*(waykit.heights([rows]) for rows, _ in gpu.DENSE if rows <= 256))
    shared = set().union(*(waykit.heights([rows]) for rows, _ in gpu.DENSE if rows > 256))
    assert alone == {64, 128, 192, 256} and shared == {192, 256}
    assert waykit.heights(gpu.COUNTS) == alone
    stages = {(k + 63) // 64 for k in gpu.INPUTS}
    assert min(stages) == 1 and max(stages) > 8  # shorter than every ring, and longer
