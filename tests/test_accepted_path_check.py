"""The device check of an accepted path's nodes, compiled for the host: a node that
it lets pass must keep both of its rows inside the cache, whatever the rest of the
path holds, since each thread looks its own node's blocks up."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gqa_attention_cu_gb300", "csrc")


@pytest.fixture(scope="module")
def node_ok(tmp_path_factory):
    d = tmp_path_factory.mktemp("path")
    src, lib = d / "path.cpp", d / "path.so"
    src.write_text('#include "pva_path.h"\n'
                   'extern "C" int node_ok(const int32_t* path, int i, int past, long long rows) {\n'
                   "  return pva::path_node_ok(path, i, past, rows);\n}\n")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", str(lib), str(src)], check=True)
    fn = ctypes.CDLL(str(lib)).node_ok
    fn.argtypes = [ctypes.POINTER(ctypes.c_int32), ctypes.c_int, ctypes.c_int, ctypes.c_longlong]
    return lambda path, i, past, rows: bool(fn((ctypes.c_int32 * len(path))(*path), i, past, rows))


def paths():
    big = 2 ** 31 - 1
    yield list(range(64)) + [0, 1] + list(range(2, 64)), 0, 64
    yield list(range(-100, 28)), 0, 64
    yield [-3, -2, -1, 0], 15, 16
    yield [-big - 1] * 3 + [big], big, big
    yield list(range(-5, 5)), big - 3, big
    r = random.Random(1)
    for _ in range(300):
        n, rows = r.randint(1, 40), r.randint(1, 60)
        path = [r.choice([r.randint(-3, 60), i, i + r.randint(0, 3)]) for i in range(n)]
        yield path, r.randint(0, rows), rows


def test_looked_up_rows_lie_in_the_cache(node_ok):
    for path, past, rows in paths():
        for i, x in enumerate(path):
            if node_ok(path, i, past, rows):
                assert 0 <= past + i < rows and 0 <= past + x < rows, (path, i, past, rows)


def test_a_path_passes_whole_if_it_rises_inside_the_cache(node_ok):
    for path, past, rows in paths():
        sound = path[0] >= 0 and all(a < b for a, b in zip(path, path[1:])) and past + path[-1] < rows
        assert all(node_ok(path, i, past, rows) for i in range(len(path))) == sound
    assert all(node_ok([0, 2, 5, 6], i, 3, 10) for i in range(4))
