"""The split of the dense paged attention among the CTAs, and what its join accepts as a record: the
header is plain C++, compiled here by the host compiler."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dsa_sparse_attention_mla_gb300", "csrc")


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    d = tmp_path_factory.mktemp("split")
    src = d / "split.cc"
    src.write_text('#include "dsa_paged_split.h"\nusing namespace dsa::paged;\nextern "C" {\n'
                   "int share_of(int c, int total, int G) { return share(c, total, G); }\n"
                   "int max_ctas() { return kMaxCtas; }\n"
                   "int valid(int row, int first, int last, int total, long long nrows, int G, int block) {\n"
                   "  return record_valid(row, first, last, total, nrows, G, block);\n}\n}\n")
    lib = d / "split.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    lib = ctypes.CDLL(str(lib))
    lib.valid.argtypes = [ctypes.c_int] * 4 + [ctypes.c_longlong] + [ctypes.c_int] * 2
    return lib


def test_shares(split):
    rng = random.Random(0)
    for total in [1, 2, 151, 152, 153, 10 ** 6, 2 ** 31 - 1] + [rng.randrange(1, 2 ** 31) for _ in range(50)]:
        for G in (1, 2, 148, 152, split.max_ctas()):
            assert [split.share_of(c, total, G) for c in range(G + 1)] == [c * total // G for c in range(G + 1)]


@pytest.mark.parametrize("nrows,G,block", [(7, 152, 3), (5000, 152, 3), (152, 152, 3)])
def test_records(split, nrows, G, block):
    def ok(row, first, last, total):
        return bool(split.valid(row, first, last, total, nrows, G, block))

    row = 4000 if nrows > G else block
    assert ok(row, 0, 0, 1) and ok(row, 0, G - 1, 2 ** 31 - 1) and ok(row, 5, 9, 77)
    for bad in (-1, -2 ** 31, nrows, 2 ** 31 - 1):
        assert not ok(bad, 5, 9, 77)
    for first, last in ((-1, 9), (5, G), (9, 5), (5, 2 ** 31 - 1), (-2 ** 31, -1), (G, G)):
        assert not ok(row, first, last, 77)
    for total in (0, -1, -2 ** 31):
        assert not ok(row, 5, 9, total)
    # at most G rows: a block joins its own row alone
    assert ok(block + 1, 5, 9, 77) == (nrows > G)
