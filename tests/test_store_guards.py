"""The debug builds' store guard (CPU only): its condition, compiled for the
host, at the edges of a buffer; and, on the sources, that every global store of
the router, the row calls, the FP8 block quantizers and the FP8 block GEMM is
guarded by the addresses that it writes (a guard on the index that was just
compared with the same bound could never fail)."""
import ctypes
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "fp4_fp8_quantization_gb300", "csrc")


@pytest.fixture(scope="module")
def inside(tmp_path_factory):
    d = tmp_path_factory.mktemp("bounds")
    src = d / "b.cpp"
    src.write_text('#include "bounds.h"\n'
                   'extern "C" int inside(const void *at, int64_t n, const void *buf, int64_t size)\n'
                   '{ return moeq::range_inside(at, n, buf, size); }\n')
    lib = str(d / "b.so")
    subprocess.run(["g++", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", lib], check=True)
    f = ctypes.CDLL(lib).inside
    f.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64]
    return f


@pytest.mark.parametrize("base", [0x1000, 0x7F00_0000_0000])
def test_guard_condition_at_the_edges(inside, base):
    assert inside(base, 16, base, 64) and inside(base + 48, 16, base, 64)
    assert not inside(base - 1, 16, base, 64)          # before the buffer
    assert not inside(base - 16, 16, base, 64)
    assert not inside(base + 49, 16, base, 64)         # across its end
    assert not inside(base + 64, 1, base, 64)
    assert inside(base + 63, 1, base, 64)
    assert not inside(base, 65, base, 64)
    assert not inside(base, 4, base, 0)                # an empty buffer
    assert inside(base + (5 << 32), 16, base, (5 << 32) + 16)
    assert not inside(base + (5 << 32) + 1, 16, base, (5 << 32) + 16)


STORES = [r"\bst_global_v4\(", r"\btma_store_2d\(", r"\*reinterpret_cast<uint[24] \*>\([^;=]*\) =",
          r"\bp\.(?:dw|ids|weights|scales|out)\[[^\]]*\] =", r"\bscales\[[^\]]*\] =",
          r"(?<!\w )\*(?:ids|weights|scale|out|o) =", r"\bstore_logit<DT>\("]


def unguarded(src):
    """(stores found, lines of those without a guard): the guard is in the
    condition before the store, at most a few lines up."""
    src = re.sub(r"//[^\n]*", "", src)
    found, bad = 0, []
    for pattern in STORES:
        for m in re.finditer(pattern, src):
            before = src[max(0, m.start() - 900):m.start()]
            found += 1
            if not re.search(r"\b(?:store_fits|grad_fits<DT>)\(|store_ok\(cur\.row >= 0 ", before):
                bad.append(src.count("\n", 0, m.start()) + 1)
    return found, bad


def test_the_scan_finds_a_store_without_guard():
    assert unguarded("if (a < b) *out = v;") == (1, [1])
    assert unguarded("if (store_ok(a < b, e)) st_global_v4(o, 1, 2, 3, 4);") == (1, [1])
    assert unguarded("if (store_fits(o, 16, c, n, e)) st_global_v4(o, 1, 2, 3, 4);") == (1, [])


@pytest.mark.parametrize("name,least", [("gate.cu", 5), ("rows.cu", 3), ("fp8_block.cu", 4),
                                        ("gemm_fp8_block.cu", 3)])
def test_stores_are_guarded_by_address(name, least):
    with open(os.path.join(CSRC, name)) as f:
        found, bad = unguarded(f.read())
    assert found >= least and not bad, (found, bad)
