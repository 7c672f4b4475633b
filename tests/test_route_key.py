"""The keys of the routing's choice (csrc/route_key.h), compiled for the host: they
order values and experts, and say what they do not hold of a value."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest

from sparse_shard_exchange_amd import build

SOURCE = """
#include "route_key.h"
extern "C" int key(float v, unsigned expert, unsigned names) { return pw::route_key(v, expert, names); }
extern "C" unsigned lacks(float v, unsigned names) { return pw::key_lacks(v, names); }
extern "C" float back(int key) { return pw::unordered(key); }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    at = tmp_path_factory.mktemp("key")
    (at / "key.hip").write_text(SOURCE)
    out = str(at / "key.so")
    subprocess.run([build.HIPCC, *build.COMMON, "-w", "-I", build.CSRC, "-shared", str(at / "key.hip"), "-o", out], check=True, timeout=120)
    lib = C.CDLL(out)
    lib.key.argtypes, lib.key.restype = [C.c_float, C.c_uint, C.c_uint], C.c_int
    lib.lacks.argtypes, lib.lacks.restype = [C.c_float, C.c_uint], C.c_uint
    lib.back.argtypes, lib.back.restype = [C.c_int], C.c_float
    return lib


def bf16(v):
    return (np.asarray(v, np.float32).view(np.uint32) & 0xffff0000).view(np.float32)


@pytest.mark.parametrize("names", [3, 15, 63, 255])
def test_bf16_values_of_either_sign_are_held_whole_and_ordered(lib, names):
    rng = np.random.default_rng(names)
    v = bf16(np.concatenate([rng.standard_normal(200) * 3, [-1.0, -0.5, 1.0, 0.0, -3e38, 3e38], rng.integers(-2, 3, 50)]))
    assert not any(lib.lacks(float(x), names) for x in v)
    e = rng.integers(0, names + 1, v.size)
    keys = np.array([lib.key(float(x), int(i), names) for x, i in zip(v, e)])
    assert np.array_equal(np.argsort(-keys, kind="stable"), np.lexsort((np.arange(v.size), e, -v)))


@pytest.mark.parametrize("names", [3, 15, 63, 255])
def test_values_of_more_bits_say_so(lib, names):
    rng = np.random.default_rng(names)
    v = rng.standard_normal(500).astype(np.float32)
    lacks = np.array([lib.lacks(float(x), names) for x in v])
    assert np.array_equal(lacks, v.view(np.uint32) & names) and (lacks != 0).mean() > 0.6
    keys = np.array([lib.key(float(x), 0, names) for x in v])
    order = np.argsort(-v)
    assert np.all(np.diff(keys[order]) <= 0)                 # never against the values' order
    near = np.array([lib.back(int(k) & ~names) for k in keys])
    assert np.all(np.abs(near - v) <= names * 2.0 ** -23 * np.abs(v))
