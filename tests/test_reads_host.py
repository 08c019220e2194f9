"""The places that the GEMM kernels' direct-to-LDS loads read, computed on the CPU by the functions
that the kernels use: every load is whole and inside its matrix, or dropped by its vector offset."""
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
I64 = ctypes.c_int64


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("reads") / "reads.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-shared", "-fPIC", os.path.join(HERE, "host_model", "reads.cpp"),
                    "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.f8_bad_reads.restype = ctypes.c_long
    lib.f8_bad_reads.argtypes = [ctypes.c_int] + [I64] * 5
    lib.bf16_bad_reads.restype = ctypes.c_long
    lib.bf16_bad_reads.argtypes = [ctypes.c_int] * 4 + [I64] * 4
    return lib


@pytest.mark.parametrize("tile", range(11))
def test_f8_tiles_read_inside_their_matrices(model, tile):
    """One token or row up to more than the widest tile, whole tiles among them, K of whole and half steps, wide rows."""
    for M in (1, 8, 33, 64, 128, 136, 256, 264, 385, 520):
        for N in (1, 7, 33, 64, 192, 200, 257, 300):
            for K, pad in ((64, 0), (192, 48), (256, 4096)):
                assert model.f8_bad_reads(tile, M, N, K, K + pad, (M + 7) // 8 * 8 + pad) == 0, (M, N, K, pad)


@pytest.mark.parametrize("asteps", [2, 4], ids=["sparse", "dense"])
@pytest.mark.parametrize("bm,bn,lw", [(64, 64, 4), (128, 128, 4), (128, 256, 8), (192, 128, 4), (256, 256, 4), (256, 512, 8)])
def test_bf16_tiles_read_inside_their_matrices(model, bm, bn, lw, asteps):
    for M in (1, 32, 33, 64, 129, 192, 256, 300, 420, 513):
        for N in (1, 9, 64, 130, 257):
            for K, pad in ((64, 0), (192, 8), (256, 2048)):
                assert model.bf16_bad_reads(bm, bn, lw, asteps, M, N, K, K + pad) == 0, (M, N, K, pad)
