"""Cluster sizes of the pool's plans and of the verification (csrc/pool_rules.h, built for the host):
up to eight CTAs, which every device schedules, or sixteen, the one larger size for which the
launches ask the device and keep its answer. CPU only."""
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("pool_host") / "pool_host.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", os.path.join(HERE, "host", "pool_host.cpp"),
                    "-I", os.path.join(ROOT, "exact_io_aware_13_gb300", "csrc"), "-o", out], check=True)
    lib = ctypes.CDLL(out)
    lib.host_plan_ctas.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int]
    return lib


@pytest.mark.parametrize("num_sms", [1, 16, 132, 148, 152])
def test_verification(host, num_sms):
    sizes = [*range(0, 70_000, 997), 4095, 4096, 28_672, 32_767, 32_768, 50_257, 61_439, 61_440, 128_256, 256_000,
             2 ** 30]
    for B in [*range(1, 80), 100, 152, 608, 609, 5000, 2 ** 26]:
        for V in sizes:
            n = host.host_verify_ctas(num_sms, B, V)
            assert 1 <= n <= 8 or n == 16, (B, V, n)
            assert n <= V // 4096 + 1                         # a CTA has something to read
            assert n == 1 or n * B <= 4 * num_sms             # and all of them are held at once


def test_plans(host):
    for one, each in ((12288, 4096), (2048, 2048), (16384, 16384)):
        last = 1
        for work in [0, 1, one, one + 1, *range(0, 40 * each, each // 2), 2 ** 31 - 1]:
            n = host.host_plan_ctas(work, one, each)
            assert n in (1, 2, 4, 8, 16)
            assert (n == 1) == (work <= max(one, each))
        for work in range(0, 40 * each, each):
            n = host.host_plan_ctas(work, one, each)
            assert n >= last
            last = n
