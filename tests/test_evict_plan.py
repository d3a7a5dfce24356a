"""How many CTAs share a request in the eviction, by what the device can hold: the rule alone, compiled for the host."""
import ctypes as C
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_mla_decode_paged_gb300", "csrc")


@pytest.fixture(scope="module")
def cluster(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, so = d / "plan.cpp", d / "plan.so"
    src.write_text('#include "smla_evict_plan.h"\nextern "C" int cluster(int requests, int cols, int sms, int most) {\n'
                   '  return smla::evict_cluster(requests, cols, sms, most);\n}\n')
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(so)], check=True)
    return C.CDLL(str(so)).cluster


def test_a_whole_device(cluster):
    assert [cluster(1, n, 152, 16) for n in (1, 8192, 8193, 16385, 32769, 327680, 327681, 1 << 30)] == [1, 1, 2, 4, 8, 8, 16, 16]
    assert [cluster(r, 400000, 152, 16) for r in (9, 10, 19, 20, 38, 39, 76, 77, 65535)] == [16, 8, 8, 4, 4, 2, 2, 1, 1]


@pytest.mark.parametrize("most", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("requests", [1, 2, 9, 40, 200])
@pytest.mark.parametrize("cols", [1, 9000, 70000, 340000, 1 << 30])
def test_never_more_than_the_device_holds(cluster, most, requests, cols):
    """Where 16 CTAs do not fit, 8 read the keys anew; where the device holds fewer, it gets fewer."""
    n = cluster(requests, cols, 152, most)
    assert n <= most and n == min(most, cluster(requests, cols, 152, 16))
