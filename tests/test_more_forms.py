"""Which kernel takes which sizes, as the host rules have it (no call here reaches a kernel)."""

import subprocess

import pytest

from int8_hadamard_rotated_convrot_gb300 import build as cbuild

SOURCE = r"""
#include <cstdint>
#include <cstdio>
#include <cstdlib>
namespace convrot { bool gated_few_takes(int64_t m, int64_t n, int64_t k); }
int main(int n, char **v)
{
    for (int i = 1; i + 2 < n; i += 3) printf("%d\n", convrot::gated_few_takes(atoll(v[i]), atoll(v[i + 1]), atoll(v[i + 2])));
}
"""


@pytest.fixture(scope="module")
def few_takes(tmp_path_factory):
    cbuild.build()
    source, program = (tmp_path_factory.mktemp("forms") / name for name in ("forms.cpp", "forms"))
    source.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-o", str(program), str(source), "-L", cbuild.BUILD, "-lconvrot", "-Wl,-rpath," + cbuild.BUILD], check=True)

    def run(*sizes):
        r = subprocess.run([str(program), *(str(v) for s in sizes for v in s)], check=True, capture_output=True, text=True)
        return [line == "1" for line in r.stdout.split()]

    return run


def test_rows_past_128_go_where_k_is_shared_out(few_takes):
    """m, n, k. Long and narrow layers keep the kernel that shares k out up to 256 rows; the others leave it at 129."""
    narrow = [(m, n, k) for m in (129, 200, 256) for n, k in ((640, 13824), (1, 13824), (3840, 5120), (1920, 1280))]
    assert all(few_takes(*narrow))
    wide = [(m, n, k) for m in (129, 256) for n, k in ((13824, 5120), (5120, 1280), (2560, 640), (2560, 1280), (8, 64), (1 << 30, 1 << 30))]
    assert not any(few_takes(*wide))
    assert all(few_takes((1, 13824, 5120), (128, 13824, 5120), (128, 8, 1))) and not any(few_takes((257, 640, 13824), (1 << 30, 1, 1 << 30)))
