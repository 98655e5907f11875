"""Kernels that allocate tensor memory never wait for each other's: blocks that
fit an SM side by side by their shared memory have 512 columns together at most.

A host test: what each launch asks for, over every size that is accepted."""

import itertools
import os
import subprocess

import pytest

from int8_hadamard_rotated_convrot_gb300 import build as cbuild

SM_SHARED, BLOCK_RESERVE, COLUMNS = 228 * 1024, 1024, 512

# prints "columns bytes", one line for each launch
SOURCE = r"""
#include <cstdint>
#include <cstdio>
#include <initializer_list>
namespace convrot {
int lora_down_shared(int r);
bool fp8_few_takes(int64_t m, int64_t n, int64_t k);
bool fp8_few_quantizes(int64_t m, int64_t n, int64_t k);
int fp8_few_shared(int64_t m, int64_t n, int64_t k, bool quantize, int *columns);
}
int main()
{
    using namespace convrot;
    for (int r = 16; r <= 256; r += 16) printf("512 %d\n", lora_down_shared(r));
    for (int64_t m : {1, 2, 3, 5, 8, 13, 16, 17, 24, 32, 33, 48, 64, 65, 100, 128, 129, 300, 1000, 4000, 9000})
        for (int64_t n : {1, 128, 200, 640, 1024, 2056, 5120, 13824, 40000, 152064})
            for (int64_t k = 1; k <= 133144; k += k < 2048 ? 97 : k < 20000 ? 509 : 8111) {
                if (!fp8_few_takes(m, n, k)) continue;
                int columns = 0;
                const int packed = fp8_few_shared(m, n, k, false, &columns);
                printf("%d %d\n", columns, packed);
                if (fp8_few_quantizes(m, n, k)) printf("%d %d\n", columns, fp8_few_shared(m, n, k, true, &columns));
            }
}
"""


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    cbuild.build()
    folder = tmp_path_factory.mktemp("tmem")
    source, program = folder / "shapes.cpp", folder / "shapes"
    source.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-o", str(program), str(source), "-L", cbuild.BUILD, "-lconvrot",
                    "-Wl,-rpath," + cbuild.BUILD], check=True)
    lines = subprocess.run([str(program)], check=True, capture_output=True, text=True).stdout.split("\n")
    return {tuple(map(int, line.split())) for line in lines if line}


def test_no_mix_of_blocks_needs_more_columns_than_an_sm_has(launches):
    least = {}
    for columns, shared in launches:
        assert columns % 32 == 0 and 0 < columns <= COLUMNS and shared <= 227 * 1024
        least[columns] = min(shared, least.get(columns, shared))
    assert set(least) == {128, 256, 512}
    fits = SM_SHARED // (min(least.values()) + BLOCK_RESERVE)
    for n in range(1, fits + 2):
        for mix in itertools.combinations_with_replacement(sorted(least), n):
            if sum(least[c] + BLOCK_RESERVE for c in mix) <= SM_SHARED:
                assert sum(mix) <= COLUMNS, mix


def test_every_allocation_is_under_the_rule():
    """Kernels that allocate: the ones above, and those whose launch size is checked where it is defined."""
    found = set()
    for name in os.listdir(cbuild.CSRC):
        text = open(os.path.join(cbuild.CSRC, name)).read()
        if "tcgen05.alloc" in text:
            found.add(name)
            assert "tmem_share(" in text or "> kTmemAlone" in text, name
    assert found == {"block_fp8_few.cu", "block_fp8_gemm.cu", "gemm_tc.cu", "lora.cu"}
