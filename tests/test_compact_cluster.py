"""How many CTAs of a cluster the compaction gives a sequence, head and pool: the host's choice, compiled by
itself (no CUDA call), for devices that hold clusters of 16, of the portable 8, or fewer."""
import pathlib
import shutil
import subprocess

import pytest

CSRC = pathlib.Path(__file__).resolve().parent.parent / "gemm_conv_chains_gb300" / "csrc"
PROGRAM = """
#include <cstdio>
#include "decoder.h"
int main() {
  long long items;
  int wave, tokens, sms, most;
  while (std::scanf("%lld %d %d %d %d", &items, &wave, &tokens, &sms, &most) == 5)
    std::printf("%d\\n", b2b::compact_ctas(items, wave, tokens, sms, most));
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    headers = pathlib.Path(nvcc).resolve().parent.parent / "include"
    if not (headers / "cuda_runtime.h").exists() or shutil.which("g++") is None:
        pytest.skip("no CUDA headers or no g++")
    at = tmp_path_factory.mktemp("cluster")
    (at / "choose.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", str(headers), "-I", str(CSRC), "-I", str(CSRC.parent.parent / "include"),
                    "-o", str(at / "choose"), str(at / "choose.cpp")], check=True)

    def run(rows):
        text = "".join(" ".join(map(str, r)) + "\n" for r in rows)
        out = subprocess.run([str(at / "choose")], input=text, capture_output=True, text=True, check=True).stdout
        return [int(x) for x in out.split()]
    return run


def test_no_cluster_is_larger_than_the_device_holds(choose):
    rows = [(items, wave, tokens, sms, most) for items in (1, 2, 4, 9, 38, 76, 152, 10 ** 9) for wave in (64, 128, 256)
            for tokens in (1, 64, 65, 700, 30011, 2 ** 31 - 1) for sms in (16, 132, 152) for most in (16, 8, 4, 2, 1)]
    for (items, wave, tokens, sms, most), ctas in zip(rows, choose(rows)):
        assert 1 <= ctas <= most and ctas & (ctas - 1) == 0
        if ctas > 1:                                 # half as many would leave SMs idle, and tokens to a later wave
            assert items * ctas // 2 < sms and ctas // 2 * wave < tokens
        if ctas < most:
            assert items * ctas >= sms or ctas * wave >= tokens


def test_one_long_sequence(choose):
    assert choose([(4, 256, 30011, 152, most) for most in (16, 8, 4, 2, 1)]) == [16, 8, 4, 2, 1]
    assert choose([(1024, 64, 6, 152, 16), (256, 256, 4096, 152, 16), (4, 256, 700, 152, 16)]) == [1, 1, 4]
