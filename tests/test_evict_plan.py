"""How hyb_evict_select is laid out over a cluster of CTAs, compiled by itself for
the host: every entry has a place, and no cluster is larger than the device allows."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "compressed_sparse_sliding_b200", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "evict_plan.cuh"
int main()
{
    int B, Nc, sms, cluster;
    while (std::scanf("%d %d %d %d", &B, &Nc, &sms, &cluster) == 4) {
        const hyb::EvictPlan p = hyb::evict_plan(B, Nc, sms, cluster);
        std::printf("%d %d %d\n", p.ranks, p.keys, p.slice);
    }
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host compiler")
def test_every_entry_has_a_place(tmp_path):
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-x", "c++", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    sizes = [1, 2, 1000, 2047, 4096, 4099, 32768, 32769, 65537, 262144, 262145, 300001, 524288, 524289, 600001,
             (1 << 30) - 1]
    cases = [(B, Nc, sms, cluster) for B in (1, 2, 9, 64, 148, 65535) for Nc in sizes for sms in (148, 16, 1)
             for cluster in (16, 8)]
    out = subprocess.run([str(exe)], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True,
                         text=True, check=True).stdout.split("\n")
    for (B, Nc, sms, cluster), line in zip(cases, out):
        ranks, keys, piece = map(int, line.split())
        assert ranks in (1, 2, 4, 8, 16) and ranks <= cluster
        if keys:
            assert keys in (1, 2, 4, 8, 16, 32) and ranks * keys * 1024 >= Nc
        else:      # read again in every pass, by clusters that any device can place
            assert Nc > cluster * 32 * 1024 and ranks == 8 and ranks * piece >= Nc and piece % 4 == 0
