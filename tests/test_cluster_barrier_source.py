"""Source rule of the cluster kernels (CPU only): the aligned cluster barrier is undefined where a
warp's lanes come to it apart, which no run shows reliably, so every one of them has the lanes brought
together directly ahead of it."""
import pathlib
import re

CSRC = pathlib.Path(__file__).resolve().parents[1] / "persistent_megakernel_decode_04_b200" / "csrc"


def test_aligned_cluster_barriers_come_after_a_warp_barrier():
    found = 0
    for p in sorted(list(CSRC.glob("*.cu")) + list(CSRC.glob("*.cuh"))):
        lines = [line.split("//")[0].strip() for line in p.read_text().splitlines()]
        lines = [line for line in lines if line]
        for at, line in enumerate(lines):
            if re.search(r"barrier\.cluster\.(arrive|wait)[\w.]*\.aligned", line):
                found += 1
                assert "__syncwarp();" in lines[at - 1], f"{p.name}: {line}"
    assert found >= 2
