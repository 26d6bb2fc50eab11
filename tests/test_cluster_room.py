"""The shared memory that a cluster's launch may ask for covers every plan:
the receive buffer of (rows, CTAs) is not largest at the most CTAs, since each
CTA's slice is rounded up (16 rows over 15 CTAs need more than over 16)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_gqa_decode_06_gb300", "csrc")
SMS = 152

PROGRAM = """
#include <cstdio>
#include "split_mma.cuh"
using pgd::ClusterRecv;
int main() {
  const int dims[] = {64, 128, 256};
  for (int D : dims)
    for (int rows = 1; rows <= 16; ++rows)
      for (int S = 2; S <= 16; ++S)
        std::printf("%d %d %d %d %d\\n", D, rows, S, ClusterRecv::of(rows, D, S).bytes,
                    ClusterRecv::limit(D));
}
"""


@pytest.fixture(scope="module")
def pkg():
    from paged_gqa_decode_06_gb300 import build
    build.build()
    import paged_gqa_decode_06_gb300 as p
    p.load_library()
    return p


@pytest.fixture(scope="module")
def room(tmp_path_factory):
    """{(head_dim, rows, CTAs): (bytes of the receive buffer, the launchers' limit)}"""
    from paged_gqa_decode_06_gb300 import build
    d = tmp_path_factory.mktemp("room")
    (d / "room.cu").write_text(PROGRAM)
    r = subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I",
                        CSRC, str(d / "room.cu"), "-o", str(d / "room")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    out = subprocess.run([str(d / "room")], check=True, capture_output=True, text=True).stdout
    rows = [[int(x) for x in line.split()] for line in out.splitlines()]
    return {(D, n, S): (need, limit) for D, n, S, need, limit in rows}


def test_every_receive_buffer_is_within_the_limit(room):
    assert len(room) == 3 * 16 * 15
    for key, (need, limit) in room.items():
        assert need <= limit, key


def test_every_cluster_plan_is_within_the_limit(pkg, room):
    """What the planners choose by themselves, and what a caller may ask for."""
    chosen = set()
    for D, Hq, Hkv, T in ((256, 16, 1, 1), (256, 32, 2, 1), (256, 64, 4, 1), (256, 16, 2, 2),
                          (128, 16, 1, 1), (128, 8, 2, 4), (64, 16, 1, 1), (64, 12, 4, 5)):
        for batch in (1, 2, 4):
            for bound in range(257, 7000, 61):
                for schedule in (0, 2):
                    p = pkg.DecodeAttnParams(batch, Hq, Hkv, D, 16, 512, 4096, bound, 0.1, 0, 0, 0,
                                             0, T, 0, schedule)
                    for plan_of in (pkg.decode_attn_make_plan, pkg.decode_attn_quant_make_plan):
                        try:
                            plan = plan_of(p, SMS)
                        except pkg.DecodeAttnError:
                            assert schedule == 2  # no cluster for this shape
                            continue
                        if plan.cluster:
                            heads = plan.grid_y  # shards of a cluster lie along x
                            rows = T * (Hq // heads)
                            need, limit = room[D, rows, plan.cluster]
                            assert need <= limit, (plan.as_dict(), D, rows)
                            chosen.add((D, rows, plan.cluster, schedule))
    assert any(c[:3] == (256, 16, 15) and c[3] == 0 for c in chosen)
    assert (64, 16, 15, 2) in chosen and (128, 16, 15, 2) in chosen
