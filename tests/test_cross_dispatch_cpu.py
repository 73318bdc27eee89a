"""The rules that choose among the cross attention kernels' forms (no GPU)."""

import os
import subprocess

import pytest

from exact_tiled_attention_08_gb300 import build, fa


def test_clusters_only_where_they_fit_and_pay(tmp_path):
    """Clusters of the forward, where the device holds 15, 36 and 76 of 8, 4 and 2 CTAs on 152 SMs."""
    source = tmp_path / "clusters.cu"
    source.write_text("""
#include "fa_cross_fwd.cuh"
int main() {
  const fa::CrossClusterFit fit{{15, 36, 76}}, none{{0, 0, 0}};
  for (int rows = 1; rows <= 128; rows += 127)
    for (bool alike : {false, true})
      for (int items = 1; items <= 200; ++items)
        for (int blocks = 1; blocks <= 2048; ++blocks) {
          const int c = fa::cross_cluster(items, blocks, rows, alike, 152, fit);
          if (c != 1 && c != 2 && c != 4 && c != 8) return 1;
          if (c > 1 && items > fit.clusters[c == 8 ? 0 : c == 4 ? 1 : 2]) return 2;  // a second wave of clusters
          if (blocks == 1 && c != 1) return 3;
          // a long item: a cluster of few CTAs would leave SMs without work
          if (blocks >= 256 && items * c < 100 && c > 1) return 4;
          if (fa::cross_cluster(items, blocks, rows, alike, 152, none) != 1) return 5;
        }
  if (fa::cross_cluster(8, 16, 4, true, 152, fit) != 8 || fa::cross_cluster(33, 16, 1, true, 152, fit) != 4) return 6;
  if (fa::cross_cluster(33, 1024, 1, true, 152, fit) != 1 || fa::cross_cluster(8, 512, 4, true, 152, fit) != 1) return 7;
  return 0;
}
""")
    program = tmp_path / "clusters"
    subprocess.run([build._nvcc(), *build.ARCH_FLAGS, "-std=c++17", "-I", build.CSRC_DIR, "-o", str(program), str(source)],
                   check=True, capture_output=True)
    assert subprocess.run([str(program)]).returncode == 0


@pytest.mark.parametrize("d", [64, 128])
def test_backward_workspace_has_room_for_the_runs_that_there_can_be(d):
    """Runs of cut items: at most one for each query block of each key block, and 608 in all."""
    build.build_library()
    run = 2 * 128 * d * 4
    for B, H, Hkv, Nq, Nk in [(1, 1, 1, 129, 1), (1, 2, 1, 64, 129), (1, 2, 1, 65, 129), (2, 8, 2, 300, 500), (4, 32, 8, 2000, 900)]:
        R, heads = H // Hkv * Nq, B * Hkv
        nqb, nkb = -(-R // 128), -(-Nk // 128)
        runs = 0 if nqb == 1 else min(608, heads * nqb * nkb)
        others = (heads * R * d * 4 if nkb > 1 else 0) + 2 * heads * nqb * 128 * 4
        got = fa.fa_cross_bwd_workspace_bytes(B, H, Hkv, Nq, Nk, d)
        assert runs * run + others <= got <= runs * run + others + 2048, (B, H, Hkv, Nq, Nk)
