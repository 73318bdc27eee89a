"""The rules that choose among the cross attention kernels' forms (no GPU)."""

import os
import subprocess

from exact_tiled_attention_08_gb300 import build


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
