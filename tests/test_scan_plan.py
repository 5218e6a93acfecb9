"""How the gated recurrence's launches are laid out, on the host: the library's own choice,
compiled with the questions to the CUDA runtime answered here instead of by a device."""
from __future__ import annotations

import os
import subprocess

from mel_spectrogram_gb300 import build

FAKES = r"""
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <cstdio>
#include <cstdlib>
#include <cstring>

static int largest = 16;  // blocks of a cluster that the device takes
static bool fails = false;  // whether questions are answered with an error
static int asked = 0;
static cudaError_t device_is(int* d) { *d = 0; return cudaSuccess; }
template <typename... A> static cudaError_t attribute_is(A...) { return cudaSuccess; }
template <typename K> static cudaError_t clusters_are(int* n, K, const cudaLaunchConfig_t* c) {
  ++asked;
  if (fails) return cudaErrorMemoryAllocation;
  const int ranks = (int)c->attrs[0].val.clusterDim.x;
  *n = ranks > largest ? 0 : 4 * 152 / ranks;
  return cudaSuccess;
}
#define cudaGetDevice device_is
#define cudaFuncSetAttribute attribute_is
#define cudaOccupancyMaxActiveClusters clusters_are
#include "fm_ops_scan.cu"

template <bool BACKWARD>
static scan::Split split_of(const scan::ScanParams& p) { return scan::Kernels<__nv_bfloat16, 8, BACKWARD, true>::split(p); }
static fm_scan_args args_of(long long batch, long long frames, long long channels, long long bytes) {
  fm_scan_args a{};
  a.batch = batch, a.frames = frames, a.channels = channels, a.dtype = FM_BF16;
  a.workspace = (void*)64, a.workspace_bytes = bytes;
  return a;
}
"""

# every stretch's sums, and where the row starts, lie in the workspace that was handed over
WORKSPACES = r"""
template <bool BACKWARD>
static int check(const fm_scan_args& a, int* cut) {
  const scan::Split s = split_of<BACKWARD>(params(&a));
  if (s.stretches <= 1) return 0;
  ++*cut;
  const long long writes = (s.stretches + 1LL) * a.batch * a.channels * 8;
  if (writes <= a.workspace_bytes) return 0;
  printf("%s %lld x %lld x %lld writes %lld bytes into %lld\n", BACKWARD ? "backward" : "forward", (long long)a.batch,
         (long long)a.frames, (long long)a.channels, writes, (long long)a.workspace_bytes);
  return 1;
}
int main(int, char** argv) {
  largest = atoi(argv[1]);
  int bad = 0, cut = 0;
  for (long long batch : {1, 2, 9, 300})
    for (long long frames : {100, 1000, 2416, 4000, 4095, 4096, 9000, 360001})
      for (long long channels : {1, 8, 16, 40, 80, 512, 4096, 8200}) {
        const fm_scan_args whole = args_of(batch, frames, channels, 0);
        const long long need = fm_scan_workspace(&whole);
        for (long long bytes : {0LL, 16LL, 4096LL, need - 1, need, need + 1, 1LL << 20}) {
          if (bytes < 0) continue;
          const fm_scan_args a = args_of(batch, frames, channels, bytes);
          bad += check<false>(a, &cut) + check<true>(a, &cut);
        }
      }
  printf("%d beyond, %d cut\n", bad, cut);
  return bad != 0 || cut == 0;
}
"""


def run(tmp_path, program, *args):
    source, exe = tmp_path / "plan.cu", tmp_path / "plan"
    source.write_text(FAKES + program)
    cmd = [build.nvcc(), *build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", f"-I{build.INCLUDE}", f"-I{build.CSRC}",
           str(source), "-o", str(exe), build.build(), "-Xlinker", f"-rpath={build.PKG}"]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    return [subprocess.run([str(exe), a], capture_output=True, text=True, env={**os.environ}) for a in args]


def test_stretches_stay_within_the_workspace(tmp_path):
    for r in run(tmp_path, WORKSPACES, "16", "8", "2"):
        assert r.returncode == 0, r.stdout + r.stderr


# a question that failed once is asked again; one that was answered is not
FAILURES = r"""
int main(int, char**) {
  const fm_scan_args a = args_of(1, 360001, 8, 1 << 20);
  const scan::ScanParams p = params(&a);
  fails = true;
  const scan::Split none = split_of<false>(p);
  if (none.ranks != 1 || none.stretches != 1 || none.rounds <= 0) return 1;
  int before = asked;
  fails = false;
  const scan::Split some = split_of<false>(p);
  if (asked == before) return 2;
  before = asked;
  const scan::Split again = split_of<false>(p);
  if (asked != before) return 3;
  printf("%d blocks, %d stretches\n", some.ranks, some.stretches);
  return some.stretches > 1 && again.stretches == some.stretches && again.ranks == some.ranks ? 0 : 4;
}
"""


def test_failed_questions_are_asked_again(tmp_path):
    (r,) = run(tmp_path, FAILURES, "")
    assert r.returncode == 0, (r.returncode, r.stdout, r.stderr)
