"""CPU: the limits of the attention kernels' work slots (csrc/attn_view.cuh), compiled for the host."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SLOTS = r"""
#include <climits>
#include <cstdio>
#include "attn_view.cuh"
using namespace sf;
int main() {
  const long long rows = 1ll << 26;   // rows x heads per key/value head that a call accepts, all in one sequence
  const int tiles[] = {8, 16, 128}, logs[] = {3, 4, 7};
  for (int k = 0; k < 3; ++k) {
    const int cu[2] = {0, (int)rows};
    for (long long t = rows / tiles[k] - 3; t < rows / tiles[k]; ++t) {
      const int idx = slot_index(t - slot_base(cu, 0, 1, logs[k], 1));
      if (idx != t) return printf("tile %lld of %d rows has index %d\n", t, tiles[k], idx), 1;
    }
    if (slot_index(LLONG_MAX / 2) * (long long)tiles[k] > INT_MAX) return printf("rows of %d do not fit\n", tiles[k]), 1;
  }
  return 0;
}
"""

ORDER = r"""
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "attn_view.cuh"
using namespace sf;
int main() {
  srand(2);
  for (int trial = 0; trial < 2000; ++trial) {
    const int n = 1 + rand() % 40, T = rand() % 600, log = 3 + rand() % 5;
    std::vector<int> cu(n + 1);
    for (int& x : cu) x = rand() % (T + 1);
    if (trial % 4) std::sort(cu.begin(), cu.end());
    if (trial % 4 == 2) cu[rand() % (n + 1)] += rand() % 7 - 3;
    bool wrong = false, found = false;
    for (int i = 0; i < n; ++i) wrong = wrong || cu[i] < 0 || cu[i + 1] > T || cu[i] > cu[i + 1];
    for (long long u = 0; u < (T >> log) + n; ++u) found = found || bad_offsets(cu.data(), u, n, T);
    if (wrong != found) return printf("trial %d: offsets %s, reported %d\n", trial, wrong ? "wrong" : "fine", found), 1;
  }
  return 0;
}
"""


def run_on_host(source, tmp_path):
    nvcc = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
    if shutil.which(nvcc) is None:
        pytest.skip("nvcc not available")
    src, exe = tmp_path / "slots.cu", tmp_path / "slots"
    src.write_text(source)
    inc = os.path.join(ROOT, "streaming_speaker_diarization_b200", "csrc")
    r = subprocess.run([nvcc, "-std=c++17", "-arch=sm_100a", "-I", inc, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_the_last_tile_of_the_largest_call_has_a_slot(tmp_path):
    run_on_host(SLOTS, tmp_path)


def test_offsets_out_of_order_are_found_whatever_sequences_own_slots(tmp_path):
    run_on_host(ORDER, tmp_path)
