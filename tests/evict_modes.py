"""How paged_kv_evict shares a request's keys and holds their weights, by the
library's own rule (csrc/va_budget.h), compiled into a small host program."""
import os
import shutil
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MODES = ("whole", "halves", "reread")

_SOURCE = r"""
#include <stdio.h>
#include "va_budget.h"
int main() {
  long long units, most;
  int chunks, sms, n;
  while (scanf("%lld %d %d %lld %d", &units, &chunks, &sms, &most, &n) == 5) {
    const int cluster = va::evict_cluster(units, chunks, sms), cap = va::evict_slice_cap(most, cluster);
    const int slice = va::evict_slice(n, cluster);
    printf("%d %d %d %d\n", cluster, cap, slice, va::evict_held(slice, cap));
  }
  return 0;
}
"""


def shapes(tmp_path, asked):
    """asked: (units, 16-byte chunks of a K and V row, SMs, max_kv_len, keys of a
    request).  Returns (cluster, weights of two bytes a CTA has room for, keys it
    looks after, mode) of each."""
    src, exe = str(tmp_path / "shape.cpp"), str(tmp_path / "shape")
    with open(src, "w") as f:
        f.write(_SOURCE)
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "speculative_decoding_verify_gqa_gb300", "csrc"), "-I", cuda,
                    src, "-o", exe], check=True)
    text = "".join("%d %d %d %d %d\n" % a for a in asked)
    out = subprocess.run([exe], input=text, check=True, capture_output=True, text=True).stdout.split()
    rows = [tuple(map(int, out[i:i + 4])) for i in range(0, len(out), 4)]
    assert len(rows) == len(asked)
    return [r[:3] + (MODES[r[3]],) for r in rows]
