"""Arithmetic of moe_linear's kernels at the largest sizes it accepts, run on the
host: the functions are those of the kernels' header."""
import subprocess

from routed_shared_experts_b200 import build

SRC = r"""
#include "linear.cuh"
#include <cstdio>

template <int OS>
int check() {
  int bad = 0;
  const int sizes[] = {1, 15, 16, 17, 31, 32, 33, 1000, (1 << 28) - 1, 1 << 28, (1 << 29) - 1, 1 << 29, (1 << 29) + 1,
                       (1 << 30) - 1, 1 << 30};
  for (const int N : sizes)
    for (long long back = 0; back < N; back = back < 70 ? back + 1 : back * 2) {
      for (const long long n0 : {back, N - 1 - back}) {
        if (n0 % (64 / OS) != 0) continue;  // chunks start on whole 64-byte columns
        const long long left = (N - n0) * OS;
        const int want = static_cast<int>(left < 64 ? left : 64);
        const int got = moe::chunk_bytes<OS>(N, static_cast<int>(n0));
        if (got != want && bad++ < 5) printf("OS %d N %d n0 %lld: %d, expected %d\n", OS, N, n0, got, want);
      }
    }
  return bad;
}

int main() { return check<2>() + check<4>() ? 1 : 0; }
"""


def _run(tmp_path, source):
    src, exe = tmp_path / "host.cu", tmp_path / "host"
    src.write_text(source)
    cmd = [build._nvcc(), "-O1", "-std=c++17", *build.ARCH, "-cudart", "static", "-I", build.INCLUDE, "-I", build.CSRC,
           "-o", str(exe), str(src)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    return subprocess.run([str(exe)], capture_output=True, text=True)


def test_chunk_bytes_up_to_the_largest_rows(tmp_path):
    """Bytes of a 64-byte chunk that a row of N values holds: T > 64 rows of 2^29
    fp32 results (140 GB) fit a GPU, and their chunks are whole."""
    run = _run(tmp_path, SRC)
    assert run.returncode == 0, run.stdout


TAIL = r"""
#include "linear.cuh"
#include <cstdio>

// A phase barrier as a count of completed phases: a wait on parity p passes when the
// current phase's parity is not p.
static bool passes(int completed, unsigned p) { return (completed & 1u) != p; }

int main() {
  int bad = 0;
  for (int n = 0; n < 50; ++n) {
    int used[2] = {0, 0};
    for (int j = 0; j < n; ++j) ++used[j & 1];
    for (int acc = 0; acc < 2; ++acc) {
      const int uses = moe::acc_uses(n, acc);
      if (uses != used[acc]) ++bad;
      if (uses == 0) continue;
      // before an accumulator's use the MMA thread has seen all releases but the last
      const unsigned p = moe::last_release_parity(uses);
      if (passes(uses - 1, p) || !passes(uses, p)) ++bad;
    }
  }
  printf("%d\n", bad);
  return bad != 0;
}
"""


def test_the_last_release_of_an_accumulator_is_waited_for(tmp_path):
    """The pair kernel's MMA thread ends with a wait for the release after each
    accumulator's last use: the wait must not pass on the release before it."""
    run = _run(tmp_path, TAIL)
    assert run.returncode == 0, run.stdout
