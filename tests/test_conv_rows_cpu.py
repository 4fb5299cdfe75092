"""Rows of the final states that the convolution's backward reads for a token, by the library's own index
functions compiled for the host: never outside the states, whatever the packed offsets say, and the right
ones where they are consistent."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include <cstdio>
#include <vector>
#include "gdn_layer.cuh"

int main() {
    // consistent; ending early (a batch padded at its end); empty at the end; out of order; beyond the tokens
    const std::vector<std::vector<int>> all = {{0, 30, 71}, {0, 0, 71}, {0, 71, 71}, {0, 30, 60}, {0, 0}, {0, 1}, {0, 60, 60},
                                               {0, 180, 71}, {0, -5, 71}, {3, 30, 71}, {0, 60, 20}, {90, 100}};
    for (size_t i = 0; i < all.size(); ++i) {
        const std::vector<int> &cu = all[i];
        const int N = (int)cu.size() - 1, total = 71;
        const gdn::SeqMap m{cu.data(), N, total, total};
        for (int w1 = 1; w1 <= 3; ++w1) {
            std::vector<int> seen((size_t)N * w1, 0);
            // every pair of a sequence and a token, the walk behind the last sequence's end among them
            for (int n = 0; n < N; ++n)
                for (int t = 0; t < total; ++t) {
                    const long long k = gdn::kept_row(n, m.end(n), t, w1);
                    if (k < 0) continue;
                    if (k >= (long long)N * w1) {
                        printf("offsets %d, W %d: token %d of sequence %d reads row %lld of %d\n", (int)i, w1 + 1, t, n, k, N * w1);
                        return 1;
                    }
                    if (i < 3 && t >= m.begin(n)) {
                        if (k != (long long)n * w1 + w1 - (m.end(n) - t)) return 2;
                        ++seen[k];
                    }
                }
            for (int n = 0; i < 3 && n < N; ++n) {  // each of a sequence's last tokens in one row, once
                const int len = m.end(n) - m.begin(n);
                for (int j = 0; j < w1; ++j)
                    if (seen[(size_t)n * w1 + j] != (j >= w1 - len)) return 3;
            }
        }
    }
    return 0;
}
"""


def test_rows_of_the_final_states(tmp_path):
    from gated_deltanet_chunked_rule_b200 import build
    src, exe = tmp_path / "rows.cu", tmp_path / "rows"
    src.write_text(SOURCE)
    r = subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", build.CSRC,
                        "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, (r.returncode, r.stdout)
