"""Host and index arithmetic of the norm kernels, without a GPU: the functions of csrc/dwc_norm_host.h are
compiled with the host compiler and run over the sizes where they could go wrong."""
import os
import shutil
import subprocess

import pytest

from depthwise_convolution_nhwc_gb300 import _build


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    """Compile a main() against the header and return its output."""
    cuda = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc_path())), "include")

    def compile_and_run(body, head=""):
        d = tmp_path_factory.mktemp("host")
        src, exe = str(d / "t.cpp"), str(d / "t")
        with open(src, "w") as f:
            f.write(f'#include <cstdio>\n{head}\n#include "dwc_norm_host.h"\nint main() {{\n{body}\nreturn 0;\n}}\n')
        cxx = os.environ.get("CXX") or shutil.which("g++") or "c++"
        r = subprocess.run([cxx, "-std=c++17", "-O1", f"-I{_build.CSRC}", f"-I{cuda}", src, "-o", exe],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stdout + r.stderr
        return r.stdout

    return compile_and_run


def test_every_copy_names_an_aligned_address_inside_the_tensor(run):
    """Rows of C channels start r * C mod 8 elements past a vector boundary; a thread's vectors lie at columns
    8 k - shift.  What a copy of 16 bytes names must be a multiple of 16 bytes past the tensor's base and not
    before it, for granules past the row's end (copies of nothing) as for the others."""
    out = run(r"""
    long long copies = 0, empty = 0, bad = 0;
    for (int C = 1; C <= 700; ++C)
        for (int row = 0; row < 17; ++row) {
            const int shift = static_cast<int>((static_cast<long long>(row) * C) & 7);
            for (int n = 4; n <= 8; n += 4)                     // fp32, 16-bit types
                for (int col = -shift; col < C + 600; col += n) {
                    const long long at = static_cast<long long>(row) * C + dwc::copy_column(col, C, n);
                    ++copies;
                    empty += col >= C;
                    bad += at < 0 || at % n != 0 || (col < C && dwc::copy_column(col, C, n) != col);
                }
        }
    std::printf("%lld %lld %lld", copies, empty, bad);
    """)
    copies, empty, bad = map(int, out.split())
    assert copies > empty > 10 ** 6 and bad == 0


def test_cluster_counts_are_kept_by_device_and_shape(run):
    """Shapes that alternate are asked for once each; another device has its own answer; no answer is not kept."""
    out = run(r"""
    dwc::ClusterCounts counts;
    int asked = 0, wrong = 0;
    for (int i = 0; i < 10; ++i)
        for (int device = 0; device < 2; ++device)
            for (int threads = 256; threads <= 512; threads += 32)
                for (int cluster = 2; cluster <= 8; cluster *= 2) {
                    const int want = 1000 * device + threads + cluster;
                    wrong += counts.get(device, 65536, threads, cluster, [&] { ++asked; return want; }) != want;
                }
    std::printf("%d %d ", asked, wrong);
    int failed = 0;
    for (int i = 0; i < 3; ++i) failed += counts.get(0, 1, 32, 2, [&] { return 0; }) == 0;
    std::printf("%d %d", failed, counts.get(0, 1, 32, 2, [&] { return 5; }));
    """)
    assert out.split() == [str(2 * 9 * 3), "0", "3", "5"]


def test_more_shapes_than_places_are_answered_all_the_same(run):
    out = run(r"""
    dwc::ClusterCounts counts;
    int wrong = 0;
    for (int i = 0; i < 2; ++i)
        for (int k = 1; k <= 1000; ++k) wrong += counts.get(0, k, 32, 2, [&] { return k; }) != k;
    std::printf("%d", wrong);
    """)
    assert out == "0"
