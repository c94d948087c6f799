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
