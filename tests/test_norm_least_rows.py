"""How the norm's gradient shares rows out over CTAs: the rule by rows, groups a CTA and SMs, on the host."""
import os
import subprocess

from counted_notify_sync_gb300 import builder

SOURCE = r"""
#include <cstdio>
#include "rms_norm_kernels.cuh"
int main()
{
    const long rows[] = {1, 2, 3, 4, 5, 8, 9, 16, 17, 64, 100, 152, 153, 256, 304, 305, 500, 608, 609, 777, 2000, 5000, 100000, 2147483647};
    const int groups[] = {1, 2, 4, 8, 32};
    for (long r : rows)
        for (int g : groups) {
            const int each = cns::norm_least_rows(r, g, 152);
            std::printf("%ld %d %d %d\n", r, g, each, cns::norm_ctas(r, g, each, 304));
        }
    return 0;
}
"""


def test_ctas_up_to_the_sms_before_rows_to_a_group(tmp_path):
    (tmp_path / "r.cu").write_text(SOURCE)
    subprocess.run([os.path.join(builder.cuda_home(), "bin", "nvcc"), *builder.ARCH, "-O1", "-std=c++17", "-I", builder.INCLUDE,
                    "-I", builder.CSRC, "-o", str(tmp_path / "r"), str(tmp_path / "r.cu")], check=True)
    lines = subprocess.run([str(tmp_path / "r")], check=True, capture_output=True, text=True).stdout.splitlines()
    assert len(lines) == 24 * 5
    for line in lines:
        rows, groups, each, ctas = map(int, line.split())
        assert 1 <= each <= 4 and 1 <= ctas <= 304
        filled = -(-rows // groups)
        if filled <= 4:
            assert ctas == 1                       # one launch
        elif filled <= 152:
            assert each == 1 and ctas == filled    # no SM idles while a group has a second row
        elif filled <= 4 * 152:
            assert ctas <= 152 and (each - 1) * 152 < filled
        else:
            assert each == 4 and ctas == min(304, -(-rows // (4 * groups)))
