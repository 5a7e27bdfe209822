"""How the norm's kernels join the values of a row's warps, which lie in shared memory from a multiple of four places on
for each group of threads.  Groups have no barrier in common, so a group's result must not depend on the places that its
own warps do not write.  Host code alone, no GPU."""
import os
import subprocess

import pytest

from counted_notify_sync_gb300 import builder

SOURCE = r"""
#include <cmath>
#include <cstdio>
#include "rms_norm_kernels.cuh"

struct Sum { __host__ __device__ float operator()(float a, float b) const { return a + b; } };
struct Most { __host__ __device__ float operator()(float a, float b) const { return a != a || b != b ? NAN : a > b ? a : b; } };

// all shapes that with_shape launches, gradient or not: what no warp of the group has written is NaN
template <int G, int GROUPS>
void check()
{
    using J = cns::Joined<G, GROUPS>;
    for (int group = 0; group < GROUPS; ++group) {
        float4 s[J::kSize / 4];
        float *at = reinterpret_cast<float *>(s);
        for (int i = 0; i < J::kSize; ++i)
            at[i] = NAN;
        float sum = 0.f, most = 0.f;
        for (int w = 0; w < G / 32; ++w) {
            const float v = static_cast<float>((w * 7 + group * 3) % 32 + 1);
            at[group * J::kRoom + w] = v;
            sum += v;
            most = most > v ? most : v;
        }
        const float4 *of = s + group * (J::kRoom / 4);
        std::printf("%d %d %d %d\n", G, group, J::fold(of, Sum()) == sum, J::fold(of, Most()) == most);
    }
}

template <int G>
void both()
{
    check<G, cns::norm_groups(G, false)>();
    check<G, cns::norm_groups(G, true)>();
}

int main()
{
    both<64>(); both<96>(); both<128>(); both<160>(); both<192>(); both<224>(); both<256>();
    both<320>(); both<384>(); both<448>(); both<512>(); both<1024>();
    return 0;
}
"""


@pytest.fixture(scope="module")
def lines(tmp_path_factory):
    at = tmp_path_factory.mktemp("join")
    (at / "join.cu").write_text(SOURCE)
    subprocess.run([os.path.join(builder.cuda_home(), "bin", "nvcc"), *builder.ARCH, "-O1", "-std=c++17", "-I", builder.INCLUDE,
                    "-I", builder.CSRC, "-o", str(at / "join"), str(at / "join.cu")], check=True)
    got = subprocess.run([str(at / "join")], check=True, capture_output=True, text=True).stdout
    return [tuple(map(int, line.split())) for line in got.splitlines()]


def test_a_groups_result_is_its_own_warps(lines):
    assert {g for g, *_ in lines} == {64, 96, 128, 160, 192, 224, 256, 320, 384, 448, 512, 1024}
    assert max(group for _, group, *_ in lines) == 3          # the gradient's 64 threads a row: four groups a CTA
    for line in lines:
        assert line[2:] == (1, 1), line
