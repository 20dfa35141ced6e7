"""4-bit pages without a GPU: what the append takes fp32's rotation to be off by."""
import math
import os
import random
import struct
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "host_offloaded_kv_gb300", "csrc")


def compiled(tmp_path, body):
    """Runs a program over the header's functions; its output's words."""
    from host_offloaded_kv_gb300 import _build

    src = tmp_path / "probe.cu"
    src.write_text('#include <cstdio>\n#include <initializer_list>\n#include "clo_rotate_exact.cuh"\nusing namespace clo;\n' + body)
    exe = str(src)[:-3]
    subprocess.run([_build._nvcc(), "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-I", CSRC, str(src), "-o", exe], check=True)
    return subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()


def f32(x):
    return struct.unpack("f", struct.pack("f", x))[0]


def test_error_of_a_rotated_element_counts_every_rounding(tmp_path):
    # x = m (p cos - q sin): p^2 + q^2 is (r / m)^2 with r the rotated pair's length, so |p| + |q| <= sqrt(2) r / m and |p cos| + |q sin| <= r / m.
    # u: half a step of fp32, relative; sine and cosine are off by 7.5e-8 each.
    u = 2.0 ** -24
    rng = random.Random(1)
    pairs = [(f32(abs(rng.gauss(0, 1))), f32(abs(rng.gauss(0, 1)) * 2.0 ** rng.uniform(-20, 20))) for _ in range(300)]
    pairs += [(1.0, 1.0), (1.0, 0.0), (0.0, 1.0), (3.0, 4.0), (1e30, 1e-30)]
    rows = ", ".join("{%sf, %sf}" % (x.hex(), y.hex()) for x, y in pairs)
    got = compiled(tmp_path, "int main() { const float p[][2] = {%s}; for (auto& v : p) for (bool one : {true, false}) printf(\"%%.9g \", rotation_error(v[0], -v[1], one)); }" % rows)
    for i, (x, y) in enumerate(pairs):
        r = math.hypot(x, y)
        for k, magnitude in enumerate((0.0, u)):
            # sines, product with q, sums with the magnitude; then the sum, the quotient by the group's scale, an end of the interval
            need = (7.5e-8 * math.sqrt(2.0) + u + magnitude) * r + 3 * u * max(x, y)
            assert float(got[2 * i + k]) >= need * (1 + 1e-5), (x, y, k)  # (products of two of the errors: far below 1e-5 of one)


def test_zeros_of_either_sign_are_one_code(tmp_path):
    # every pair of codes in every place, between neighbours of which some differ
    got = compiled(tmp_path, r'''
int main() {
  for (int k = 0; k < 8; ++k)
    for (unsigned lo = 0; lo < 16; ++lo)
      for (unsigned hi = 0; hi < 16; ++hi) {
        const uint32_t rest = 0x1908a3f0u & ~(15u << 4 * k);
        uint32_t low = rest | lo << 4 * k;
        const uint32_t d = codes_differ(&low, rest | hi << 4 * k);
        printf("%u %u %d ", d, low >> 4 * k & 15u, (low & ~(15u << 4 * k)) == rest);
      }
}
''')
    at = iter(map(int, got))
    for k in range(8):
        for lo in range(16):
            for hi in range(16):
                zeros = lo & 7 == 0 and hi & 7 == 0
                want = 0 if lo == hi or zeros else 1 << 4 * k
                assert (next(at), next(at), next(at)) == (want, 0 if zeros and lo != hi else lo, 1), (k, lo, hi)
