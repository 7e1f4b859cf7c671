"""The sums that a drawn token comes from, on the host: the functions are taken from the kernel's source, compiled with traps on every
operation that C++ leaves undefined (signed overflow, shifts of negative numbers), and compared with whole numbers."""
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

from test_step_sources import text

SHIMS = r"""
#include <cfenv>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <vector>
#define __device__
#define __forceinline__ inline
using u64 = unsigned long long;
static uint32_t __float_as_uint(float f) { uint32_t u; memcpy(&u, &f, 4); return u; }
static float __saturatef(float f) { return f != f ? 0.0f : f < 0.0f ? 0.0f : f > 1.0f ? 1.0f : f; }
template <class F> static float toward_zero(F f) { const int was = fegetround(); fesetround(FE_TOWARDZERO); volatile float r = f(); fesetround(was); return r; }
static float __fadd_rz(volatile float a, volatile float b) { return toward_zero([&] { return a + b; }); }
static float __fmaf_rz(float a, float b, float c) { return toward_zero([&] { volatile float x = a, y = b, z = c; return std::fma((float)x, (float)y, (float)z); }); }
struct Row { const float *p, *q; int gone; };
"""
MAIN = r"""
int main()
{
    int32_t head[2];  // values of a row, whether a second one follows
    if (fread(head, 4, 2, stdin) != 2) return 2;
    std::vector<float> p(head[0]), q(head[0]);
    if (fread(p.data(), 4, p.size(), stdin) != p.size()) return 2;
    if (head[1] && fread(q.data(), 4, q.size(), stdin) != q.size()) return 2;
    u64 sum = 0;
    for (int lane = 0; lane < 32; ++lane) {
        const Row row{p.data(), q.data(), -1};
        sum += head[1] ? lane_sum<8, true>(row, 0, head[0], lane) : lane_sum<16, false>(row, 0, head[0], lane);
    }
    printf("%llu\n", sum);
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    s = text("verify.cu")
    # the calls above are those of the kernel
    assert "lane_sum<8, true>" in s and "lane_sum<16, false>" in s
    taken = re.search(r"struct Pieces \{.*?(?=template <int THREADS>)", s, re.S)[0]
    at = tmp_path_factory.mktemp("sums")
    source, out = os.path.join(at, "sums.cpp"), os.path.join(at, "sums")
    with open(source, "w") as f:
        f.write(SHIMS + taken + MAIN)
    subprocess.run([gxx, "-std=c++17", "-O1", "-frounding-math", "-ffp-contract=off", "-w", "-fsanitize=undefined",
                    "-fsanitize-undefined-trap-on-error", source, "-o", out, "-lm"], check=True)
    return out


def _run(program, p, q=None):
    data = np.array([len(p), q is not None], np.int32).tobytes() + p.astype(np.float32).tobytes() + (b"" if q is None else q.astype(np.float32).tobytes())
    done = subprocess.run([program], input=data, capture_output=True)
    assert done.returncode == 0, f"ended with {done.returncode}: an operation that C++ leaves undefined"
    return int(done.stdout)


def _units(p):
    p = np.nan_to_num(np.clip(np.float32(p).astype(np.float64), 0, 1), nan=0.0)
    return [int(v) for v in np.floor(np.ldexp(p, 62))]


ROWS = {
    "ordinary": lambda g, n: g.dirichlet(np.ones(n)),
    "few likely": lambda g, n: g.dirichlet(np.full(n, 0.01)),
    "one certain": lambda g, n: np.eye(1, n, n // 2)[0],
    "tiny": lambda g, n: np.exp2(-g.uniform(0, 90, n)) / n,
    "odd": lambda g, n: np.where(np.arange(n) % 7 == 0, np.nan, np.where(np.arange(n) % 5 == 0, -1.0, g.dirichlet(np.ones(n)))),
}


@pytest.mark.parametrize("n", [1, 15, 32, 33, 511, 512, 5003])
@pytest.mark.parametrize("kind", ROWS)
def test_sums_are_exact_and_defined(program, kind, n):
    g = np.random.default_rng(n)
    p, q = ROWS[kind](g, n), ROWS["ordinary"](g, n)
    assert _run(program, p) == sum(_units(p)) % 2 ** 64
    for a, b in ((p, q), (q, p)):
        assert _run(program, a, b) == sum(max(x - y, 0) for x, y in zip(_units(a), _units(b))) % 2 ** 64
