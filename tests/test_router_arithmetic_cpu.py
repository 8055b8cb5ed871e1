"""Arithmetic of the training router that a GPU run shows only in rare cases: its own pieces, compiled for the host."""
import os
import subprocess

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_fp8_mixture_topk_gb300", "csrc", "router.cuh")
SHIM = r"""
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#define __device__
#define __forceinline__ inline
using std::fma;
static uint64_t bits(double v) { uint64_t b; memcpy(&b, &v, 8); return b; }
static double number(uint64_t b) { double v; memcpy(&v, &b, 8); return v; }
static int __double2loint(double v) { return (int)(uint32_t)bits(v); }
static int __double2hiint(double v) { return (int)(uint32_t)(bits(v) >> 32); }
static double __hiloint2double(int hi, int lo) { return number((uint64_t)(uint32_t)hi << 32 | (uint32_t)lo); }
"""


def run(tmp_path, pieces, main):
    """What a host program of these pieces of the source ((first words, words after the end)) prints."""
    text = open(SOURCE).read()
    code = SHIM
    for begin, end in pieces:
        at = text.index(begin)
        code += text[at:text.index(end, at)]
    (tmp_path / "a.cpp").write_text(code + "int main() {\n" + main + "\n}\n")
    subprocess.run(["g++", "-std=c++17", "-O2", "-ffp-contract=off", "-o", str(tmp_path / "a"), str(tmp_path / "a.cpp")], check=True)
    return subprocess.run([str(tmp_path / "a")], check=True, capture_output=True, text=True).stdout.split()


def test_slack_of_keys_covers_their_error(tmp_path):
    """For each number of experts a lane, in units of 2^-24.  The factor that softmax scores share: V - 1 additions in a lane and 5
    across lanes, the exponentials' 2 ulp (4) and the rounding of their arguments (1.44 of the mean exponent, which ln 1024 = 6.94
    bounds), the reciprocal's 2 ulp (4), twice the largest bias.  Of each of two keys its own score's part: exponential 4, product
    or quotient 2 and sums 1 each."""
    got = run(tmp_path, [("constexpr float kRel", "// Scores from logits")], r"""
    const float b = 0.37f;
#define ONE(V) printf("%d %.9g %.9g ", V, key_slack<V, false>(b, 0.01f), key_slack<V, true>(b, 0.01f));
    ONE(1) ONE(2) ONE(4) ONE(8) ONE(16) ONE(32) ONE(64)
    printf("%.9g", kRel);""")
    u, b = 2.0 ** -24, 0.37
    rel = float(got.pop())
    for V, soft, sigm in zip(*[iter(got)] * 3):
        shared = (int(V) - 1 + 5 + 4 + 1.44 * 6.94 + 4) * u
        own = 2 * (4 + 2 + 1) * u
        assert float(soft) >= 2 * b * shared + own * b, V
        assert float(sigm) >= own * b + 2 * 2.0 ** -23.5, V
        assert rel >= own


@pytest.fixture(scope="module")
def exponential(tmp_path_factory):
    """Largest errors, in 2^-53 of the value, of exp64 and of sigmoid64 over ranges of the argument, and what is not in order."""
    main = r"""
    uint64_t state = 1;
    const auto uniform = [&] {   // of [0, 1)
        state = state * 6364136223846793005ull + 1442695040888963407ull;
        return (double)(state >> 11) * 0x1p-53;
    };
    const auto off = [](double got, long double want) { return (double)(fabsl((long double)got - want) / want * 0x1p53L); };
    for (double range : {1e-12, 1e-6, 0.005, 0.0108304, 0.022, 1.0, 40.0, 693.0}) {
        double e = 0, s = 0, t = 0;
        for (int i = 0; i < 200000; ++i) {
            const double x = -range * uniform();
            e = fmax(e, off(exp64(x), expl((long double)x)));
            s = fmax(s, off(sigmoid64(x), expl((long double)x) / (1.0L + expl((long double)x))));
            t = fmax(t, off(sigmoid64(-x), 1.0L / (1.0L + expl((long double)x))));
        }
        printf("%g %g %g %g ", range, e, s, t);
    }
    // next to the table's borders, and fp32 neighbours in order
    double e = 0;
    int wrong = 0;
    for (int i = 0; i < 2000; ++i) {
        const float c = -(float)((i + 0.5) * 0.6931471805599453 / 32);
        float x = c;
        for (int j = 0; j < 50; ++j) x = nextafterf(x, 0.0f);
        double before = exp64(x);
        for (int j = 0; j < 100; ++j) {
            x = nextafterf(x, -1e9f);
            const double v = exp64(x);
            wrong += v > before;
            before = v;
            e = fmax(e, off(v, expl((long double)x)));
        }
    }
    printf("border %g %d %d", e, wrong, exp64(0.0) == 1.0 && exp64(-694.0) == 0.0 && exp64(-INFINITY) == 0.0);
"""
    return run(tmp_path_factory.mktemp("exp"), [("__device__ const double kPowers[32]", "// Orders equal fp64 keys")], main)


def test_exponential_of_near_keys(exponential):
    """exp64: a table entry and the last step round once each (2 of 2^-53 together), the argument's reduction, the series and its end
    are below 2^-7 of that; a score adds its sum's and its quotient's rounding.  The test's own 2^-63 counts little."""
    at = exponential.index("border")
    for r, e, s, t in zip(*[iter(exponential[:at])] * 4):
        assert float(e) <= 2.25, f"exp64 within {r}: {e}"
        assert float(s) <= 4.5 and float(t) <= 4.5, f"sigmoid64 within {r}: {s}, {t}"
    assert float(exponential[at + 1]) <= 2.25
    assert exponential[at + 2:] == ["0", "1"]   # neighbours in order; the ends
