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
