"""Whether strided tensors share memory (csrc/strided.h), against a byte map; a small program of the host."""
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include "strided.h"
int main() {
    long long a[6], b[6];
    while (std::scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld", a, a + 1, a + 2, a + 3, a + 4, a + 5, b, b + 1, b + 2,
                      b + 3, b + 4, b + 5) == 12) {
        const kv::Strided x = {reinterpret_cast<void *>(a[0]), a[1], a[2], a[3], a[4], a[5]};
        const kv::Strided y = {reinterpret_cast<void *>(b[0]), b[1], b[2], b[3], b[4], b[5]};
        std::printf("%d %d\n", kv::meet(x, y), kv::folds(x));
    }
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    d = tmp_path_factory.mktemp("strided")
    (d / "ask.cc").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-I",
                    os.path.join(ROOT, "q8_matrix_vector_gb300", "csrc"), str(d / "ask.cc"), "-o", str(d / "ask")], check=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, (*a, *b))) for a, b in cases)
        out = subprocess.run([str(d / "ask")], input=text, check=True, capture_output=True, text=True).stdout.split()
        return [(bool(int(m)), bool(int(f))) for m, f in zip(out[0::2], out[1::2])]

    return run


def cells(t):
    at, rows, row, heads, head, size = t
    return [at + r * row + h * head + i for r in range(rows) for h in range(heads) for i in range(size)]


def test_against_a_map_of_bytes(ask):
    rng = random.Random(0)
    cases = []
    for _ in range(20000):
        row, size = rng.choice([0, *range(1, 40)]), rng.randint(1, 6)
        heads = (rng.randint(1, 4), rng.choice([0, *range(1, 12)]))
        a = (10000 + rng.randint(0, 60), rng.randint(1, 5), row, *heads, size)
        other = rng.choice([row, row, row, 0, rng.randint(1, 40)])
        b = (10000 + rng.randint(0, 60), rng.randint(1, 5), other, rng.randint(1, 4), rng.choice([heads[1], rng.randint(0, 12)]), rng.randint(1, 6))
        cases.append((a, b))
    told = 0
    for (a, b), (met, folds) in zip(cases, ask(cases)):
        x, y = cells(a), cells(b)
        share = not set(x).isdisjoint(y)
        differ = a[2] != b[2] and a[2] and b[2] and a[1] > 1 and b[1] > 1
        if differ:  # refused where the stretches meet
            assert met or not share
            assert met or max(x) < min(y) or max(y) < min(x)
        else:
            told += 1
            assert met == share, (a, b)
        assert folds == (len(set(x)) < len(x)), a
    assert told > 10000


def test_parts_of_one_tensor_are_apart_however_long(ask):
    """q, k and v of [n, 32 + 8 + 8 heads, 128] f16, of [n, heads, 3, 128], and with more rows than bytes can be listed."""
    n, d = 2 ** 31 - 1, 256
    row = 48 * d
    q, k, v = (4096, n, row, 32, d, d), (4096 + 32 * d, n, row, 8, d, d), (4096 + 40 * d, n, row, 8, d, d)
    assert ask([(q, k), (q, v), (k, q), (q, q)]) == [(False, False)] * 3 + [(True, False)]
    parts = [(4096 + i * d, 1000, 8 * 3 * d, 8, 3 * d, d) for i in range(3)]
    assert ask([(parts[0], parts[1]), (parts[2], parts[1])]) == [(False, False)] * 2
    # a view of k's heads one further, a row behind, and one element into the next part
    assert ask([((4096 + 33 * d, n, row, 8, d, d), k), ((4096 + row + 32 * d, 5, row, 8, d, d), k),
                ((4096 + 2, n, row, 32, d, d), k)]) == [(True, False)] * 3
    # strides up to the largest that are taken
    far = 2 ** 42
    assert ask([((4096, n, far, 65535, 2 ** 40, 2 ** 18), (4096, 1, 0, 1, 0, 8)),
                ((4096 + 2 ** 18, n, far, 2, 2 ** 40, 2 ** 18), (4096, n, far, 2, 2 ** 40, 2 ** 18))]) == [(True, True), (False, False)]
