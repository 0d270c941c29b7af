"""Outputs of the decayed attention over strided views: what shares memory with an input or another
output is refused whatever the strides and however many sequences there are, before any CUDA
call (no pointer here is read), and the decision (csrc/overlap.h) is the one that counting
every byte gives, in microseconds."""
import ctypes
import os
import random
import subprocess
import time

import pytest

BAD = 1
F, FAR = 1 << 24, 1 << 34       # aligned, never dereferenced; between buffers


def at(i):
    return F + i * FAR


@pytest.fixture(scope="module")
def la():
    import linear_attention_elu_gb300 as m
    return m


def forward(la, B, H, N, D, st, o, dt=1):
    """q, k and v of strides st far from one another, o of the same strides at `o`."""
    return la._lib.la_decay_attn_fwd(at(0), at(1), at(2), at(3), 1.0, None, None, None, o, (ctypes.c_int64 * 12)(*(st * 4)),
                                     B, H, N, D, D, dt, at(8), 1 << 33, None)


def backward(la, B, H, N, D, st, dq, dk, dv):
    return la._lib.la_decay_attn_bwd(at(0), at(1), at(2), at(3), at(4), 1.0, None, dq, dk, dv,
                                     (ctypes.c_int64 * 21)(*(st * 7)), B, H, N, D, D, 1, at(9), 1 << 33, None)


def layouts(B, H, N, D):
    """Heads of a cache that holds more; q, k and v side by side in every head; half the sequences of a token."""
    return [((2 * H + 1) * (N + 5) * D, (N + 5) * D, D), (N * H * 3 * D, 3 * D, H * 3 * D), (D, (N + 1) * 2 * B * D, 2 * B * D)]


@pytest.mark.parametrize("B", [2, 256, 257, 4000])
@pytest.mark.parametrize("i", [0, 1, 2])
def test_strided_views_are_refused_for_any_number_of_sequences(la, B, i):
    H, N, D = 3, 60, 64
    st = layouts(B, H, N, D)[i]
    row = 2 * D
    for t in range(3):
        assert forward(la, B, H, N, D, st, at(t)) == BAD
        assert forward(la, B, H, N, D, st, at(t) + row // 2) == BAD
        assert forward(la, B, H, N, D, st, at(t) - row // 2) == BAD
        # The last rows of one on the first of the other.
        last = 2 * ((B - 1) * st[0] + (H - 1) * st[1] + (N - 1) * st[2])
        assert forward(la, B, H, N, D, st, at(t) + last) == BAD
        assert forward(la, B, H, N, D, st, at(t) - last) == BAD
    assert backward(la, B, H, N, D, st, at(6), at(6), at(8)) == BAD
    assert backward(la, B, H, N, D, st, at(6), at(7), at(6) + row // 2) == BAD
    assert backward(la, B, H, N, D, st, at(6), at(7), at(7) + last) == BAD
    assert backward(la, B, H, N, D, st, at(6), at(3), at(7)) == BAD


@pytest.fixture(scope="module")
def decide(tmp_path_factory):
    """csrc/overlap.h by itself."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    d = tmp_path_factory.mktemp("overlap")
    (d / "o.cpp").write_text("""#include "overlap.h"
extern "C" int decide(const int64_t* a, const int64_t* b) {
    auto rows = [](const int64_t* v) {
        return la::Rows3{reinterpret_cast<const void*>(v[0]), v[1], {v[2], v[3], v[4]}, {v[5], v[6], v[7]}};
    };
    return la::overlap(rows(a), rows(b));
}
""")
    lib = str(d / "o.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I",
                    os.path.join(root, "linear_attention_elu_gb300", "csrc"), str(d / "o.cpp"), "-o", lib], check=True)
    f = ctypes.CDLL(lib).decide
    return lambda *rows: bool(f(*((ctypes.c_int64 * 8)(*r) for r in rows)))


def covered(p, row, n0, n1, n2, s0, s1, s2):
    return {p + a * s0 + b * s1 + c * s2 + e for a in range(n0) for b in range(n1) for c in range(n2) for e in range(row)}


def test_the_decision_is_that_of_every_byte(decide):
    rng = random.Random(3)
    seen = [0, 0]
    for i in range(6000):
        row, n = rng.randint(1, 4), [rng.randint(1, 5) for _ in range(3)]
        nested = [0] * 3
        reach = row
        for k in rng.sample(range(3), 3):                       # a tensor's view
            nested[k] = reach + rng.choice([0, 0, 1, 3])
            reach += (n[k] - 1) * nested[k]
        any_strides = lambda: [rng.randint(-20, 40) for _ in range(3)]  # noqa: E731
        x = [1000, row, *n, *(nested if i % 4 else any_strides())]
        y = [1000 + rng.randint(-reach, reach), rng.randint(1, 4), *(n if i % 2 else [rng.randint(1, 5) for _ in range(3)]),
             *(nested if i % 4 in (1, 2) else any_strides())]
        want = not covered(*x).isdisjoint(covered(*y))
        assert decide(x, y) == want and decide(y, x) == want, (x, y)
        seen[want] += 1
    assert min(seen) > 1000


@pytest.mark.parametrize("B,H,N,D", [(256, 8, 60, 64), (65535, 1, 4, 64), (8, 32, 65536, 128)])
def test_views_between_one_another_are_told_apart_at_once(decide, B, H, N, D):
    row = 2 * D
    rows = lambda p, s: [p, row, B, H, N, *(2 * t for t in s)]  # noqa: E731
    apart = {0: 2 * H * (N + 5) * D, 1: row, 2: 2 * B * D}     # the next heads, columns, sequences
    for i, st in enumerate(layouts(B, H, N, D)):
        x, y = rows(at(0), st), rows(at(0) + apart[i], st)
        took = []
        for _ in range(20):
            t = time.perf_counter()
            assert not decide(x, y)
            took.append(time.perf_counter() - t)
        assert min(took) < 1e-4
        assert decide(x, rows(at(0) + 1, st))
