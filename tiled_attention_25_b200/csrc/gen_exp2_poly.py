"""Generate exp2_poly.h: a minimax polynomial for 2^f on [-1/2, 1/2].

The forward kernel evaluates part of its exponentials on the FMA pipe
instead of the special-function unit: 2^x = 2^n * 2^f with n = round(x),
f = x - n (Cody and Waite's additive range reduction), and 2^f from a
polynomial whose coefficients minimise the maximum RELATIVE error on
[-1/2, 1/2] (Remez exchange algorithm).  The probabilities are rounded to
bfloat16 (relative step 2^-8) right after, so degree 3 (relative error below
8e-5) leaves the polynomial far under that rounding, and each evaluation one
FMA shorter than degree 4 (below 3e-6).

Run:  python tiled_attention_25_b200/csrc/gen_exp2_poly.py  (rewrites exp2_poly.h)
"""
import os

import numpy as np

DEGREE = 3
LO, HI = -0.5, 0.5


def remez_relative(deg, lo, hi, iters=30):
    f = lambda x: np.exp2(x)
    n = deg + 2
    # Chebyshev extrema as the initial reference
    k = np.arange(n)
    x = (lo + hi) / 2 + (hi - lo) / 2 * np.cos(np.pi * k[::-1] / (n - 1))
    grid = np.linspace(lo, hi, 200001)
    for _ in range(iters):
        # solve sum_j c_j x_i^j + (-1)^i E f(x_i) = f(x_i)  (relative equi-oscillation)
        A = np.zeros((n, n))
        for i in range(n):
            A[i, :deg + 1] = x[i] ** np.arange(deg + 1)
            A[i, deg + 1] = (-1) ** i * f(x[i])
        sol = np.linalg.solve(A, f(x))
        c = sol[:deg + 1]
        err = (np.polyval(c[::-1], grid) - f(grid)) / f(grid)
        # new reference: extrema of the error on each sign-alternating segment
        sign = np.sign(err)
        idx = [0] + list(np.nonzero(np.diff(sign))[0] + 1) + [len(grid)]
        ext = []
        for a, b in zip(idx[:-1], idx[1:]):
            seg = np.abs(err[a:b])
            ext.append(a + int(np.argmax(seg)))
        if len(ext) != n:
            break
        x = grid[ext]
    err = (np.polyval(c[::-1], grid) - f(grid)) / f(grid)
    return c, float(np.max(np.abs(err)))


def main():
    c, e = remez_relative(DEGREE, LO, HI)
    c32 = c.astype(np.float32)
    grid = np.linspace(LO, HI, 200001)
    e32 = float(np.max(np.abs((np.polyval(c32.astype(np.float64)[::-1], grid) - np.exp2(grid)) / np.exp2(grid))))
    lines = [
        "// Generated by gen_exp2_poly.py: minimax (relative error) polynomial for 2^f,",
        f"// f in [{LO}, {HI}], degree {DEGREE}; max relative error {e:.3e} (float64",
        f"// coefficients), {e32:.3e} with the float32 coefficients below.",
        "#pragma once",
        "",
        "namespace attn25 {",
        "",
    ]
    for i, v in enumerate(c32):
        lines.append(f"constexpr float kExp2C{i} = {float(v)!r}f;")
    lines += ["", "}  // namespace attn25", ""]
    out = os.path.join(os.path.dirname(os.path.abspath(__file__)), "exp2_poly.h")
    with open(out, "w") as fh:
        fh.write("\n".join(lines))
    print(out, e, e32)


if __name__ == "__main__":
    main()
