"""Write tm_exp2_poly5.h: the degree-5 fit of 2^f on f in [-1/2, 1/2], by the
method of gen_exp2_poly.py, for sums whose terms need fp32's precision.

    python gen_exp2_poly5.py          # rewrites tm_exp2_poly5.h next to this script
"""
import os

from gen_exp2_poly import NODES, fit

DEGREE = 5


def main():
    c, err = fit(DEGREE)
    here = os.path.dirname(os.path.abspath(__file__))
    lines = [
        "// Generated by gen_exp2_poly5.py; do not edit.",
        "// 2^f ~ c0 + c1 f + ... + c5 f^5 on [-1/2, 1/2]: relative-error least squares on",
        f"// {NODES} Chebyshev nodes; max relative error of the float32 coefficients {err:.3e}.",
        "#pragma once",
    ]
    for i, ci in enumerate(c):
        lines.append(f"#define TM_EXP2_P5_C{i} {float(ci)!r}f")
    with open(os.path.join(here, "tm_exp2_poly5.h"), "w") as fh:
        fh.write("\n".join(lines) + "\n")


if __name__ == "__main__":
    main()
