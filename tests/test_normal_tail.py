"""The polynomial of GELU's tail as the source has it, against erfc in 64 bits."""
import math
import os
import re

import numpy as np

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "decode_moe_mul_amd", "csrc", "epilogue.hpp")


def test_the_tails_error_is_what_its_comment_says():
    text = open(SOURCE).read()
    start = text.index("// Phi(-|v|)")
    text = text[start:text.index("\n}\n", start)]
    said = float(re.search(r"([\d.]+e-\d+)", text).group(1))
    scale = float(np.float32(re.search(r"fabsf\(v\), ([\d.]+)f", text).group(1)))
    coef = [float(np.float32(c)) for c in re.findall(r"p = (?:fmaf\(p, t, )?(-?[\d.]+)f", text)]
    assert len(coef) == 9 and abs(scale * math.sqrt(2) - 0.4) < 1e-7
    worst = 0.0
    for i in range(0, 26001):
        z = i / 1000
        t = 1 / (1 + scale * math.sqrt(2) * z)
        p = 0.0
        for c in coef:
            p = p * t + c
        want = 0.5 * math.erfc(z)
        if want < 1e-300:
            break
        worst = max(worst, abs(0.5 * p * t * math.exp(-z * z) / want - 1))
    assert 0.9 * said < worst <= said
