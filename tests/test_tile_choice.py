"""The products' choice of a tile, read from the sources: every tile that is compiled is
the rule's choice at some size."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "decode_moe_mul_amd", "csrc")
UNITS = 256
LISTS = [("mx4gemm.hip", False), ("mx8linear.hip", False), ("mx4glu.hip", True),
         ("mx8glu.hip", True), ("q8linear.hip", False), ("q8linear.hip", True)]
CHOICE = re.compile(r"choice<\w+<(\d), (\d), (\d), (\d), (\d)>, \w+>\((\d), ([\d.]+)f"
                    r"(?:, ([\d.]+)f)?\)")


def _choices(name, pair):
    """(rows, columns, tiles to a unit, us of a round, us of one tile to a unit)."""
    text = re.sub(r"\s*\n\s*", " ", open(os.path.join(CSRC, name)).read())
    text = text[text.index(" choices[] = {"):]
    text = text[:text.index("};")]
    got = []
    for m in CHOICE.finditer(text):
        wr, wc, tm, tn, _, slots = (int(v) for v in m.groups()[:6])
        us = float(m.group(7))
        got.append((32 * wr * tm, 32 * wc * tn // (2 if pair else 1), slots, us,
                    float(m.group(8) or us)))
    assert len(got) == text.count("choice<")
    return got


def _rounds(choice, R, N):
    rows, cols, slots, us, alone = choice
    whole, last = divmod(-(-R // rows) * -(-N // cols), slots * UNITS)
    return us * whole + (0 if last == 0 else alone if last <= UNITS else us)


@pytest.mark.parametrize("name,pair", LISTS)
def test_every_tile_is_the_choice_somewhere(name, pair):
    choices = _choices(name, pair)
    rows = [17, 33, 64, 100, 150, 200, 260, 333, 400, 512, 700, 1000, 1024, 1500, 2048, 4096]
    cols = [32 * n for n in range(1, 48)] + [2048, 2624, 3904, 4096, 7168, 8192, 14336, 28672]
    won = set()
    for R in rows:
        for N in cols:
            times = [_rounds(c, R, N) for c in choices]
            won.add(times.index(min(times)))
    assert won == set(range(len(choices)))


def test_the_sums_over_long_k_are_tested_with_every_tile():
    pytest.importorskip("torch")
    from test_gpu_block_long import TILES
    files = {"mxfp4": ("mx4gemm.hip", "mx4glu.hip"), "mxfp8": ("mx8linear.hip", "mx8glu.hip"),
             "q8": ("q8linear.hip", "q8linear.hip")}
    for (fmt, pair), sizes in TILES.items():
        choices = _choices(files[fmt][pair], pair)
        assert len(sizes) == len(choices)
        for i, (_, R, N) in enumerate(sizes):
            times = [_rounds(c, R, N) for c in choices]
            assert times.index(min(times)) == i
