"""How 4-bit products and input gradients are computed (test helper): the plan of
their tiles from the source's own tables, in its fp32 arithmetic."""
import os
import re
from dataclasses import dataclass

import numpy as np

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_weight_mixture_02_amd", "csrc")
F = np.float32


def _table(src, name):
    """(bn, bm, res, lat, thr, c) of each tile; the three as [bf16 results, fp32 results]."""
    body = re.search(name + r"\[\] = \{\n(.*?)\n\};", src, re.S)[1]
    out = []
    for line in re.findall(r"\{(\d+), (\d+), (\d+), \{(.*?)\}, \{(.*?)\}, \{(.*?)\}\}", body):
        out.append((*map(int, line[:3]), *[[F(v.strip().rstrip("f")) for v in g.split(",")] for g in line[3:]]))
    return out


def _source():
    src = open(os.path.join(CSRC, "fp4.hip")).read()
    stages = []
    for fp4 in (True, False):
        each = []
        for n in re.findall(r"gemm<Fp4Tile<\d, \d, \d, \d, (.*?), FP4>>", src):
            m = re.match(r"FP4 \? (\d) : (\d)", n)
            each.append(int(m[1 if fp4 else 2]) if m else int(n))
        stages.append(each)
    tables = _table(src, "FP4_SHAPE"), _table(src, "BF16_SHAPE")
    assert [len(t) for t in (*tables, *stages)] == [9] * 4
    return tables, stages


TABLES, STAGES = _source()   # of 4-bit products, of bf16 ones


@dataclass
class Plan:
    tile: int
    bn: int
    bm: int
    whole: int      # tiles that are computed whole, and
    rest: int       # in parts of K
    splits: int
    several: bool   # workgroups take several whole tiles, one after the other
    us: float


def plan(M, N, K, f32, fp4):
    """Of a result M x N summed over K (a whole number of 64 if not fp4).  None:
    the kernel for up to 16 rows."""
    if fp4 and M <= 16 and N >= 1024:
        return None
    f32 = int(f32)
    kb = -(-K // 256) if fp4 else K // 64
    table, stages = TABLES[0 if fp4 else 1], STAGES[0 if fp4 else 1]
    best = least = None
    for i, (bn, bm, res, lat, thr, c) in enumerate(table):
        tiles = -(-N // bn) * -(-M // bm)

        def launch(groups, blocks):
            if groups == 0:
                return F(0)
            w = -(-groups // 256)
            block = thr[f32] * F(w) if w > 1 and thr[f32] * F(w) > lat[f32] else lat[f32]
            return F(block * F(blocks) + c[f32] * F(-(-w // res)))

        us = launch(tiles, kb)
        if least is None or us < least:
            best, least = (i, tiles, 0, 1), us
        rest = tiles % (256 * res)
        if rest == 0 or rest > 128:
            continue
        s = min(kb // 3, 256 // rest)
        if s < 2:
            continue
        join = F(6 if tiles > rest else 3) + F(s * rest * bn * min(M, bm)) * F(8) / F(4e6)
        split = F(launch(tiles - rest, kb) + launch(rest * s, -(-kb // s)) + join)
        if split < least:
            best, least = (i, tiles - rest, rest, s), split
    i, whole, rest, s = best
    bn, bm = table[i][:2]
    scales = (-(-bm // 128) + -(-bn // 128)) * 1024 if fp4 else 0
    held = 256 * (160 * 1024 // (stages[i] * ((bn + bm) * 128 + scales)))
    return Plan(i, bn, bm, whole, rest, s, bn * bm >= 128 * 128 and whole > held and kb > stages[i], float(least))
