"""Which tile csrc/i8_gemm.hip takes for a product, from the tiles and the costs that stand there.

The tiles (`using I8Few = I8Tile<...>`) and their costs (`chunk_ns<I8Few>(n, E, units, 45, 68)`) are
read from the source, so that a change of either moves what these tests select too.
"""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "mxfp4_mixture_experts_route_amd", "csrc", "i8_gemm.hip")
FEW_ROWS, FEW_VALUES = 8, 24 * 1024     # i8_linear: rows and values of the one-launch kernel


def tiles():
    """[(name, rows, channels, ns of one round, ns of each of several: dense, routed)], in order."""
    text = open(SOURCE).read()
    size = {m[0]: (int(m[1]), int(m[2])) for m in
            re.findall(r"using (I8\w+) = I8(?:Tile|Direct)<(\d+), (\d+)[^>]*>;", text)}
    out = []
    for name, one, each in re.findall(
            r"chunk_ns<(I8\w+)>\(n, E, units, (\d+), ([^()]+?)\)", text):
        routed, dense = re.fullmatch(r"counts \? (\d+) : (\d+)|(\d+)", each).group(1, 2)
        if routed is None:
            routed = dense = each
        out.append((name, *size[name], int(one), int(dense), int(routed)))
    assert [t[0] for t in out] == list(size), "every tile has a cost"
    return out


def tile_of(rows, N, experts=0, glu=False):
    """The tile of a dense product of `rows` rows, or of a routed one with `rows` = mpad."""
    E, n = (experts, -(-rows // experts)) if experts else (1, rows)
    units = 2 * -(-(N // 2) // 16) if glu else -(-N // 16)
    best = None
    for name, bm, bn, one, dense, routed in tiles():
        if experts and name == "I8Big":
            continue
        count = E * -(-n // bm) * -(-units // (bn // 16))
        rounds = -(-count // 256)
        ns = one if rounds == 1 else rounds * (routed if experts else dense)
        if best is None or ns < best[0]:
            best = (ns, name)
    return best[1]
