"""Attention over the 8-bit key/value cache by every kernel that a plan can name: each call is made
so that its plan has the wanted kernel and split, which is checked, with tokens and rows of its
own (idle sequences and absent blocks bring it there).  Error bounds: test_gpu_kv.py."""
import numpy as np
import pytest

from test_gpu_kv import Pair, msq, scattered  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def steered(msq, p, heads, table, lens, counts, want, causal, window):
    """table, lens and counts with idle sequences and absent blocks added, so that the plan has
    (tile rows, wavefronts, join) as wanted; the largest number of parts that it may have."""
    P, own = p.gpu.block_tokens, len(table[0])
    for more in (0, 10, 30, 60, 100, 200, 255, 300):
        for width in (own, 2 * own, 4 * own, 64, 256, 1024, 4096):
            if width < own or (more + len(lens)) * width > 4_000_000:
                continue
            plan = msq.kv_attention_plan(p.gpu, sum(counts), heads, len(lens) + more, width, max(counts),
                                         causal=causal, window=window)
            if (plan["tile_rows"], plan["wavefronts"], plan["join"]) == want:
                table = np.concatenate([table, np.full((len(lens), width - own), -1)], 1)
                table = np.concatenate([table, np.full((more, width), -1)])
                return table, list(lens) + [0] * more, list(counts) + [0] * more
    pytest.fail(f"no plan with {want}")


ONE, MORE = "none", "launch"
FEW = [(D, 16, 4, join, H, G, lens, counts, way)
       for D in (64, 128, 256)
       for join, H, G, lens, counts in ((ONE, 2, 3, [300, 33, 0], [5, 1, 2]), ("inside", 1, 4, [3000, 100], [1, 1]),
                                        (MORE, 1, 8, [9000, 100], [4, 2]))
       for way in ((True, 0), (True, 1800), (False, 0))
       if not (join == MORE and way[1])]
SHORT, LONG, WIDE = [1500, 700, 33], [5000], [1500, 700]
MANY = [(64, 4, ONE, 1, 4, SHORT, [70, 64, 33], [(True, 0), (True, 900), (False, 0)]),
        (64, 4, MORE, 1, 4, SHORT, [70, 64, 33], [(True, 0), (True, 3500), (False, 0)]),
        (64, 8, ONE, 1, 4, WIDE, [512, 300], [(True, 0), (True, 900), (False, 0)]),
        (64, 8, MORE, 2, 4, LONG, [150], [(True, 0), (False, 0)]),
        (128, 4, ONE, 1, 4, SHORT, [70, 64, 33], [(True, 900)]),
        (128, 4, ONE, 2, 4, [600, 300], [150, 290], [(True, 0), (True, 200), (False, 0)]),
        (128, 4, MORE, 1, 4, SHORT, [70, 64, 33], [(True, 900)]),
        (128, 8, ONE, 1, 4, SHORT, [70, 64, 33], [(True, 0), (True, 3500), (False, 0)]),
        (128, 8, ONE, 2, 4, LONG, [150], [(True, 900)]),
        (128, 8, MORE, 2, 4, LONG, [150], [(True, 0), (True, 3500), (False, 0)]),
        (256, 4, ONE, 1, 4, SHORT, [70, 64, 33], [(True, 0), (True, 900), (False, 0)]),
        (256, 4, MORE, 1, 4, SHORT, [70, 64, 33], [(True, 0), (True, 900), (False, 0)])]
CASES = FEW + [(D, 32 * W, W, *rest, way) for D, W, *rest, ways in MANY for way in ways]


@pytest.mark.parametrize("D,tile,waves,join,H,G,lens,counts,way", CASES)
def test_every_kernel(msq, D, tile, waves, join, H, G, lens, counts, way):
    causal, window = way
    print(f"D={D} rows={tile} {join} lens={lens} counts={counts} causal={causal} window={window}", flush=True)
    rng = np.random.default_rng(D + window)
    table, blocks = scattered(rng, lens, 64)
    p = Pair(msq, blocks, H, D, 64, seed=40, fill=float("nan"))
    p.write(table, [0] * len(lens), lens)
    q = rng.normal(size=(sum(counts), H * G, D)) * 1.5
    call = steered(msq, p, H * G, table, lens, counts, (tile, waves, join), causal, window)
    p.attend(q, *call, causal=causal, window=window)
    p.attend(q, *call, causal=causal, window=window, dtype=torch.float32, out=torch.bfloat16)
    p.attend(q, *call, causal=causal, window=window, dtype=torch.float32)
