"""kv_attention_bf16 over items of many key tiles a CTA whose running maximum
moves: by less than the range P may take (the reference moves one tile later),
by more (the tile is done again), in some rows of a warp and not in others.

Scores.  With scale = ln 2 / 2 a score in powers of two is half of q.k.  The
first two values of D carry it: q has a one at value t % 2 of token t, K holds
whole numbers there, exact in bf16 (levels past 512 come in steps of 4); the other values are small and normal.  A
level lasts `hold` tiles, and a period is
  plateau   every key at the level;
  spike     one key `rise` (in powers of two) above, the others 60 below it;
  low       all keys 60 below the spike;
  low
with the next plateau at the spike's level.  Rows that end within the low
tiles weigh 128 keys of the plateau against one spike of 2^rise: of 10, an
eighth of the result is what the rescale of sums and O left of the plateau.

Tolerance.  Products of the first values are exact; a score's sum of at most D
terms, none above S = the largest |q.k|, is off by at most D 2^-23 S (each
addition rounded or cut at 2^-23 of the partial sum), E = that times scale.
Probabilities are then off by a factor of e^E in numerator and denominator, on
top of what test_gpu_layer_ops.py allows."""
import math

import pytest
import torch

from test_gpu_layer_ops import DEV, HALF_ULP, Cache, attention_64, gen, i32, lib, normal, within  # noqa: F401

pytestmark = pytest.mark.gpu

SCALE = math.log(2) / 2
TILE = 128


def key_levels(g, s, rises, hold, shift):
    """[s] scores in powers of two: periods as above, the tiles of one kind of row `shift` tiles behind the other's."""
    level, out, at = 0.0, [], 0
    tiles = -(-s // TILE) + shift
    while len(out) < tiles:
        rise = rises[at % len(rises)]
        at += 1
        plain = torch.full((TILE,), level)
        low = torch.full((TILE,), level + rise - 60)
        for _ in range(hold):
            out.append(plain)
        for i in range(hold):
            spike = low.clone()
            if i == 0:
                spike[int(torch.randint(0, TILE, (1,), generator=g))] = level + rise
            out.append(spike)
        out += [low] * (2 * hold)
        level += rise
    v = torch.cat(out[shift:tiles])[:s]
    return v - (v.max() // 2)


MAXIMA = {
    # cached, new, Hq, Hkv, D, window, rises, hold
    "chunk-d64-deferred": ([4000], [1024], 16, 8, 64, 0, [10], 1),
    "chunk-d128-deferred": ([4000], [1024], 16, 8, 128, 0, [10, 12], 1),
    "chunk-d96-redone": ([4000], [1024], 16, 8, 96, 0, [96], 1),
    "chunk-d128-both": ([4000], [1024], 16, 8, 128, 0, [10, 100, 30, 10], 1),
    "chunk-d64-both": ([2500, 1300], [700, 333], 32, 8, 64, 0, [10, 100, 10], 1),
    "chunk-d128-window": ([4000], [1024], 16, 8, 128, 1900, [10, 40], 1),
    # one row tile an item: each stream has every other key tile
    "decode-64-d128": ([1500 + 17 * i for i in range(64)], [1] * 64, 16, 8, 128, 0, [10, 12], 2),
    "decode-64-d64": ([1500 + 17 * i for i in range(64)], [1] * 64, 16, 8, 64, 0, [10, 100], 2),
    "decode-24-d96": ([2600 + 55 * i for i in range(24)], [2] * 24, 16, 8, 96, 0, [100, 10], 2),
    "tokens-40-d128": ([2000 + 90 * i for i in range(16)], [40] * 16, 8, 8, 128, 0, [10], 1),
}


def key_tiles(ctx, new, group, window):
    """Key tiles of one kv head: blocks of two row tiles of TILE // group tokens."""
    n, step = 0, 2 * (TILE // group)
    for c, m in zip(ctx, new):
        for i in range(0, m, step):
            lo = max(0, c + i - window + 1) // TILE if window else 0
            n += (c + min(m, i + step) - 1) // TILE - lo + 1
    return n


@pytest.mark.parametrize("name", MAXIMA)
def test_attention_maxima_that_move_in_long_items(lib, name):  # noqa: F811
    ctx, new, Hq, Hkv, D, window, rises, hold = MAXIMA[name]
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    assert key_tiles(ctx, new, Hq // Hkv, window) * Hkv >= 3 * ctas  # every CTA goes through several tiles
    g, host = gen(D + sum(rises)), torch.Generator().manual_seed(len(ctx) + sum(rises))
    seq = [c + n for c, n in zip(ctx, new)]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    c = Cache(g, seq, Hkv, D, 16, std=0.25)
    for r, s in enumerate(seq):
        for i in range(2):
            levels = key_levels(host, s, rises, hold, 2 * hold * i)
            c.keys[r][..., i] = (2 * levels).to(DEV)[:, None].bfloat16()
            assert torch.equal(c.keys[r][:, 0, i].float().cpu(), 2 * levels)
        j = torch.arange(s, device=DEV)
        c.k[c.table[r].long()[j // 16], :, j % 16] = c.keys[r]
    q = normal(g, cu[-1], Hq, D, dtype=torch.bfloat16, std=0.5)
    q[..., :2] = 0
    t = torch.arange(cu[-1], device=DEV)
    q[t, :, t % 2] = 1
    out, lse = lib.kv_attention_bf16(q, c.k, c.v, c.table, i32(cu), i32(seq), scale=SCALE, window=window, want_lse=True)
    want, z, size = attention_64(q, c.keys, c.values, cu, seq, SCALE, window)
    largest = max(k[..., :2].abs().max().item() for k in c.keys) + 0.125 * D * 16  # |normal| about 4 on either side at most
    off = D * 2.0 ** -23 * largest * SCALE
    within(out, want, HALF_ULP * want.abs() + (HALF_ULP + 2 * off) * size, "out")
    within(lse, z, 2.0 ** -15 + off + 2.0 ** -19 * z.abs(), "lse")
