"""kv_attention_bf16 where its values are unusual: scores of NaN and
infinity.  Bounds, the 64-bit reference and the cache are those of
test_gpu_layer_ops.py."""
import math

import pytest
import torch

from test_gpu_layer_ops import DEV, Cache, check_attention, gen, i32, lib, normal  # noqa: F401

pytestmark = pytest.mark.gpu


# ---- kv_attention_bf16: scores of NaN and infinity ---------------------------------

def softmax_rows(q, keys, values, cu, seq, scale, window):
    """out, lse and sum_j p_j |v_j| by the definition, NaN and infinities included; rows without a key give zeros and
    -inf."""
    T, Hq, D = q.shape
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=DEV)
    size = torch.zeros_like(out)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=DEV)
    for r, s in enumerate(seq):
        a, b = cu[r], cu[r + 1]
        if s <= 0:
            continue
        k, v = (x[r].double().repeat_interleave(Hq // x[r].shape[1], 1) for x in (keys, values))
        p, j = s - (b - a) + torch.arange(b - a, device=DEV)[:, None], torch.arange(s, device=DEV)
        seen = (j <= p) & (j > p - (window or s + b))
        score = torch.einsum("thd,jhd->htj", q[a:b].double(), k) * scale
        score = score.masked_fill(~seen, -math.inf)
        some = seen.any(-1)
        w = torch.softmax(score[:, some], -1)
        out[a:b][some] = torch.einsum("htj,jhd->thd", w, v)
        size[a:b][some] = torch.einsum("htj,jhd->thd", w, v.abs())
        lse[a:b][some] = torch.logsumexp(score[:, some], -1).t()
    return out, lse, size


UNUSUAL = {
    # cached tokens, new tokens, Hq, Hkv, D, window
    "whole-items": ([200, 90], [1, 1], 8, 2, 128, 0),                 # one row tile, not split
    "split-few-rows": ([2000, 1500], [1, 2], 8, 2, 128, 0),           # joined a warp per row
    "split-many-rows": ([900, 300], [40, 25], 8, 2, 64, 0),           # joined a lane per row
    "two-row-tiles": ([0] * 80, [140] * 80, 2, 2, 64, 0),             # an item or two a CTA
    "windowed": ([700, 20], [60, 180], 4, 2, 96, 130),
    "rows-without-keys": ([-5, -200, 300], [9, 280, 1], 4, 2, 128, 0),
}


@pytest.mark.parametrize("what", ["nan-query", "nan-key", "inf-key", "all-minus-inf"])
@pytest.mark.parametrize("name", UNUSUAL)
def test_attention_passes_nan_and_infinity_on(lib, name, what):  # noqa: F811
    """A NaN or +inf among the scores that a row sees makes the row NaN, as do scores that are all -inf; a score of
    -inf beside others has weight zero; other rows are as without them."""
    ctx, new, Hq, Hkv, D, window = UNUSUAL[name]
    g = gen(len(name) + len(what))
    seq = [c + n for c, n in zip(ctx, new)]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    c = Cache(g, seq, Hkv, D, 16)
    q = normal(g, cu[-1], Hq, D, dtype=torch.bfloat16)
    for r in range(0, len(seq), 2):
        key = max(0, seq[r] - max(1, new[r] // 2))  # half of the new tokens see it
        if what == "nan-query":
            q[cu[r], 1, D - 1] = math.nan
            q[cu[r + 1] - 1, Hq - 1, 0] = math.nan
        elif seq[r] > 0:
            if what == "nan-key":
                c.keys[r][key, 0, 3] = math.nan
            elif what == "inf-key":
                c.keys[r][key, 0, 3] = math.inf
                q[cu[r]:cu[r + 1], 0, 3] = 1.0
            else:
                c.keys[r][:, 0, 3] = math.inf
                q[cu[r]:cu[r + 1], 0, 3] = -1.0
            j = torch.arange(seq[r], device=DEV)
            c.k[c.table[r].long()[j // 16], :, j % 16] = c.keys[r]
    out, lse = lib.kv_attention_bf16(q, c.k, c.v, c.table, i32(cu), i32(seq), window=window, want_lse=True)
    want, z, size = softmax_rows(q, c.keys, c.values, cu, seq, D ** -0.5, window)
    bad = torch.isnan(want).any(-1)
    assert bad.any() and not bad.all()
    assert torch.isnan(out[bad]).all()
    none = bad & (z == -math.inf)
    assert what != "all-minus-inf" or none.any()
    assert (lse[none] == -math.inf).all() and torch.isnan(lse[bad & ~none]).all()
    check_attention(out[~bad], lse[~bad], (want[~bad], z[~bad], size[~bad]))
