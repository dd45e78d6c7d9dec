"""Values that are not finite behind weights that underflow to 0: they reach the
rows that see them, and no others, on every route."""
import numpy as np
import pytest
import torch

from step_harness import error_bound, i32, reference
from test_gpu_step import _case

pytestmark = pytest.mark.gpu

SHAPES = [(8, 2, 64, 16, "f32"), (8, 2, 32, 5, "f32"), (8, 2, 64, 16, "bf16"),
          (32, 8, 128, 64, "bf16"), (8, 4, 128, 8, "bf16")]
BATCH = ([70, 0, 5, 130, 9], [200, 3, 1, 40, 1])


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("prefix", [0, 300])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_values_of_weight_zero(rbkv, shape, prefix, value):
    """Scores of -1600 or less and below 100 for all other keys: exp underflows."""
    hq, hkv, D, block, dtype = shape
    starts = np.concatenate([[0], np.cumsum(BATCH[1])])
    pokes = [(0, 0), (0, 130), (1, 1), (3, 25)]              # new tokens, of sequence 0 the first

    def change(q, kn, vn):
        q.copy_(1 + q.abs())
        for s, tok in pokes:
            kn[starts[s] + tok] = -1600 / D ** 0.5
            vn[starts[s] + tok, :, 7] = value

    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, prefix, *BATCH, pad=3, seed=8,
                                                  change=change)
    if prefix:                                               # and one key of the prefix, head 1
        b, off = int(ids[100 // block]), 100 % block
        kc[b, 1, off], vc[b, 1, off, 9] = -1600 / D ** 0.5, value
        kd, vd = kc.cuda(), vc.cuda()
    o = t.attention(q.cuda(), kd, vd, prefix_table=i32(ids) if prefix else None,
                    prefix_len=prefix).cpu()[:rows].double()
    t.device_status()
    hit = torch.zeros(rows, hq, D, dtype=torch.bool)
    for s, tok in pokes:
        hit[starts[s] + tok:starts[s + 1], :, 7] = True
    if prefix:
        g = hq // hkv
        hit[:, g:2 * g, 9] = True
    assert not torch.isfinite(o[hit]).any()
    if value != value:
        assert torch.isnan(o[hit]).all()
    ref = reference(want, q, kc, torch.where(torch.isfinite(vc), vc, torch.zeros((), dtype=vc.dtype)),
                    ids, prefix)
    err = (o - ref[0]).abs()
    assert (err[~hit] <= error_bound(ref, D, dtype)[~hit]).all()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("prefix", [0, 300])
def test_rows_of_scores_minus_infinity(rbkv, shape, prefix):
    """Every key of KV head 1 scores -inf for sequence 1's and 4's rows: they are
    0 there.  For sequence 0's only one of them does: it counts for nothing."""
    hq, hkv, D, block, dtype = shape
    starts = np.concatenate([[0], np.cumsum(BATCH[1])])
    g = hq // hkv

    def change(q, kn, vn):
        for s in (1, 4):                                     # q . k = -inf with dim 3 alone
            q[starts[s]:starts[s + 1], g:2 * g] = 0
            q[starts[s]:starts[s + 1], g:2 * g, 3] = float("inf")
        q[starts[0]:starts[1], g:2 * g, 3] = 1.0
        kn[starts[0] + 20, 1, 3] = float("-inf")

    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, prefix, *BATCH, pad=3, seed=9,
                                                  change=change)
    places = [(ids, p) for p in range(prefix)]
    places += [(want.table[s], p) for s in (1, 4) for p in range(int(want.ctx[s]))]
    for table, p in places:                                  # (sequence 0's q has dim 3 at 1)
        kc[int(table[p // block]), 1, p % block, 3] = -1.0
    o = t.attention(q.cuda(), kc.cuda(), vd, prefix_table=i32(ids) if prefix else None,
                    prefix_len=prefix).cpu()[:rows].double()
    t.device_status()
    empty = torch.zeros(rows, hq, D, dtype=torch.bool)
    for s in (1, 4):
        empty[starts[s]:starts[s + 1], g:2 * g] = True
    # 0 . -1 and inf . -1: the sum is -inf, all others are finite
    assert (o[empty] == 0).all()
    finite_k = torch.nan_to_num(kc.double(), neginf=-1e3)    # (weight exp(-88) or less)
    ref = reference(want, torch.nan_to_num(q.float(), 0, 0, 0), finite_k, vc, ids, prefix)
    err = (o - ref[0]).abs()
    assert (err[~empty] <= error_bound(ref, D, dtype)[~empty]).all()
