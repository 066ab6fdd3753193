"""mk_tree_attention with infinite and NaN values among the drafts: they reach the nodes that see
them and nobody else, wherever in a block's tiles they lie."""
import numpy as np
import pytest
import torch

import persistent_megakernel_decode_04_b200 as mk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
BF, HF = torch.bfloat16, torch.float16


def attend(q, k, v, parents, lens, scale=0.125, o=None):
    o = torch.zeros_like(q) if o is None else o
    mk.mk_tree_attention(q, k, v, o, parents, None, lens, scale)
    return o


def make(B, n, hq, hkv, d, S, dtype, q_dtype=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(B, n, hq, d, generator=g).to(q_dtype or dtype).to(DEV)
    k, v = (torch.randn(B, hkv, S, d, generator=g).to(dtype).to(DEV) for _ in range(2))
    return q, k, v


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,wide", [(BF, False), (HF, False), (BF, True)])
@pytest.mark.parametrize("B,n,hq,hkv,lens", [
    (40, 256, 4, 2, [0, 10, 61]),   # more units than the device runs at once: one block takes all the tiles
    (2, 130, 4, 2, [0, 10]),
    (1, 256, 2, 2, [37]),
    (3, 100, 8, 1, [0, 63, 1]),
])
def test_in_every_tile_and_every_group_of_keys(d, dtype, wide, B, n, hq, hkv, lens):
    """Every fourth node is a leaf with infinities and NaN, so that each group of four keys of each
    tile with drafts has some; all other nodes hang on nodes without.  Where nobody sees them the
    bits are those of the same call with zeros in their place."""
    lens = (lens * B)[:B]
    S = -(-(max(lens) + n) // 64) * 64
    q, k, v = make(B, n, hq, hkv, d, S, dtype, torch.float32 if wide else None, seed=n + d)
    leaf = np.arange(n) % 4 == 3
    parents = np.zeros(n, dtype=np.int32)
    rng = np.random.default_rng(n)
    for i in range(1, n):
        near = [x for x in range(max(0, i - 9), i) if not leaf[x]]
        parents[i] = int(rng.choice(near))
    parents[0] = -1
    parents = torch.from_numpy(np.tile(parents, (B, 1))).to(DEV)
    zeros, bad = v.clone(), v.clone()
    col = torch.arange(d, device=DEV)
    kind = [float("inf"), float("-inf"), float("nan")]
    marked = torch.zeros(B, n, d, dtype=torch.bool, device=DEV)  # values of nodes that are not finite
    for b in range(B):
        for x in np.nonzero(leaf)[0].tolist():
            at = (col % 5) == x % 5
            zeros[b, :, lens[b] + x, at] = 0.0
            bad[b, :, lens[b] + x, at] = kind[x // 4 % 3]
            marked[b, x] = at
    t = torch.tensor(lens, dtype=torch.int32, device=DEV)
    want = attend(q, k, zeros, parents, t)
    assert want.isfinite().all()
    seen = marked[:, :, None].expand(B, n, hq, d)
    value = torch.tensor([kind[x // 4 % 3] for x in range(n)], device=DEV)[None, :, None, None].expand(B, n, hq, d)
    for _ in range(20):  # which warp comes first is a matter of timing
        got = attend(q, k, bad, parents, t)
        assert torch.equal(got[~seen], want[~seen])
        g, w = got[seen].float(), value[seen]
        assert torch.equal(g.isnan(), w.isnan()) and torch.equal(g.nan_to_num(0, 1, -1), w.nan_to_num(0, 1, -1))
    assert mk.mk_tree_attention_status() == mk.MK_OK


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("B,S", [(1, 640), (2, 4096), (300, 200)])  # clusters of several sizes, single blocks
def test_scores_of_minus_infinity(B, S, d, dtype):
    """A key of -infinity has no weight; a node that sees no others is 0 / 0."""
    n, hq, hkv, ln = 4, 4, 2, 150
    q, k, v = make(B, n, hq, hkv, d, S, dtype, seed=d)
    q[..., 0] = 1.0
    k[:, 0, :ln + 1, 0] = float("-inf")  # of the first KV head: all cached rows and node 0
    parents = torch.tensor([[-1, 0, 1, 0]] * B, dtype=torch.int32, device=DEV)
    parents[:, 3] = 7                    # not a tree's
    lens = torch.full((B,), ln, dtype=torch.int32, device=DEV)
    got = attend(q, k, v, parents, lens)
    assert mk.mk_tree_attention_status() == mk.MK_OK
    assert got[:, 0, :2].isnan().all()
    assert torch.equal(got[:, 1, :2], v[:, 0, ln + 1][:, None].expand(B, 2, d))  # itself alone
    two = k[:, 0, ln + 1:ln + 3].double()
    p = torch.softmax(torch.einsum("bhd,brd->bhr", q[:, 2, :2].double(), two) * 0.125, -1)
    want = torch.einsum("bhr,brd->bhd", p, v[:, 0, ln + 1:ln + 3].double())
    # output and weights rounded to half an eps each, of |v| below 8; fp32 steps below 2^-12
    assert ((got[:, 2, :2].double() - want).abs() <= 8 * (torch.finfo(dtype).eps + 2.0 ** -12)).all()
    assert (got[:, 3] == 0).all()
    assert got[:, :3, 2:].isfinite().all()
