"""mk_tree_attention against its 64-bit definition."""
import numpy as np
import pytest
import torch

import persistent_megakernel_decode_04_b200 as mk
from _speculative import attention_bound, attention_rows, random_tree, wide_bound

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
BF, HF = torch.bfloat16, torch.float16


def make(B, n, hq, hkv, d, S, lens, kind="tree", dtype=BF, seed=0, n_nodes=None, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    q = (torch.randn(B, n, hq, d, generator=g) * spread).to(dtype)
    k, v = (torch.randn(B, hkv, S, d, generator=g).to(dtype) for _ in range(2))
    parents = np.stack([random_tree(rng, n, kind) for _ in range(B)])
    return dict(q=q, k=k, v=v, parents=torch.from_numpy(parents), lens=torch.tensor(lens, dtype=torch.int32),
                n_nodes=None if n_nodes is None else torch.tensor(n_nodes, dtype=torch.int32))


def run(x, scale, o=None, stream=None):
    t = {key: None if val is None else val.to(DEV) for key, val in x.items()}
    if o is None:
        o = torch.full_like(t["q"], 7.0)
    mk.mk_tree_attention(t["q"], t["k"], t["v"], o, t["parents"], t["n_nodes"], t["lens"], scale, stream)
    assert mk.mk_tree_attention_status(stream) == mk.MK_OK
    return o.cpu()


def check(x, scale, got):
    ref, a = attention_rows(x["q"], x["k"], x["v"], x["parents"], x["n_nodes"], x["lens"], scale)
    skip = ref.isnan()
    assert (got[skip] == 7.0).all(), "a row behind the last node was written"
    fin = torch.where(x["v"].double().isfinite(), x["v"].double(), 0.0)
    err = (got.double() - ref).abs()[~skip]
    room = attention_bound(ref, a, fin, x["q"].dtype)[~skip]
    assert (err <= room).all(), (err / room).max()


@pytest.mark.parametrize("B,n,hq,hkv,d,S,lens", [
    (1, 1, 4, 2, 64, 64, [0]),            # one key: the node itself
    (1, 1, 32, 8, 128, 1024, [551]),      # single-token decode form
    (1, 5, 32, 8, 128, 1024, [551]),
    (2, 7, 4, 4, 64, 300, [1, 290]),
    (3, 33, 6, 2, 128, 700, [126, 127, 128]),  # drafts around a tile's end
    (2, 64, 4, 1, 64, 512, [300, 0]),     # two row tiles; an empty cache
    (1, 65, 14, 2, 128, 400, [255]),      # 7 heads per KV head; odd tile counts
    (2, 256, 4, 2, 64, 600, [257, 344]),  # the most nodes; a cache filled to its last row
    (1, 3, 128, 1, 128, 260, [200]),      # 128 heads per KV head: one node per row tile
    (1, 2, 71, 1, 64, 300, [129]),
    (4, 16, 8, 8, 64, 2100, [2000, 3, 1024, 77]),
])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_matches_the_definition(B, n, hq, hkv, d, S, lens, dtype):
    x = make(B, n, hq, hkv, d, S, lens, dtype=dtype, seed=n)
    check(x, d ** -0.5, run(x, d ** -0.5))


@pytest.mark.parametrize("B,n,hq,hkv,d,S,lens", [
    (1, 1, 4, 2, 64, 64, [0]), (2, 7, 32, 8, 128, 1024, [551, 1017]), (3, 33, 6, 2, 128, 700, [126, 127, 128]),
    (2, 65, 14, 2, 64, 900, [255, 830]), (12, 13, 16, 16, 128, 300, [20 * b for b in range(12)]),
])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_fp32_queries_and_outputs_over_a_16_bit_cache(B, n, hq, hkv, d, S, lens, dtype):
    x = make(B, n, hq, hkv, d, S, lens, dtype=dtype, seed=n)
    x["q"] = torch.randn(B, n, hq, d, generator=torch.Generator().manual_seed(n + 1))
    scale = d ** -0.5
    got = run(x, scale)
    ref, a = attention_rows(x["q"], x["k"], x["v"], x["parents"], None, x["lens"], scale)
    err = (got.double() - ref).abs()
    room = wide_bound(ref, a, x["v"], dtype)
    assert (err <= room).all(), (err / room).max()
    narrow = run(dict(x, q=x["q"].to(dtype)), scale).double() - ref  # the same without the low parts
    assert err.square().mean().sqrt().item() <= narrow.square().mean().sqrt().item() / 8  # (one key: 0 and 0)
    # NaN in rows that are not seen, and a negative scale, as in the other form
    y = dict(x, k=x["k"].clone(), v=x["v"].clone())
    for b in range(B):
        y["k"][b, :, lens[b] + n:], y["v"][b, :, lens[b] + n:] = float("nan"), float("inf")
    assert torch.equal(run(y, scale), got)
    assert torch.equal(run(dict(x, q=-x["q"]), -scale), got)


@pytest.mark.parametrize("kind", ["chain", "star", "forest"])
@pytest.mark.parametrize("n", [2, 31, 32, 130])
def test_tree_shapes(kind, n):
    x = make(2, n, 4, 2, 64, 400, [0, 150], kind=kind, seed=n)
    check(x, 0.125, run(x, 0.125))


def test_nodes_in_use_and_lengths_out_of_range():
    # counts above n and below 0, lengths beyond the cache and negative: clamped, nothing else written
    x = make(5, 20, 4, 2, 64, 256, [100, 250, 9999, -5, 7], n_nodes=[13, 20, 20, 99, -3], seed=3)
    check(x, 0.125, run(x, 0.125))


def test_nodes_without_a_tree_get_zeros():
    x = make(1, 12, 4, 2, 64, 256, [140], kind="chain", seed=4)
    x["parents"][0, 4] = 9    # a later node
    x["parents"][0, 8] = -7
    got = run(x, 0.125)
    check(x, 0.125, got)
    assert (got[0, 4:] == 0).all() and (got[0, :4] != 0).any()


@pytest.mark.parametrize("scale", [-0.125, 3.0, 1e-4])
def test_scales(scale):
    x = make(1, 40, 8, 2, 64, 600, [500], seed=5, spread=0.3 if abs(scale) > 1 else 1.0)
    check(x, scale, run(x, scale))


@pytest.mark.parametrize("dtype", [BF, HF])
def test_rows_that_a_node_does_not_see_have_no_influence(dtype):
    # NaN and infinities behind the last node, in other branches and in other sequences
    x = make(2, 40, 8, 2, 128, 512, [200, 380], kind="tree", dtype=dtype, seed=6, n_nodes=[40, 33])
    want = run(x, 0.1)
    y = dict(x, k=x["k"].clone(), v=x["v"].clone())
    y["k"][0, :, 240:], y["v"][0, :, 240:] = float("nan"), float("inf")
    y["k"][1, :, 413:], y["v"][1, :, 413:] = float("inf"), float("nan")
    assert torch.equal(run(y, 0.1), want)
    # a draft with infinite and NaN values: its descendants get them, everyone else is as before
    y["v"][0, 1, 200 + 5, 3], y["v"][0, 1, 200 + 5, 100] = float("-inf"), float("nan")
    got = run(y, 0.1)
    from _speculative import ancestors
    anc = ancestors(x["parents"][0], 40)
    sees = torch.tensor([5 in a for a in anc])
    assert 0 < sees.sum() < 40
    assert torch.equal(got[1], want[1]) and torch.equal(got[0, ~sees], want[0, ~sees])
    assert torch.equal(got[0, :, :4], want[0, :, :4])  # the other KV head
    mine = got[0, sees][:, 4:]
    assert (mine[..., 3] == float("-inf")).all() and mine[..., 100].isnan().all()
    mine[..., 3] = mine[..., 100] = 0
    ref = want[0, sees][:, 4:].clone()
    ref[..., 3] = ref[..., 100] = 0
    assert torch.equal(mine, ref)


def test_infinite_scores_and_values_that_are_seen():
    x = make(1, 4, 2, 2, 64, 256, [150], kind="chain", seed=7)
    x["k"][0, 0, 10] = float("nan")       # committed row: every node of that head is NaN
    x["v"][0, 1, 20, 5] = float("inf")
    got = run(x, 0.125)
    assert got[0, :, 0].isnan().all()
    assert (got[0, :, 1, 5] == float("inf")).all() and got[0, :, 1, 6].isfinite().all()


def test_strided_operands_and_the_decoders_cache_layout():
    B, n, hq, hkv, d, S = 2, 9, 8, 2, 64, 320
    x = make(B, n, hq, hkv, d, S, [77, 300], seed=8)
    cache = torch.zeros(3, 2, B, hkv, S, d, dtype=BF, device=DEV)  # [layer][K|V][B][kv head][row][d]
    cache[1, 0].copy_(x["k"])
    cache[1, 1].copy_(x["v"])
    bits = cache.view(torch.int16)                                 # as Megakernel.kv_view gives it
    qq = torch.zeros(n, hq, B, 2 * d, dtype=BF, device=DEV).permute(2, 0, 1, 3)[..., :d]
    qq.copy_(x["q"])
    o = torch.full((B, hq, n, d + 8), 7.0, dtype=BF, device=DEV).transpose(1, 2)[..., :d]
    mk.mk_tree_attention(qq, bits[1, 0], bits[1, 1], o, x["parents"].to(DEV), None, x["lens"].to(DEV), 0.125)
    check(x, 0.125, o.cpu())
    # keys and values side by side in one row, rows of all heads together
    kv = torch.zeros(B, S, hkv, 2 * d, dtype=BF, device=DEV).transpose(1, 2)
    kv[..., :d], kv[..., d:] = x["k"].to(DEV), x["v"].to(DEV)
    o = torch.full((B, n, hq, d), 7.0, dtype=BF, device=DEV)
    mk.mk_tree_attention(x["q"].to(DEV), kv[..., :d], kv[..., d:], o, x["parents"].to(DEV), None, x["lens"].to(DEV), 0.125)
    check(x, 0.125, o.cpu())


def test_long_cache_beyond_32_bit_offsets():
    # 2 sequences x 4 heads x 2.2 M rows of 128 values: offsets pass 2^31 elements
    B, hkv, S, d, n = 2, 4, 2_200_000, 128, 3
    k = torch.zeros(B, hkv, S, d, dtype=BF, device=DEV)
    v = torch.zeros(B, hkv, S, d, dtype=BF, device=DEV)
    x = make(B, n, hkv, hkv, d, 512, [0, 0], kind="chain", seed=9)
    lens = torch.tensor([400, S - n], dtype=torch.int32)
    x["lens"] = torch.tensor([400, 400], dtype=torch.int32)
    k[0, :, :512], v[0, :, :512] = x["k"][0].to(DEV), x["v"][0].to(DEV)
    # the long sequence: keys of zeros (score 0) and one far row that takes nearly all the weight
    k[1, :, S - n - 5] = 100.0
    v[1, :, S - n - 5] = 3.0
    q = x["q"].to(DEV)
    q[1] = 1.0
    o = torch.full_like(q, 7.0)
    mk.mk_tree_attention(q, k, v, o, x["parents"].to(DEV), None, lens.to(DEV), 0.5)
    assert mk.mk_tree_attention_status() == mk.MK_OK
    assert (o[1] == 3.0).all()
    one = {key: val[:1] if val is not None else None for key, val in x.items()}
    check(one, 0.5, o[:1].cpu())


def test_streams_and_graphs():
    x = make(2, 12, 8, 2, 128, 640, [500, 130], seed=10)
    t = {key: None if val is None else val.to(DEV) for key, val in x.items()}
    outs = [torch.full_like(t["q"], 7.0) for _ in range(3)]
    st = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s, o in zip(st, outs):  # two calls that may overlap
        for _ in range(20):
            mk.mk_tree_attention(t["q"], t["k"], t["v"], o, t["parents"], None, t["lens"], 0.1, s)
    for s in st:
        s.synchronize()
    check(x, 0.1, outs[0].cpu())
    assert torch.equal(outs[0], outs[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mk.mk_tree_attention(t["q"], t["k"], t["v"], outs[2], t["parents"], None, t["lens"], 0.1,
                             torch.cuda.current_stream())
    y = make(2, 12, 8, 2, 128, 640, [3, 600], seed=11)
    for key in ("q", "k", "v", "parents", "lens"):
        t[key].copy_(y[key])
    graph.replay()
    check(y, 0.1, outs[2].cpu())


def test_a_wait_that_runs_out_is_reported():
    x = make(1, 4, 4, 2, 64, 512, [300], seed=12)
    mk.mk_attention_set_wait_timeout_ns(20_000_000)
    try:
        mk.mk_attention_debug_drop_unit(1)
        t = {key: None if val is None else val.to(DEV) for key, val in x.items()}
        o = torch.zeros_like(t["q"])
        mk.mk_tree_attention(t["q"], t["k"], t["v"], o, t["parents"], None, t["lens"], 0.1)
        assert mk.mk_tree_attention_status() == mk.MK_ERR_DEVICE_TIMEOUT
        assert "timed out" in mk.mk_last_error()
    finally:
        mk.mk_attention_debug_drop_unit(-1)
        mk.mk_attention_set_wait_timeout_ns(2_000_000_000)
    assert mk.mk_tree_attention_status() == mk.MK_OK
    check(x, 0.1, run(x, 0.1))
