"""mk_tree_verify where its contract is easy to miss; the answers are the definition's."""
import numpy as np
import pytest
import torch

import persistent_megakernel_decode_04_b200 as mk
from test_tree_verify_gpu import DEV, call, check, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [5, 1001, 50257, 300001])
def test_draft_rows_of_nodes_without_children_need_not_exist(dtype, V):
    """Chains whose draft has a row for every node but the last: the last node's place is the next
    sequence's first row, and behind the last sequence there is nothing of the draft's (room that
    holds NaN here).  Walks that end on the leaf, and walks that end before it."""
    B, n = 4, 4
    x = inputs(B, n, V, "chain", True, dtype, seed=V)
    x["u"][0] = x["u"][3] = 0.0  # every draft accepted
    x["u"][1, 2] = x["u"][2, 1] = 0.999
    want = check(**x)
    assert want[0] == n and want[3] == n
    room = torch.full((B * (n - 1) + 1, V), float("nan"), dtype=dtype, device=DEV)
    room[:B * (n - 1)] = x["draft"][:, :n - 1].reshape(-1, V).to(DEV)
    short = room.as_strided((B, n, V), ((n - 1) * V, V, 1))
    t = {key: None if val is None else val.to(DEV) for key, val in x.items() if key != "draft"}
    path, n_path, nxt = (torch.full(s, 77, dtype=torch.int32, device=DEV) for s in ((B, n), (B,), (B,)))
    ws = torch.full((mk.mk_tree_verify_workspace_bytes(B, n, V),), 255, dtype=torch.uint8, device=DEV)
    mk.mk_tree_verify(t["target"], short, t["tokens"], t["parents"], None, t["u"], t["r"], None, None, path, n_path,
                      nxt, ws)
    for got, ref in zip((path, n_path, nxt), call(**x)):
        assert torch.equal(got.cpu(), ref)


@pytest.mark.parametrize("V", [37, 128255])
def test_leaves_of_trees_are_drawn_from_the_target_alone(V):
    x = inputs(6, 12, V, "tree", True, torch.bfloat16, seed=V)
    leaf = torch.ones(6, 12, dtype=torch.bool)
    leaf.scatter_(1, x["parents"].clamp(min=0).long(), False)
    x["u"][:3] = 0.0
    check(**x)
    want = call(**x)
    assert any(leaf[b, want[0][b, want[1][b] - 1]] for b in range(6))
    x["draft"][leaf] = float("nan")
    for got, ref in zip(call(**x), want):
        assert torch.equal(got, ref)
