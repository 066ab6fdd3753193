"""mk_tree_verify against its definition in extended precision: whole numbers, equal."""
import numpy as np
import pytest
import torch

import persistent_megakernel_decode_04_b200 as mk
from _speculative import random_tree, verify_walk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def call(target, draft, tokens, parents, n_nodes, u, r, temperature, draft_temperature, stream=None):
    B, n, V = target.shape
    i32 = lambda *s: torch.full(s, 77, dtype=torch.int32, device=DEV)  # noqa: E731
    path, n_path, nxt = i32(B, n), i32(B), i32(B)
    ws = torch.full((mk.mk_tree_verify_workspace_bytes(B, n, V),), 255, dtype=torch.uint8, device=DEV)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    mk.mk_tree_verify(dev(target), dev(draft), dev(tokens), dev(parents), dev(n_nodes), dev(u), dev(r),
                      dev(temperature), dev(draft_temperature), path, n_path, nxt, ws, stream)
    return path.cpu(), n_path.cpu(), nxt.cpu()


def check(target, draft, tokens, parents, n_nodes, u, r, temperature, draft_temperature):
    path, n_path, nxt = call(target, draft, tokens, parents, n_nodes, u, r, temperature, draft_temperature)
    B, n, V = target.shape
    num = lambda t, b, other: other if t is None else float(t[b])  # noqa: E731
    lengths = []
    for b in range(B):
        want, tok, margin = verify_walk(
            target[b].float().numpy(), None if draft is None else draft[b].float().numpy(), tokens[b].numpy(),
            parents[b].numpy(), n if n_nodes is None else min(max(int(n_nodes[b]), 0), n), u[b].numpy(), float(r[b]),
            num(temperature, b, 1.0), num(draft_temperature, b, 1.0))
        assert margin > 1e-11, "the inputs sit on a border: choose others"
        got = path[b].tolist()
        assert int(n_path[b]) == len(want) and got == want + [-1] * (n - len(want)), (b, got, want)
        assert int(nxt[b]) == tok, (b, int(nxt[b]), tok)
        lengths.append(len(want))
    return lengths


def inputs(B, n, V, kind, sampled, dtype=torch.float32, seed=0, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    parents = torch.from_numpy(np.stack([random_tree(rng, n, kind) for _ in range(B)]))
    target = torch.randn(B, n, V, generator=g) * spread
    draft = (target + torch.randn(B, n, V, generator=g) * 0.5).to(dtype)
    target = target.to(dtype)
    tokens = torch.zeros(B, n, dtype=torch.int32)
    for b in range(B):
        for c in range(1, n):
            row = draft[b, max(int(parents[b, c]), 0)].float()
            if sampled:
                tokens[b, c] = torch.multinomial(torch.softmax(row, 0), 1, generator=g)[0]
            else:
                rank = int((parents[b, :c] == parents[b, c]).sum())
                tokens[b, c] = row.topk(min(rank + 1, V)).indices[-1]
    return dict(target=target, draft=draft if sampled else None, tokens=tokens, parents=parents, n_nodes=None,
                u=torch.rand(B, n, generator=g), r=torch.rand(B, generator=g), temperature=None,
                draft_temperature=None)


@pytest.mark.parametrize("kind", ["chain", "tree", "star", "forest"])
@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("n,V", [(1, 1000), (2, 5), (7, 1001), (33, 8193), (12, 50257)])
def test_matches_the_definition(kind, sampled, n, V):
    x = inputs(3, n, V, kind, sampled, seed=n + V)
    check(**x)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [9, 4097, 32003, 128256])
def test_types_and_vocabularies(dtype, V):
    x = inputs(2, 6, V, "tree", True, dtype, seed=V)
    x["temperature"], x["draft_temperature"] = torch.tensor([0.7, 1.4]), torch.tensor([1.1, 0.6])
    check(**x)


def test_paths_of_every_length_and_greedy_sequences_in_one_batch():
    x = inputs(12, 9, 300, "chain", True, seed=1, spread=4.0)
    x["temperature"] = torch.tensor([0.0, 0.5, 1.0, 0.0, 1.0, 1.0, 0.9, 0.0, 2.0, 1.0, 1.0, 1.0])
    for b in (0, 3, 7):  # greedy: the chain follows the target for 3, 8 and 0 steps
        best = x["target"][b].argmax(-1).to(torch.int32)
        x["tokens"][b, 1:] = best[:-1]
        if b == 0:
            x["tokens"][b, 4] += 1
        if b == 7:
            x["tokens"][b, 1] += 1
    x["u"][4] = 0.0        # accepts whatever has a probability
    x["n_nodes"] = torch.tensor([9, 9, 4, 9, 9, 1, 0, 9, 50, -2, 9, 2], dtype=torch.int32)
    lengths = check(**x)
    assert lengths[0] == 4 and lengths[3] == 9 and lengths[7] == 1 and lengths[4] == 9
    assert lengths[6] == 0 and lengths[9] == 0 and len(set(lengths)) >= 4


def test_greedy_takes_the_lowest_of_equal_logits():
    x = inputs(2, 3, 20000, "chain", False, seed=2)
    x["target"][0, 0, [19000, 700, 12000]] = 50.0
    x["target"][1, 0, [9000, 15000]] = 50.0
    x["tokens"][0, 1], x["tokens"][1, 1] = 700, 15000
    x["temperature"] = torch.zeros(2)
    path, n_path, nxt = call(**x)
    assert n_path.tolist()[1] == 1 and int(nxt[1]) == 9000 and path[0, 1] == 1
    check(**x)


def test_many_siblings_rejected():
    # (a sampled draft with p > q is accepted whatever u is: the first of these are among them)
    for sampled in (True, False):
        x = inputs(2, 40, 700, "star", sampled, seed=3, spread=0.5)
        x["u"][:] = 0.999
        check(**x)
    # 39 drafts of words that the target hardly has: the rest is formed 39 times over
    x = inputs(2, 40, 700, "star", True, seed=3, spread=0.5)
    x["draft"][:, 0, 3:6] = 9.0
    x["target"][:, 0, 3:6] = -6.0
    x["tokens"][:, 1:] = 3 + torch.arange(39, dtype=torch.int32) % 3
    x["u"][:] = 0.5
    assert check(**x) == [1, 1]


def test_equal_siblings_and_tokens_outside_the_vocabulary():
    x = inputs(2, 6, 50, "star", False, seed=4)
    x["tokens"][:, 1:] = torch.tensor([[7, 7, 7, 8, 8], [-1, 50, 2**30, -(2**31), 9]], dtype=torch.int32)
    x["u"][:] = 0.9
    check(**x)
    x = inputs(2, 6, 50, "star", True, seed=4)
    x["tokens"][:, 1:] = torch.tensor([[7, 7, 7, 8, 8], [-1, 50, 2**30, -(2**31), 9]], dtype=torch.int32)
    x["u"][:] = 0.9
    check(**x)


def test_decisions_at_their_border():
    # uniform over 8: p = 1/8 exactly.  u at 1/8 rejects, one step below accepts; r at k/8 draws k
    V, n = 8, 2
    step = 2.0 ** -27
    u = torch.tensor([[0, 0.125], [0, 0.125 - step], [0, 0.125 + step]])
    x = dict(target=torch.zeros(3, n, V), draft=None, tokens=torch.full((3, n), 5, dtype=torch.int32),
             parents=torch.tensor([[-1, 0]] * 3, dtype=torch.int32), n_nodes=None, u=u,
             r=torch.tensor([0.5, 0.375, 0.0]), temperature=None, draft_temperature=None)
    path, n_path, nxt = call(**x)
    assert n_path.tolist() == [1, 2, 1]
    # sequence 0: token 5 is gone, 7 left, 0.5 x 7 = 3.5: the fourth; 1: k = 3; 2: the first
    assert nxt.tolist() == [3, 3, 0]
    # the draft sure of what the target is sure of: u just below 1 accepts
    x = dict(x, draft=torch.zeros(3, n, V), u=torch.full((3, n), 1 - 2.0 ** -24))
    assert call(**x)[1].tolist() == [2, 2, 2]


@pytest.mark.parametrize("sampled", [True, False])
def test_temperatures_near_zero_and_very_high(sampled):
    # 1e-40: the reciprocal is beyond fp32's range; the law is one-hot at the largest logit
    x = inputs(6, 9, 2001, "tree", sampled, seed=41)
    x["temperature"] = torch.tensor([1e-40, 1e-38, 1e-30, 1e-3, 1e3, 1e30])
    x["draft_temperature"] = torch.tensor([1.0, 1e-40, 0.5, 1e-3, 1e30, 2.0])
    check(**x)


@pytest.mark.parametrize("sampled,V", [(True, 128255), (True, 262144), (True, 1 << 20), (False, 1 << 20)])
def test_the_largest_vocabularies(sampled, V):
    # of a pass everything is kept, the draft's exponentials in part, nothing; more sequences than clusters of 16
    x = inputs(10 if V < 1 << 20 else 2, 4, V, "star", sampled, torch.bfloat16, seed=43)
    x["u"] = 0.5 + x["u"] / 2  # more rejections
    check(**x)


@pytest.mark.parametrize("n", [33, 256])
def test_many_certain_siblings_with_little_left(n):
    # no draft probabilities: what is left of P shrinks to less than an eighth, then further
    x = inputs(4, n, n + 40, "star", False, seed=n, spread=1.0)
    x["u"] = 0.6 + 0.4 * x["u"]
    check(**x)


def test_rows_that_are_no_distribution():
    x = inputs(4, 4, 3000, "chain", True, seed=6)
    x["u"][:] = 0.0
    x["target"][0, 0, 2000] = float("nan")
    x["target"][1, 1, :] = float("-inf")
    x["target"][2, 2, 5] = float("inf")
    x["target"][3, :, 100:] = float("-inf")  # a masked vocabulary is one
    x["tokens"][3] = 3
    path, n_path, nxt = call(**x)
    assert n_path.tolist() == [1, 2, 3, 4]
    assert nxt.tolist()[:3] == [-1, -1, -1] and 0 <= int(nxt[3]) < 100


@pytest.mark.parametrize("sampled", [True, False])
def test_rows_that_are_no_distribution_at_temperature_zero(sampled):
    x = inputs(6, 5, 3000, "chain", sampled, seed=7)
    x["tokens"][:, 1:] = x["target"].argmax(-1)[:, :-1]  # every draft is the greedy one
    x["temperature"] = torch.zeros(6)
    x["target"][0, 0, 2000] = float("nan")
    x["target"][1, 1, :] = float("-inf")
    x["target"][2, 2, 5] = float("inf")
    x["tokens"][2, 3] = 5
    x["target"][3, 3, :] = float("nan")
    x["tokens"][3, 4] = 2 ** 31 - 1
    x["target"][4, :, 100:] = float("-inf")
    x["tokens"][4, 1:] = x["target"][4].argmax(-1)[:-1]
    assert check(**x) == [1, 2, 3, 4, 5, 5]
    path, n_path, nxt = call(**x)
    assert nxt.tolist()[:4] == [-1] * 4


def test_a_rejected_token_without_a_number_leaves_no_distribution():
    x = inputs(3, 4, 500, "star", False, seed=9)
    x["u"][:] = 0.999
    for b in range(3):
        x["target"][b, 0, int(x["tokens"][b, 1 + b])] = float("nan")
    path, n_path, nxt = call(**x)
    assert n_path.tolist() == [1, 1, 1] and nxt.tolist() == [-1, -1, -1]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [2, 7, 31, 1000, 50257])
def test_a_draft_that_equals_the_target_leaves_nothing(dtype, V):
    # tokens outside the vocabulary are rejected; max(P - q, 0) is nothing, to the bit, and P stays
    x = inputs(12, 4, V, "star", True, dtype, seed=V)
    x["draft"] = x["target"].clone()
    x["tokens"][:, 1], x["tokens"][:, 2], x["tokens"][:, 3] = -1, V, V + 5
    x["temperature"] = torch.linspace(0.5, 1.6, 12)
    x["draft_temperature"] = x["temperature"].clone()
    assert check(**x) == [1] * 12


def test_odd_strides_and_unaligned_rows():
    x = inputs(2, 5, 1000, "tree", True, torch.bfloat16, seed=7)
    whole = {}
    for key, pad in (("target", 3), ("draft", 6)):
        room = torch.full((2, 5, 1000 + pad), 99.0, dtype=torch.bfloat16, device=DEV)
        room[..., 1:1001] = x[key].to(DEV)
        whole[key] = room[..., 1:1001]
    check(**x)
    want = call(**x)
    got = call(**dict(x, **whole))
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # one target row for all nodes (a stride of 0)
    one = dict(x, target=x["target"][:, :1].expand(2, 5, 1000), draft=None)
    many = dict(x, target=x["target"][:, :1].expand(2, 5, 1000).contiguous(), draft=None)
    assert all(torch.equal(a, b) for a, b in zip(call(**one), call(**many)))


def test_the_targets_law():
    """Whatever the draft, the first new token follows the target's distribution."""
    B, n, V = 16000, 4, 6
    g = torch.Generator().manual_seed(8)
    logits = torch.tensor([0.3, -1.0, 1.2, 0.0, -0.5, 0.8])
    dlogits = torch.tensor([1.0, 0.5, -0.3, 0.2, 1.5, -2.0])
    tokens = torch.multinomial(torch.softmax(dlogits, 0), B * n, True, generator=g).view(B, n).to(torch.int32)
    target, draft = logits.expand(B, n, V), dlogits.expand(B, n, V)
    for parents in ([-1, 0, 0, 0], [-1, 0, 1, 2]):
        par = torch.tensor(parents, dtype=torch.int32).expand(B, n).contiguous()
        path, n_path, nxt = call(target.contiguous(), draft.contiguous(), tokens, par, None,
                                 torch.rand(B, n, generator=g), torch.rand(B, generator=g), None, None)
        first = torch.where(n_path > 1, tokens[torch.arange(B), path[:, 1].clamp(min=0).long()], nxt)
        p = torch.softmax(logits.double(), 0)
        freq = torch.bincount(first.long(), minlength=V).double() / B
        assert ((freq - p).abs() < 5 * (p * (1 - p) / B).sqrt()).all(), (freq, p)


def test_streams_and_graphs():
    xs = [{k: None if v is None else v.to(DEV) for k, v in inputs(2, 8, 5000, "tree", True, seed=s).items()}
          for s in (9, 10)]
    want = [call(**x) for x in xs]
    B, n, V = 2, 8, 5000
    st = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for s, x in zip(st, xs):
        o = [torch.zeros(B, n, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV),
             torch.zeros(B, dtype=torch.int32, device=DEV)]
        ws = torch.zeros(mk.mk_tree_verify_workspace_bytes(B, n, V), dtype=torch.uint8, device=DEV)
        outs.append((o, ws))
    torch.cuda.synchronize()
    for rep in range(10):
        for s, x, (o, ws) in zip(st, xs, outs):
            mk.mk_tree_verify(x["target"], x["draft"], x["tokens"], x["parents"], None, x["u"], x["r"], None, None,
                              *o, ws, s)
    torch.cuda.synchronize()
    for (o, ws), w in zip(outs, want):
        assert all(torch.equal(a.cpu(), b) for a, b in zip(o, w))
    x, (o, ws) = xs[0], outs[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mk.mk_tree_verify(x["target"], x["draft"], x["tokens"], x["parents"], None, x["u"], x["r"], None, None, *o, ws,
                          torch.cuda.current_stream())
    for key in ("target", "draft", "tokens", "parents", "u", "r"):
        x[key].copy_(xs[1][key])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a.cpu(), b) for a, b in zip(o, want[1]))
