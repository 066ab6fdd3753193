"""The speculative operators together, as a decoding loop uses them: tree forward, verification,
commit, reorder, and ordinary decode steps on the cache that they leave."""
import numpy as np
import pytest
import torch

import mk_inputs as mi
import oracle
import persistent_megakernel_decode_04_b200 as mk
from _parity import ARGMAX_MARGIN, argmax_agrees, kv_close, logits_close
from _speculative import ancestors

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def model(shape, max_batch, max_seq, seed=5, tc_min=0):
    w = mi.make_weights(shape, seed=seed)
    cfg = mk.Config.from_shape(w.shape, max_batch, max_seq)
    cfg.tc_min_batch = tc_min
    return w, mk.Megakernel(cfg, w, 0)


@pytest.mark.parametrize("shape,max_batch,B,tc_min", [(mi.TINY, 1, 1, 0), (mi.TINY, 4, 3, 0), (mi.TINY, 4, 3, 5),
                                                      (mi.TINY, 16, 2, 0), (mi.TINY_QK, 1, 1, 0), (mi.TINY_QK, 16, 2, 0)])
def test_tree_forward_matches_the_oracle_on_every_path(shape, max_batch, B, tc_min):
    w, m = model(shape, max_batch, 64, tc_min=tc_min)
    rng = np.random.default_rng(B)
    T = [9 + 3 * b for b in range(B)]
    n = 7
    parents = np.array([-1, 0, 0, 1, 1, 2, 3], dtype=np.int32)
    tokens = rng.integers(0, w.shape.vocab, (B, n)).astype(np.int32)
    prompts = [mi.prompt(5, b, T[b], w.shape.vocab) for b in range(B)]
    # the prompts, one after another, as trees that are chains; each is committed whole
    lens = i32([0] * B)
    t_max = max(T)
    toks = np.zeros((B, t_max), dtype=np.int32)
    for b in range(B):
        toks[b, :T[b]] = prompts[b]
    chain = i32(np.tile(np.arange(t_max) - 1, (B, 1)))
    first = m.tree_forward(i32(toks), chain, lens, i32(T))
    lens = m.commit(i32(np.tile(np.arange(t_max), (B, 1))), i32(T), lens)
    assert lens.tolist() == T
    logits = m.tree_forward(i32(tokens), i32(np.tile(parents, (B, 1))), lens).cpu().numpy()
    assert mk.mk_tree_attention_status() == mk.MK_OK
    paths = ancestors(parents, n)
    for b in range(B):
        for i in range(n):
            ref = oracle.Decoder(w, 1, 64)
            rl = ref.prefill(np.concatenate([prompts[b], tokens[b, paths[i]]])[None])[0]
            logits_close(logits[b, i], rl, f"seq {b} node {i}")
        ref = oracle.Decoder(w, 1, 64)
        rl = ref.prefill(prompts[b][None])[0]
        logits_close(first[b, T[b] - 1].cpu().numpy(), rl, f"prompt {b}")
        kv_close(m.kv_view()[:, :, b:b + 1, :, :T[b], :].cpu().numpy(), ref.get_cache(T[b]), f"cache {b}")
    m.close()


@pytest.mark.parametrize("sampled", [False, True])
def test_greedy_speculation_emits_the_greedy_text(sampled):
    """Drafts that are sometimes right: whatever they are, the tokens are the target's own choices;
    then plain decode steps go on from the committed cache."""
    w, m = model(mi.TINY, 4, 128)
    B, V, T, n = 3, w.shape.vocab, 8, 9
    rng = np.random.default_rng(1)
    prompts = np.stack([mi.prompt(7, b, T, V) for b in range(B)])
    m.prefill(i32(prompts[:, :T - 1]))  # the last prompt token is the first tree's root
    lens = i32([T - 1] * B)
    text = [list(prompts[b]) for b in range(B)]
    ws = torch.empty(mk.mk_tree_verify_workspace_bytes(B, n, V), dtype=torch.uint8, device=DEV)
    oracles = [oracle.Decoder(w, 1, 128) for _ in range(B)]
    rl = [oracles[b].prefill(prompts[b][None])[0] for b in range(B)]
    accepted = 0
    for step in range(6):
        parents = np.tile(np.array([-1, 0, 0, 1, 1, 2, 3, 3, 6], dtype=np.int32), (B, 1))
        tokens = rng.integers(0, V, (B, n)).astype(np.int32)
        for b in range(B):
            tokens[b, 0] = text[b][-1]
            if step % 3 != 2:  # the true continuation along 0-1-3, or 0-2-5
                ref = oracle.Decoder(w, 1, 128)
                t = oracle.argmax(ref.prefill(np.array(text[b], dtype=np.int32)[None])[0])
                for node in ((1, 3, 6) if step % 3 == 0 else (2, 5)):
                    tokens[b, node] = t
                    t = oracle.argmax(ref.decode(np.array([t], dtype=np.int32))[0])
        logits = m.tree_forward(i32(tokens), i32(parents), lens)
        path, n_path, nxt = i32(np.zeros((B, n))), i32([0] * B), i32([0] * B)
        mk.mk_tree_verify(logits, torch.randn_like(logits) if sampled else None, i32(tokens), i32(parents), None,
                          torch.rand(B, n, device=DEV), torch.rand(B, device=DEV), torch.zeros(B, device=DEV),
                          torch.ones(B, device=DEV) if sampled else None, path, n_path, nxt, ws)
        new_lens = m.commit(path, n_path, lens)
        assert (new_lens == lens + n_path).all()
        for b in range(B):
            kept = path[b, 1:int(n_path[b])].tolist()
            accepted += len(kept)
            for t in [int(tokens[b, i]) for i in kept] + [int(nxt[b])]:
                margin = np.sort(rl[b].astype(np.float64))[-2:]
                assert t == oracle.argmax(rl[b]) or margin[1] - margin[0] <= ARGMAX_MARGIN
                text[b].append(t)
                rl[b] = oracles[b].decode(np.array([t], dtype=np.int32))[0]
            assert int(new_lens[b]) == len(text[b]) - 1
        lens = new_lens
    assert accepted >= 2 * B
    m.set_positions(lens.tolist())
    for b in range(B):
        kv_close(m.kv_view()[:, :, b:b + 1, :, :int(lens[b]), :].cpu().numpy(), oracles[b].get_cache(int(lens[b])), f"seq {b}")
    got, nt = m.decode(i32([text[b][-1] for b in range(B)]))
    for b in range(B):
        logits_close(got[b].cpu().numpy(), rl[b], f"decode after speculation, seq {b}")
        assert argmax_agrees(got[b].cpu().numpy(), rl[b], int(nt[b]))
    assert m.sync_status() == mk.MK_OK
    m.close()


def test_forked_prompt_decodes_like_its_source():
    w, m = model(mi.TINY, 4, 64)
    T = 11
    prompt = mi.prompt(3, 0, T, w.shape.vocab)
    m.prefill(i32(prompt[None]))
    lens = m.reorder(i32([0, 0, 0, 0]), i32([T, 0, 5, 9]))
    assert lens.tolist() == [T] * 4
    m.set_positions(lens.tolist())
    toks = [3, 500, 77, 3]
    got, _ = m.decode(i32(toks))
    for b in range(4):
        ref = oracle.Decoder(w, 1, 64)
        ref.prefill(prompt[None])
        logits_close(got[b].cpu().numpy(), ref.decode(np.array([toks[b]], dtype=np.int32))[0], f"fork {b}")
    assert torch.equal(got[0], got[3])
    m.close()


def test_tree_forward_at_the_caches_end():
    w, m = model(mi.TINY, 2, 32)
    prompts = np.stack([mi.prompt(4, b, 30, w.shape.vocab) for b in range(2)])
    m.prefill(i32(prompts))
    before = m.kv_view().clone()
    toks = i32([[1, 2, 3, 4, 5]] * 2)
    logits = m.tree_forward(toks, i32([[-1, 0, 1, 2, 3]] * 2), i32([30, 12]))
    for b, ln in ((0, 30), (1, 12)):
        ref = oracle.Decoder(w, 1, 32)
        ref.prefill(prompts[b][None, :ln])
        for i in range(min(5, 32 - ln)):
            logits_close(logits[b, i].cpu().numpy(), ref.decode(np.array([i + 1], dtype=np.int32))[0], f"{b} {i}")
    after = m.kv_view()
    assert torch.equal(after[:, :, 0, :, :30], before[:, :, 0, :, :30])
    assert torch.equal(after[:, :, 1, :, :12], before[:, :, 1, :, :12])
    assert torch.equal(after[:, :, 1, :, 17:], before[:, :, 1, :, 17:])
    with pytest.raises(mk.MkError):
        m.tree_forward(i32([[0] * 40] * 2), i32([[-1] * 40] * 2), i32([0, 0]))  # 80 rows: scratch for 64
    m.close()


def test_nodes_not_in_use_leave_the_cache_alone():
    w, m = model(mi.TINY, 4, 48)
    prompts = np.stack([mi.prompt(4, b, 20, w.shape.vocab) for b in range(4)])
    m.prefill(i32(prompts))
    before = m.kv_view().clone()
    toks = i32([[1, 2, 3, 4, 5, 6]] * 3)
    par = i32([[-1, 0, 0, 1, 2, 3]] * 3)
    use = [2, 0, 99]
    got = m.tree_forward(toks, par, i32([20, 7, 20]), i32(use))
    after = m.kv_view().clone()
    for b, ln, nn in ((0, 20, 2), (1, 7, 0), (2, 20, 6), (3, 20, 0)):
        assert torch.equal(after[:, :, b, :, :ln], before[:, :, b, :, :ln])
        assert torch.equal(after[:, :, b, :, ln + nn:], before[:, :, b, :, ln + nn:])
    every = m.tree_forward(toks, par, i32([20, 7, 20]))
    for b, nn in ((0, 2), (2, 6)):
        assert torch.equal(got[b, :nn], every[b, :nn])
    m.close()


def test_a_whole_step_replayed_from_a_graph():
    """Forward, verification and commit captured once, then replayed with other drafts: what the
    same calls give one by one."""
    w, m = model(mi.TINY, 2, 96)
    B, n, V, T = 2, 6, w.shape.vocab, 10
    prompts = np.stack([mi.prompt(8, b, T, V) for b in range(B)])
    m.prefill(i32(prompts))
    start = m.kv_view().clone()
    rng = np.random.default_rng(3)
    tokens, parents = i32(np.zeros((B, n))), i32(np.tile([-1, 0, 0, 1, 2, 4], (B, 1)))
    lens, new_lens = i32([T] * B), i32([0] * B)
    u, r = torch.zeros(B, n, device=DEV), torch.zeros(B, device=DEV)
    temperature = torch.full((B,), 0.2, device=DEV)
    path, n_path, nxt = i32(np.zeros((B, n))), i32([0] * B), i32([0] * B)
    logits = torch.empty(B, n, V, device=DEV)
    ws = torch.empty(mk.mk_tree_verify_workspace_bytes(B, n, V), dtype=torch.uint8, device=DEV)
    stream = torch.cuda.Stream()

    def step():
        mk.mk_tree_forward(m.ctx, tokens, parents, None, lens, B, n, m.kv, logits, stream)
        mk.mk_tree_verify(logits, None, tokens, parents, None, u, r, temperature, None, path, n_path, nxt, ws, stream)
        mk.mk_cache_commit(m.kv_view(), path, n_path, lens, new_lens, stream)

    drafts = []
    for _ in range(4):
        t = rng.integers(0, V, (B, n)).astype(np.int32)
        drafts.append((t, torch.rand(B, n, device=DEV) * 0.05, torch.rand(B, device=DEV)))

    def run(go):
        m.kv_view().copy_(start)
        lens.fill_(T)
        out = []
        for t, uu, rr in drafts:
            tokens.copy_(torch.from_numpy(t))
            u.copy_(uu)
            r.copy_(rr)
            torch.cuda.synchronize()
            go()
            stream.synchronize()
            out += [path.clone(), n_path.clone(), nxt.clone(), new_lens.clone(), logits.clone()]
            lens.copy_(new_lens)
        return out + [m.kv_view().clone()]

    one_by_one = run(step)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        step()

    def replay():
        with torch.cuda.stream(stream):
            graph.replay()

    for a, b in zip(one_by_one, run(replay)):
        assert torch.equal(a, b)
    assert mk.mk_tree_attention_status() == mk.MK_OK
    m.close()


def test_two_streams_forked_and_joined_in_a_graph():
    """Attention of one stream's data beside a commit and a verification on another, joined before a
    reorder that needs both; copies and fills ahead of the kernels; replayed several times."""
    g = torch.Generator().manual_seed(11)
    B, n, hq, hkv, d, S, V = 2, 9, 8, 2, 64, 200, 3001
    q = torch.randn(B, n, hq, d, generator=g).bfloat16().to(DEV)
    src_kv = torch.randn(2, 2, B, hkv, S, d, generator=g).bfloat16().to(DEV)
    kv, o = torch.empty_like(src_kv), torch.empty_like(q)
    other = src_kv.flip(4).contiguous()
    target = torch.randn(B, n, V, generator=g).to(DEV)
    parents = i32(np.tile([-1, 0, 0, 1, 1, 2, 3, 3, 6], (B, 1)))
    tokens = target[:, :1].argsort(-1, descending=True)[:, 0, :n].to(torch.int32).contiguous()
    lens, new_lens, third, fourth = i32([150, 77]), i32([0, 0]), i32([0, 0]), i32([0, 0])
    u, r = torch.full((B, n), 1e-4, device=DEV), torch.tensor([0.2, 0.7], device=DEV)
    path, n_path, nxt = i32(np.zeros((B, n))), i32([0] * B), i32([0] * B)
    ws = torch.empty(mk.mk_tree_verify_workspace_bytes(B, n, V), dtype=torch.uint8, device=DEV)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()

    def calls():
        kv.copy_(src_kv)
        o.zero_()
        fork, join = torch.cuda.Event(), torch.cuda.Event()
        fork.record(one)
        two.wait_event(fork)
        mk.mk_tree_attention(q, kv[0, 0], kv[0, 1], o, parents, None, lens, 0.125, one)
        with torch.cuda.stream(two):
            path.fill_(-7)
            mk.mk_tree_verify(target, None, tokens, parents, None, u, r, None, None, path, n_path, nxt, ws, two)
            mk.mk_cache_commit(other, path, n_path, lens, new_lens, two)
        join.record(two)
        one.wait_event(join)
        mk.mk_cache_commit(kv, path, n_path, lens, third, one)
        mk.mk_cache_reorder(kv, i32_src, third, fourth, one)

    i32_src = i32([1, 0])
    kept = other.clone()
    with torch.cuda.stream(one):
        calls()
    torch.cuda.synchronize()
    want = [t.clone() for t in (o, path, n_path, nxt, new_lens, third, fourth, kv, other)]
    assert int(n_path.min()) > 1
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(one), torch.cuda.graph(graph, stream=one):
        calls()
    for _ in range(3):
        other.copy_(kept)
        for t in (o, path, n_path, nxt, new_lens, third, fourth, kv):
            t.fill_(3)
        torch.cuda.synchronize()
        with torch.cuda.stream(one):
            graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (o, path, n_path, nxt, new_lens, third, fourth, kv, other)):
            assert torch.equal(a, b)
    assert mk.mk_tree_attention_status() == mk.MK_OK
