"""The speculative operators on torch's streams: a call without a stream follows the caller's."""
import numpy as np
import pytest
import torch

import persistent_megakernel_decode_04_b200 as mk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Step:
    """One call of each operator on small data, without a stream argument; `fill` gives the inputs."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        B, n, hq, hkv, d, S, V = 2, 5, 4, 2, 64, 100, 999
        self.inputs = dict(
            q=torch.randn(B, n, hq, d, generator=g).bfloat16(), kv=torch.randn(2, 2, B, hkv, S, d, generator=g).bfloat16(),
            target=torch.randn(B, n, V, generator=g), u=torch.rand(B, n, generator=g) * 1e-3, r=torch.rand(B, generator=g),
            tokens=torch.randint(0, V, (B, n), generator=g, dtype=torch.int32),
            lens=torch.randint(1, S - n, (B,), generator=g, dtype=torch.int32),
            src=torch.randint(0, B, (B,), generator=g, dtype=torch.int32))
        self.ws = torch.zeros(mk.mk_tree_verify_workspace_bytes(B, n, V), dtype=torch.uint8, device=DEV)
        self.parents = i32([[-1, 0, 0, 1, 1]] * B)
        self.t = {key: torch.zeros_like(val, device=DEV) for key, val in self.inputs.items()}
        self.outs = dict(o=torch.zeros_like(self.t["q"]), path=i32(np.zeros((B, n))), n_path=i32([0] * B),
                         nxt=i32([0] * B), lens1=i32([0] * B), lens2=i32([0] * B))
        self.ready = {key: val.to(DEV) for key, val in self.inputs.items()}

    def fill(self):
        for key, val in self.ready.items():
            self.t[key].copy_(val)

    def calls(self):
        t, o = self.t, self.outs
        mk.mk_tree_attention(t["q"], t["kv"][1, 0], t["kv"][1, 1], o["o"], self.parents, None, t["lens"], 0.125)
        mk.mk_tree_verify(t["target"], None, t["tokens"], self.parents, None, t["u"], t["r"], None, None, o["path"],
                          o["n_path"], o["nxt"], self.ws)
        mk.mk_cache_commit(t["kv"], o["path"], o["n_path"], t["lens"], o["lens1"])
        mk.mk_cache_reorder(t["kv"], t["src"], o["lens1"], o["lens2"])

    def results(self):
        return [val.clone() for val in self.outs.values()] + [self.t["kv"].clone()]


def plain(step):
    step.fill()
    step.calls()
    torch.cuda.synchronize()
    want = step.results()
    for val in list(step.outs.values()) + list(step.t.values()):
        val.zero_()
    torch.cuda.synchronize()
    return want


def test_without_a_stream_a_call_waits_for_its_inputs_on_the_current_one():
    step = Step(1)
    want = plain(step)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(40_000_000)  # 20 ms before the inputs are there
        step.fill()
        step.calls()
        got = step.results()
        assert mk.mk_tree_attention_status() == mk.MK_OK
        assert s.query()  # (the status waited for this stream)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_without_a_stream_a_call_is_captured_with_the_current_one():
    step = Step(2)
    want = plain(step)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.calls()
    step.fill()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(step.results(), want):
        assert torch.equal(a, b)


def test_the_null_stream_by_its_handle():
    step = Step(3)
    want = plain(step)
    step.fill()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):  # (a blocked current stream does not hold up the NULL stream's call)
        torch.cuda._sleep(40_000_000)
        t, o = step.t, step.outs
        mk.mk_tree_attention(t["q"], t["kv"][1, 0], t["kv"][1, 1], o["o"], step.parents, None, t["lens"], 0.125, 0)
        torch.cuda.default_stream().synchronize()
        assert not torch.cuda.current_stream().query()
        with torch.cuda.stream(torch.cuda.default_stream()):
            assert torch.equal(o["o"], want[0])
