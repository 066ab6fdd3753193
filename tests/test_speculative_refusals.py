"""What the speculative-decoding entry points refuse, on the CPU: nothing is launched."""
import ctypes

import pytest
import torch

import persistent_megakernel_decode_04_b200 as mk

OK = 1 << 20  # a 16-byte aligned address that is never used


def tree_shape(**kw):
    f = dict(dtype=mk.MK_BF16, wide=0, B=2, n=8, n_q_heads=8, n_kv_heads=2, head_dim=64, max_seq=128, q_seq=8 * 8 * 64,
             q_node=8 * 64, q_head=64, k_seq=2 * 128 * 64, k_head=128 * 64, k_row=64, v_seq=2 * 128 * 64,
             v_head=128 * 64, v_row=64, o_seq=8 * 8 * 64, o_node=8 * 64, o_head=64)
    f.update(kw)
    return mk.mk_tree_shape(**f)


def attend(shape, q=OK, k=OK, v=OK, o=OK, parents=OK, n_nodes=None, lens=OK, scale=0.125):
    return mk._lib.mk_tree_attention(ctypes.byref(shape) if shape else None, q, k, v, o, parents, n_nodes, lens, scale, None)


@pytest.mark.parametrize("kw", [dict(dtype=mk.MK_FP32), dict(dtype=-1), dict(wide=2), dict(B=0), dict(n=0), dict(n=257), dict(max_seq=0),
                                dict(head_dim=96), dict(n_kv_heads=3), dict(n_kv_heads=0), dict(n_q_heads=0),
                                dict(n_q_heads=258, n_kv_heads=2), dict(q_node=4), dict(k_row=0), dict(k_row=-64),
                                dict(v_head=100), dict(o_seq=1), dict(k_seq=1 << 40)])
def test_tree_attention_shapes(kw):
    assert attend(tree_shape(**kw)) == mk.MK_ERR_INVALID_ARG
    assert mk.mk_last_error()


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(parents=None), dict(lens=None),
                                dict(q=OK + 2), dict(k=OK + 8), dict(v=OK + 4), dict(o=OK + 8), dict(scale=0.0),
                                dict(scale=float("nan")), dict(scale=float("inf"))])
def test_tree_attention_operands(kw):
    assert attend(tree_shape(), **kw) == mk.MK_ERR_INVALID_ARG
    assert attend(None) == mk.MK_ERR_INVALID_ARG


def verify(kw_shape=None, **kw):
    s = dict(dtype=mk.MK_FP32, B=2, n=8, vocab=1000, t_seq=8000, t_node=1000, d_seq=8000, d_node=1000)
    s.update(kw_shape or {})
    a = dict(target=OK, draft=OK, tokens=OK, parents=OK, n_nodes=None, u=OK, r=OK, temperature=None,
             draft_temperature=None, path=OK, n_path=OK, next_token=OK, workspace=OK)
    a.update(kw)
    return mk._lib.mk_tree_verify(ctypes.byref(mk.mk_verify_shape(**s)), *a.values(), None)


@pytest.mark.parametrize("kw", [dict(dtype=3), dict(B=0), dict(n=0), dict(n=257), dict(vocab=0), dict(vocab=(1 << 20) + 1),
                                dict(B=70000, n=1), dict(t_seq=-1), dict(t_node=-8), dict(d_node=-1)])
def test_tree_verify_shapes(kw):
    assert verify(kw) == mk.MK_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(target=None), dict(tokens=None), dict(parents=None), dict(u=None), dict(r=None),
                                dict(path=None), dict(n_path=None), dict(next_token=None), dict(workspace=None),
                                dict(workspace=OK + 8), dict(target=OK + 2), dict(draft=OK + 1)])
def test_tree_verify_operands(kw):
    assert verify(**kw) == mk.MK_ERR_INVALID_ARG


def test_verify_workspace():
    assert mk.mk_tree_verify_workspace_bytes(0, 4, 10) == 0 == mk.mk_tree_verify_workspace_bytes(1, 257, 10)
    assert mk.mk_tree_verify_workspace_bytes(2, 8, 50257) >= 2 * 2 * 8 * 7 * 12


def cache_shape(**kw):
    f = dict(n_layers=2, max_batch=4, B=3, n_kv_heads=2, max_seq=64, head_dim=64)
    f.update(kw)
    return ctypes.byref(mk.mk_cache_shape(**f))


@pytest.mark.parametrize("kw", [dict(n_layers=0), dict(B=0), dict(B=5), dict(n_kv_heads=0), dict(max_seq=0),
                                dict(head_dim=80)])
def test_cache_shapes(kw):
    assert mk._lib.mk_cache_commit(cache_shape(**kw), OK, OK, 4, OK, OK, 2 * OK, None) == mk.MK_ERR_INVALID_ARG
    assert mk._lib.mk_cache_reorder(cache_shape(**kw), OK, OK, OK, 2 * OK, None) == mk.MK_ERR_INVALID_ARG


def test_cache_operands():
    bad = mk.MK_ERR_INVALID_ARG
    assert mk._lib.mk_cache_commit(cache_shape(), OK + 8, OK, 4, OK, OK, 2 * OK, None) == bad
    assert mk._lib.mk_cache_commit(cache_shape(), OK, OK, 257, OK, OK, 2 * OK, None) == bad
    assert mk._lib.mk_cache_commit(cache_shape(), OK, None, 4, OK, OK, 2 * OK, None) == bad
    assert mk._lib.mk_cache_commit(cache_shape(), OK, OK, 4, OK, OK, OK + 8, None) == bad  # new_lens over lens
    assert mk._lib.mk_cache_reorder(cache_shape(), OK, OK, OK, OK, None) == bad
    assert mk._lib.mk_cache_reorder(cache_shape(), OK, None, OK, 2 * OK, None) == bad
    assert mk._lib.mk_cache_reorder(cache_shape(max_batch=20, B=17), OK, OK, OK, 2 * OK, None) == bad
    assert mk._lib.mk_cache_reorder(None, OK, OK, OK, 2 * OK, None) == bad


def test_new_lens_over_an_input():
    bad = mk.MK_ERR_INVALID_ARG
    far = [OK, 2 * OK, 3 * OK, 4 * OK]  # path, n_path, lens, new_lens
    for at, size in ((0, 3 * 4 * 4), (1, 12), (2, 12)):
        for end in (0, size - 4):
            a = list(far)
            a[3] = a[at] + end
            assert mk._lib.mk_cache_commit(cache_shape(), OK, a[0], 4, *a[1:], None) == bad
            assert "overlap" in mk.mk_last_error()
    for at in (OK, 2 * OK):  # src, lens
        for end in (-8, 0, 8):
            assert mk._lib.mk_cache_reorder(cache_shape(), OK, OK, 2 * OK, at + end, None) == bad


def refused(f, *a):
    with pytest.raises(mk.MkError) as e:
        f(*a)
    assert e.value.code == mk.MK_ERR_INVALID_ARG


def test_binding_refuses_tensors_that_do_not_fit():
    q, k = torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 32, 64, dtype=torch.bfloat16)
    par, ln = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    refused(mk.mk_tree_attention, q, k, k, q.clone(), par, None, ln, 0.1)          # not on a GPU
    refused(mk.mk_tree_attention, q, k.half(), k, q.clone(), par, None, ln, 0.1)   # types
    refused(mk.mk_tree_attention, q, k[..., :32], k[..., :32], q.clone(), par, None, ln, 0.1)
    refused(mk.mk_tree_attention, q, k, k[:, :1], q.clone(), par, None, ln, 0.1)
    refused(mk.mk_tree_attention, q.transpose(2, 3), k, k, q.transpose(2, 3), par, None, ln, 0.1)
    refused(mk.mk_tree_attention, q.double(), k, k, q.clone(), par, None, ln, 0.1)
    refused(mk.mk_tree_attention, q.float(), k, k, q.clone(), par, None, ln, 0.1)
    refused(mk.mk_tree_attention, q.float(), k.float(), k.float(), q.float(), par, None, ln, 0.1)
    t = torch.zeros(2, 4, 100)
    f, one = torch.zeros(2, 4), torch.zeros(2)
    out = [torch.zeros(2, 4, dtype=torch.int32), ln.clone(), ln.clone()]
    small = torch.zeros(8, dtype=torch.uint8)
    refused(mk.mk_tree_verify, t, None, par, par, None, f, one, None, None, *out, small)
    room = torch.zeros(mk.mk_tree_verify_workspace_bytes(2, 4, 100), dtype=torch.uint8)
    refused(mk.mk_tree_verify, t, t[:, :2], par, par, None, f, one, None, None, *out, room)
    refused(mk.mk_tree_verify, t, None, par, par, None, f, one, None, None, *out, room)  # not on a GPU
    kv = torch.zeros(2, 2, 3, 2, 16, 64, dtype=torch.int16)
    refused(mk.mk_cache_commit, kv, par, ln, ln, ln.clone())
    refused(mk.mk_cache_commit, kv.transpose(0, 1), par, ln, ln, ln.clone())
    refused(mk.mk_cache_reorder, kv.float(), ln, ln, ln.clone())


def test_tree_forward_refusals():
    import mk_inputs as mi
    assert mk._lib.mk_tree_forward(None, OK, OK, None, OK, 1, 4, OK, OK, None) == mk.MK_ERR_INVALID_ARG
    ctx = mk.mk_build_taskgraph(mk.Config.from_shape(mi.TINY, 2, 64).c(), -1)
    try:
        assert mk._lib.mk_tree_forward(ctx, OK, OK, None, OK, 1, 4, OK, OK, None) == mk.MK_ERR_STATE
    finally:
        mk.mk_destroy(ctx)
