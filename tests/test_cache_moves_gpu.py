"""mk_cache_commit and mk_cache_reorder: copies, compared bit for bit with plain indexing."""
import numpy as np
import pytest
import torch

import persistent_megakernel_decode_04_b200 as mk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def cache(L, B, hkv, S, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-2**15, 2**15, (L, 2, B, hkv, S, d), generator=g, dtype=torch.int16)


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def commit(kv, path, n_path, lens):
    k, new = kv.to(DEV), torch.full((lens.shape[0],), -9, dtype=torch.int32, device=DEV)
    mk.mk_cache_commit(k, path.to(DEV), n_path.to(DEV), lens.to(DEV), new)
    return k.cpu(), new.cpu()


def commit_plain(kv, path, n_path, lens):
    kv, new, S, n = kv.clone(), lens.clone(), kv.shape[4], path.shape[1]
    for b in range(lens.shape[0]):
        ln, last, rows = min(max(int(lens[b]), 0), S), -1, []
        for j in range(min(max(int(n_path[b]), 0), n)):
            x = int(path[b, j])
            if x <= last or x >= n or ln + x >= S:
                break
            rows.append(ln + x)
            last = x
        kv[:, :, b, :, ln:ln + len(rows)] = kv[:, :, b, :, rows].clone()
        new[b] = ln + len(rows)
    return kv, new


@pytest.mark.parametrize("L,B,mb,hkv,S,d,n", [(1, 1, 1, 1, 40, 64, 1), (2, 3, 4, 2, 300, 128, 13), (3, 2, 2, 3, 700, 64, 256),
                                              (1, 2, 2, 1, 600, 128, 256), (5, 16, 16, 8, 64, 128, 33)])
@pytest.mark.parametrize("keep", ["all", "some", "last", "one"])
def test_commit(L, B, mb, hkv, S, d, n, keep):
    rng = np.random.default_rng(n)
    kv = cache(L, mb, hkv, S, d, seed=n)
    path, n_path = torch.full((B, n), -1, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        rows = {"all": np.arange(n), "some": np.nonzero(rng.random(n) < 0.5)[0], "last": np.arange(n // 2, n),
                "one": np.array([n - 1])}[keep]
        path[b, :len(rows)] = torch.from_numpy(rows.astype(np.int32))
        n_path[b] = len(rows)
    lens = torch.from_numpy(rng.integers(0, S - n + 1, B).astype(np.int32))
    lens[0] = S - n  # filled to the last row
    got, want = commit(kv, path, n_path, lens), commit_plain(kv, path, n_path, lens)
    assert torch.equal(got[1], want[1]) and torch.equal(got[0], want[0])


def test_commit_ends_a_path_at_the_first_bad_entry():
    kv = cache(2, 9, 2, 64, 64, seed=1)
    path = i32([[0, 2, 3, -1], [0, 2, 2, 3], [1, 0, 2, 3], [0, 1, 4, 5], [-1, 0, 1, 2], [0, 3, 2**31 - 1, 3],
                [0, 1, 2, 3], [0, 2, 3, 3], [2, 3, 3, 3]])
    n_path = i32([3, 4, 4, 4, 4, 4, 99, 4, -4])
    lens = i32([10, 10, 10, 10, 10, 10, 62, 99, 5])
    got, want = commit(kv, path, n_path, lens), commit_plain(kv, path, n_path, lens)
    assert torch.equal(got[1], want[1]) and torch.equal(got[0], want[0])
    assert got[1].tolist() == [13, 12, 11, 12, 10, 12, 64, 64, 5]
    lens = i32([-3] * 9)
    got, want = commit(kv, path, n_path, lens), commit_plain(kv, path, n_path, lens)
    assert torch.equal(got[1], want[1]) and torch.equal(got[0], want[0])


def reorder(kv, src, lens):
    k, new = kv.to(DEV), torch.full((lens.shape[0],), -9, dtype=torch.int32, device=DEV)
    mk.mk_cache_reorder(k, src.to(DEV), lens.to(DEV), new)
    return k.cpu(), new.cpu()


def reorder_plain(kv, src, lens):
    out, new, S = kv.clone(), lens.clone(), kv.shape[4]
    B = lens.shape[0]
    for b in range(B):
        s = int(src[b])
        s = s if 0 <= s < B else b
        ln = min(max(int(lens[s]), 0), S)
        out[:, :, b, :, :ln] = kv[:, :, s, :, :ln]
        new[b] = ln
    return out, new


@pytest.mark.parametrize("src", [[0], [0, 0], [1, 0], [0, 1, 2], [2, 0, 1], [0, 0, 0, 0], [3, 3, 1, 1], [1, -1, 99, 0],
                                 [(i * 7 + 3) % 16 for i in range(16)], [i // 2 for i in range(16)],
                                 [15 - i for i in range(16)], [5] * 16, [0, 0, 5, 5, 5, 5, 9, 9, 9, 9, 9, 1, 1, 2, 2, 3]])
@pytest.mark.parametrize("L,hkv,S,d", [(2, 2, 37, 64), (1, 3, 300, 128)])
def test_reorder(src, L, hkv, S, d):
    B = len(src)
    rng = np.random.default_rng(B)
    kv = cache(L, B + 1, hkv, S, d, seed=B)
    lens = torch.from_numpy(rng.integers(0, S + 1, B).astype(np.int32))
    got, want = reorder(kv, i32(src), lens), reorder_plain(kv, i32(src), lens)
    assert torch.equal(got[1], want[1]) and torch.equal(got[0], want[0])


def test_reorder_lengths_out_of_range():
    kv = cache(2, 3, 2, 30, 64, seed=2)
    src, lens = i32([1, 2, 0]), i32([-4, 1000, 30])
    got, want = reorder(kv, src, lens), reorder_plain(kv, src, lens)
    assert torch.equal(got[1], want[1]) and torch.equal(got[0], want[0])


def test_large_cache_beyond_32_bit_offsets():
    # 2.3e9 values: the last sequence's planes start beyond 2^31 elements
    L, B, hkv, S, d = 3, 3, 2, 500_000, 128
    kv = torch.zeros(L, 2, B, hkv, S, d, dtype=torch.int16, device=DEV)
    kv[L - 1, 1, 2, 1, S - 5:] = torch.arange(5 * d, dtype=torch.int16, device=DEV).view(5, d)
    kv[L - 1, 1, 2, 1, 7] = 3
    row = kv[L - 1, 1, 2, 1, S - 2].clone()
    new = torch.zeros(B, dtype=torch.int32, device=DEV)
    mk.mk_cache_commit(kv, i32([[0, 1], [0, 1], [1, 2]]).to(DEV), i32([2, 2, 1]).to(DEV), i32([0, 5, S - 3]).to(DEV), new)
    assert new.tolist() == [2, 7, S - 2] and torch.equal(kv[L - 1, 1, 2, 1, S - 3], row)
    mk.mk_cache_reorder(kv, i32([2, 1, 2]).to(DEV), i32([0, 0, S]).to(DEV), new)
    assert new.tolist() == [S, 0, S]
    assert torch.equal(kv[:, :, 0], kv[:, :, 2]) and kv[L - 1, 1, 0, 1, 7, 0] == 3 and (kv[:, :, 1] == 0).all()


def test_graph_replays_with_new_contents():
    kv = cache(2, 2, 2, 50, 64, seed=3)
    k, new = kv.to(DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    path, n_path, lens = i32([[0, 2, 4, 5, 6, 7], [3, 5, -1, 0, 0, 0]]).to(DEV), i32([6, 2]).to(DEV), i32([11, 40]).to(DEV)
    src = i32([1, 0]).to(DEV)
    new2 = torch.zeros(2, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mk.mk_cache_commit(k, path, n_path, lens, new, torch.cuda.current_stream())
        mk.mk_cache_reorder(k, src, new, new2, torch.cuda.current_stream())
    k.copy_(kv)
    path.copy_(i32([[1, 2, 5, -1, -1, -1], [0, 1, 2, 3, 4, 5]]))
    n_path.copy_(i32([3, 6]))
    lens.copy_(i32([30, 9]))
    graph.replay()
    a, mid = commit_plain(kv, path.cpu(), n_path.cpu(), lens.cpu())
    want, end = reorder_plain(a, src.cpu(), mid)
    assert torch.equal(k.cpu(), want) and torch.equal(new.cpu(), mid) and torch.equal(new2.cpu(), end)
