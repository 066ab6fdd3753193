"""A Megakernel on a stream of its own, or called from a stream that is not its own: inputs made late
and results used at once."""
import numpy as np
import pytest
import torch

import mk_inputs as mi
import persistent_megakernel_decode_04_b200 as mk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
LATE = 40_000_000  # cycles: 20 ms


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def model(stream, max_batch=2):
    w = mi.make_weights(mi.TINY, seed=5)
    m = mk.Megakernel(mk.Config.from_shape(w.shape, max_batch, 64), w, 0, stream=stream)
    g = torch.Generator().manual_seed(1)
    cache = torch.randn(m.kv_view().shape, generator=g).bfloat16().to(DEV).view(torch.int16)
    torch.cuda.synchronize()
    m.kv_view().copy_(cache)
    torch.cuda.synchronize()
    return m


def speculate(m, ready, late=lambda: None):
    """Forward, commit and reorder, each behind inputs that `late` holds up; copies of the results."""
    t = {key: torch.zeros_like(val) for key, val in ready.items()}
    out = []
    for step in range(3):
        late()
        for key, val in ready.items():
            t[key].copy_(val)
        if step == 0:
            got = m.tree_forward(t["tokens"], t["parents"], t["lens"])
        elif step == 1:
            got = m.commit(t["path"], t["n_path"], t["lens"])
        else:
            got = m.reorder(t["src"], t["lens"])
        out.append(got.clone())  # on the current stream, at once
        out.append(m.kv_view().clone())
        del got
        for val in t.values():
            val.zero_()
    return out


@pytest.mark.parametrize("own,current", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("busy", ["own", "current"])
def test_speculative_calls_are_in_order_with_the_current_stream(own, current, handle, busy):
    rng = np.random.default_rng(3)
    ready = dict(tokens=i32(rng.integers(0, 500, (2, 4))), parents=i32([[-1, 0, 1, 1]] * 2), lens=i32([20, 33]),
                 path=i32([[0, 2, 3, -1]] * 2), n_path=i32([3, 2]), src=i32([1, 0]))
    m = model(None)
    want = speculate(m, ready)
    torch.cuda.synchronize()
    m.close()
    s = torch.cuda.Stream() if own else None
    m = model(s.cuda_stream if own and handle else s)
    here = torch.cuda.Stream() if current else torch.cuda.default_stream()
    torch.cuda.synchronize()

    def late():
        with torch.cuda.stream(here if busy == "current" else s or torch.cuda.default_stream()):
            torch.cuda._sleep(LATE)

    with torch.cuda.stream(here):
        got = speculate(m, ready, late)
    here.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    assert m.sync_status() == mk.MK_OK and mk.mk_tree_attention_status() == mk.MK_OK
    m.close()


@pytest.mark.parametrize("handle", [False, True])
def test_decode_steps_writes_no_memory_that_the_current_stream_still_uses(handle):
    s, here, n = torch.cuda.Stream(), torch.cuda.Stream(), 3
    want = None
    for stream in (None, s.cuda_stream if handle else s):
        m = model(stream)
        m.set_positions([20, 20])
        tokens = i32([3, 500])
        torch.cuda.synchronize()
        with torch.cuda.stream(here):
            torch.cuda._sleep(LATE)
            x = torch.empty((n, 2), dtype=torch.int32, device=DEV)
            x.fill_(-7)  # when the steps are long done
            del x
            picks = m.decode_steps(tokens, n)[1]
        assert m.sync_status() == mk.MK_OK
        torch.cuda.synchronize()
        want = picks.clone() if want is None else want
        assert (picks >= 0).all() and torch.equal(picks, want)
        m.close()
