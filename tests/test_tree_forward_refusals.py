"""What Megakernel.tree_forward refuses, on the CPU: nothing is launched."""
import pytest
import torch

import mk_inputs as mi
import persistent_megakernel_decode_04_b200 as mk


def test_tensors_that_are_not_on_the_models_device():
    m = mk.Megakernel.__new__(mk.Megakernel)  # a context without a device; nothing is allocated
    m.cfg, m.device, m.stream = mk.Config.from_shape(mi.TINY, 2, 64), 0, None
    m.kv = torch.zeros(8, dtype=torch.int16)
    m.ctx = mk.mk_build_taskgraph(m.cfg.c(), -1)
    ids, lens = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for n_nodes in (None, lens):
        with pytest.raises(mk.MkError) as e:
            m.tree_forward(ids, ids, lens, n_nodes)
        assert e.value.code == mk.MK_ERR_INVALID_ARG and "cuda:0" in str(e.value)
    mk.mk_destroy(m.ctx)
    m.ctx = None
