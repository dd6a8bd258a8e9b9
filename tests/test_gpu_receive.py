"""The receive kernel's dense output beside its combination, on the GPU against the oracle, bit for bit, many times over."""
import numpy as np
import pytest
import torch

import compressed_sgd_b200 as gs
import oracle
import synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,entries", [(1 << 20, 900000), ((1 << 18) + 77, 200000), (8192 * 40, 8192 * 40)])
def test_dense_sums_keep_the_own_values_that_leave_the_combination(n, entries):
    """The worker's own values leave the sum before the combination, but not the dense sum, which the same threads write from the same
    shared tile: with crowded tiles some threads are long at the one while others are still at the other."""
    gen = np.random.default_rng(n)
    host, lists, keep = [], [], []
    for w in range(2):
        idx = np.sort(gen.choice(n, entries, replace=False)).astype(np.int32)
        val = synth.gaussian(idx.size, 70 + w, sigma=1e-2)
        t = (torch.from_numpy(idx).cuda(), torch.tensor([idx.size], dtype=torch.int64, device="cuda"), torch.from_numpy(val).cuda())
        keep.append(t)
        host.append((idx, val))
        lists.append(gs.make_list(t[0], t[1], val=t[2], capacity=idx.size))
    local = synth.gaussian(n, 9, sigma=1e-2)
    want_dense, _, _ = oracle.scatter_accumulate(host, n, merged=False)
    want = oracle.combine_local(want_dense, local, 1.0, 1.0, mode=1, own_idx=host[1][0], own_val=host[1][1])
    L, want_dense, want = (torch.from_numpy(a).cuda().view(torch.int32) for a in (local, want_dense, want))
    for _ in range(50):
        st, dense = gs.status_tensor(), torch.empty(n, device="cuda")
        out = gs.accumulate_combine(lists, n, L.view(torch.float32), mode=1, own=1, dense_out=dense, d_status=st)
        assert int(st.item()) == 0
        assert torch.equal(out.view(torch.int32), want) and torch.equal(dense.view(torch.int32), want_dense)
