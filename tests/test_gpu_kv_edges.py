"""The key/value cache's calls at their edges: tables shorter than a length, values
that no rotation touches, roundings, rows far apart in size, sizes at the limits."""

import numpy as np
import pytest
import torch

from oracle import kvcache as kv
from tests.gpu_common import require_gpu, say
from tests.kv_common import FMTS, Batch, device_cache, on_gpu, random_tree, rows

pytestmark = pytest.mark.gpu

FD = [(f, d) for f in FMTS for d in (64, 128, 256)]


def _dev(x, dtype):
    return torch.tensor(x, dtype=dtype, device="cuda")


@pytest.mark.parametrize("fmt,d", FD)
@pytest.mark.parametrize("n_q,n_kv,nodes", [(4, 2, 1), (4, 2, 8), (4, 1, 8), (4, 1, 30)])
def test_tables_shorter_than_a_length(fmt, d, n_q, n_kv, nodes):
    """Positions past the table's last column are not read, and the new tokens
    stay the last ones of kv_lens: 2, 16, 32 and 120 rows, whole and split."""
    q = require_gpu()
    say("short table", fmt, d, n_q, n_kv, nodes)
    for lens, cols in (([100, 93], 6), ([100, 60], 5), ([1500, 1300], 81)):
        b = Batch(FMTS[fmt], lens, [nodes] * 2, n_q, n_kv, d, 16, seed=31)
        hidden = [np.arange(max(lens)) >= 16 * cols] * 2
        whole = b.table
        for tree in (None, random_tree([nodes] * 2, 31)):
            want, bound = b.reference(tree, hidden=hidden)
            for table in (whole[:, :cols], np.where(np.arange(whole.shape[1]) < cols, whole, -1).astype(np.int32)):
                b.table = table
                got = b.run(q, tree).double().cpu().numpy()
                b.table = whole
                assert np.all(np.abs(got - want) <= bound)
