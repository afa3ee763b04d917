"""Which kernels a balance of one sequence runs as: one workgroup up to 65,536
logits, counted by what a row costs its lanes (16 experts at least, then powers
of two up to 512); and long batches of few experts against the oracle, with the bounds of
test_gpu_balance.py."""
import numpy as np
import pytest
import torch

from oracle import moe_balance as ob
from tests import test_gpu_balance as base
from tests.helpers import max_rel_err

pytestmark = pytest.mark.gpu
DEV = "cuda"
B = base.B

CASES = [
    # (T, E, k, one workgroup)
    (64, 8, 2, True),
    (4096, 8, 2, True),
    (4097, 8, 2, False),
    (8192, 8, 2, False),
    (16384, 4, 2, False),
    (32768, 2, 1, False),
    (65536, 1, 1, False),
    (1024, 40, 3, True),
    (1500, 40, 3, False),
    (256, 130, 4, True),
    (400, 160, 4, False),
    (64, 1024, 4, True),
    (80, 805, 4, True),
    (82, 805, 4, False),
]


@pytest.mark.parametrize("T,E,k,one", CASES)
def test_kernels_of_a_balance(B, T, E, k, one):
    print(f"case balance dispatch T={T} E={E}", flush=True)
    z, idx, _, mask = base._inputs(T, E, k, 1, 0, 0.1, 0, T + E)
    buf = B.BalanceBuffers.allocate(B.make_shape(T, 256, 128, E, k))
    base._poison(buf)
    B.moe_set_kernel_timing(True)
    try:
        B.balance(buf, z, idx, None, mask)
        torch.cuda.synchronize()
        names = set(B.moe_kernel_timing_collect())
    finally:
        B.moe_set_kernel_timing(False)
    assert names == ({"balance_small"} if one else {"balance_partial", "balance_seq", "balance_finish"})
    ref = ob.balance(*(t.cpu().numpy() for t in (z, idx)), None, mask.cpu().numpy())
    assert np.array_equal(buf.counts.cpu().numpy(), ref["counts"])
    for name in ("loss", "seq_probs", "seq_scale"):
        assert max_rel_err(getattr(buf, name).cpu().numpy(), ref[name]) <= base.TOL, name
