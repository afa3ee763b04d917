"""AdamW's step at the ends of the range of eps, against the float64 oracle. The update is m
times a rounded step over root + eps, a reciprocal of one unit: 12 roundings, below 1e-6 of it, and two
of 2^-24 of w."""
import numpy as np
import pytest
import torch

from oracle import moe_adamw as oa

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from grouped_gemm_02_amd import binding
    binding.lib()
    return binding


@pytest.mark.parametrize("eps", [2.0 ** -126, 1e-30, 1e-8, 2.0 ** 100])
@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_elements_without_a_gradient_only_decay(B, eps, state):
    """Zeros among the gradients, with moments of zero: 0 / eps is 0; the others' updates are the
    formula's."""
    print(f"case eps {eps} {state}", flush=True)
    n = 1000
    g = torch.randn(n, generator=torch.Generator().manual_seed(1))
    g[::3] = 0
    p = torch.randn(n, generator=torch.Generator().manual_seed(2)).to(DEV)
    old = p.double().cpu().numpy()
    h = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=eps, weight_decay=0.1)
    buf = B.AdamWBuffers.allocate([p], state=state)
    B.adamw_step(buf, [g.to(DEV)], step=1, **h)
    x = g.double().numpy()
    want = oa.step(old, x, 0 * x, 0 * x, t=1, **h)[0]
    tol = 2e-6 * np.abs(want - old) + 3 * 2.0 ** -24 * (np.abs(old) + np.abs(want))
    assert np.all(np.abs(p.double().cpu().numpy() - want) <= tol)
