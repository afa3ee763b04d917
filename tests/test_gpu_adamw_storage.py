"""The tensors of an AdamW step where their storage, type or strides change between steps."""
import numpy as np
import pytest
import torch

from oracle import moe_adamw as oa

pytestmark = pytest.mark.gpu
DEV = "cuda"
H = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from grouped_gemm_02_amd import binding
    binding.lib()
    return binding


def _rand(*size, seed=0):
    return torch.randn(size, generator=torch.Generator().manual_seed(seed)).to(DEV)


def test_another_view_of_a_parameters_memory_is_refused(B):
    """The same address and as many elements, but other strides or another type: a step over the
    memory's order would pair elements with others' gradients."""
    for dtype, other in ((torch.float32, torch.int32), (torch.bfloat16, torch.float16)):
        p = _rand(24, 40).to(dtype)
        q = _rand(100, seed=1).to(dtype)
        buf = B.AdamWBuffers.allocate([q, p])
        whole, keep = p.data, p.clone()
        keep_q = q.clone()
        for bad in (whole.t(), whole.view(other)):
            p.data = bad
            assert p.data_ptr() == whole.data_ptr() and p.numel() == whole.numel()
            with pytest.raises(B.MoEError) as ei:
                B.adamw_step(buf, [_rand(100), _rand(*p.shape)], step=1, **H)
            assert ei.value.status == 2
            assert torch.equal(whole, keep) and torch.equal(q, keep_q)
        p.data = whole
        B.adamw_step(buf, [_rand(100), _rand(24, 40)], step=1, **H)
        assert not torch.equal(p, keep)
