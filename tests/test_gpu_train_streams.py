"""Results that the training operators and the layer allocate themselves belong to the stream
that the call is given: memory that work queued on the current stream still
uses is not handed to another stream's kernels."""
import pytest
import torch

from tests import test_gpu_ortho as base

pytestmark = pytest.mark.gpu
DEV = "cuda"
B = base.B


def _freed_block(shape, dtype):
    """Address of a block that the current stream's next allocation would take."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    t = torch.empty(shape, dtype=dtype, device=DEV)
    p = t.data_ptr()
    del t
    again = torch.empty(shape, dtype=dtype, device=DEV)
    assert again.data_ptr() == p
    del again
    return p


@pytest.mark.parametrize("as_handle", [False, True])
def test_orthogonalize_allocates_on_its_stream(B, as_handle):
    E, R, C = 3, 700, 900
    G = base._grad(E, R, C, "bf16", 1, rank=50)
    buf = B.OrthoBuffers.allocate(B.make_ortho_shape(E, R, C))
    want = B.orthogonalize(buf, G).clone()
    side = torch.cuda.Stream()
    p = _freed_block((E, R, C), torch.bfloat16)
    side.wait_stream(torch.cuda.current_stream())
    U = B.orthogonalize(buf, G, stream=side.cuda_stream if as_handle else side)
    assert U.data_ptr() != p
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(U, want)
    p = _freed_block((E, R, C), torch.bfloat16)
    assert B.orthogonalize(buf, G).data_ptr() == p   # the current stream's own block


@pytest.mark.parametrize("as_handle", [False, True])
def test_balance_bwd_allocates_on_its_stream(B, as_handle):
    T, E, k = 5000, 200, 4
    z = torch.randn((T, E), generator=torch.Generator(device=DEV).manual_seed(2), device=DEV)
    idx = torch.topk(z, k, dim=1)[1].to(torch.int32).contiguous()
    dl = torch.ones(2, device=DEV)
    buf = B.balance(B.BalanceBuffers.allocate(B.make_shape(T, 256, 128, E, k)), z, idx)
    want = B.balance_bwd(buf, z, None, None, None, True, dl).clone()
    side = torch.cuda.Stream()
    p = _freed_block((T, E), torch.float32)
    side.wait_stream(torch.cuda.current_stream())
    d = B.balance_bwd(buf, z, None, None, None, True, dl, stream=side.cuda_stream if as_handle else side)
    assert d.data_ptr() != p
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(d, want)


def test_layer_allocates_on_its_stream(B):
    T, H, I, E, k = 300, 512, 128, 8, 2
    g = torch.Generator(device=DEV).manual_seed(3)
    n = lambda *sz: torch.randn(sz, generator=g, device=DEV).bfloat16()  # noqa: E731
    x, dy, W13, W2 = n(T, H), n(T, H), 0.05 * n(E, 2 * I, H), 0.05 * n(E, H, I)
    w, idx = torch.topk(torch.rand((T, E), generator=g, device=DEV), k, dim=1)
    idx = idx.to(torch.int32).contiguous()
    buf = B.LayerBuffers.allocate(B.make_shape(T, H, I, E, k))
    y = B.forward(buf, x, idx, w, W13, W2).clone()
    grads = [t.clone() for t in B.backward(buf, dy, x, idx, w, W13, W2)]
    side = torch.cuda.Stream()
    p = _freed_block((T, H), torch.bfloat16)
    side.wait_stream(torch.cuda.current_stream())
    got = B.forward(buf, x, idx, w, W13, W2, stream=side)
    assert got.data_ptr() != p
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, y)
    p = _freed_block((E, 2 * I, H), torch.bfloat16)
    side.wait_stream(torch.cuda.current_stream())
    got = B.backward(buf, dy, x, idx, w, W13, W2, stream=side)
    assert p not in [t.data_ptr() for t in got]
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, grads):
        assert torch.equal(a, b)


def test_results_outlive_the_current_streams_work(B):
    """A result of another stream, freed while the current stream still reads
    it, is not handed out again by its own stream before that."""
    E, R, C = 4, 1024, 1024
    G = base._grad(E, R, C, "bf16", 4, rank=50)
    buf = B.OrthoBuffers.allocate(B.make_ortho_shape(E, R, C))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    U = B.orthogonalize(buf, G, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    a = torch.randn((4096, 4096), device=DEV)
    for _ in range(20):
        a = (a @ a).clamp_(-1, 1)     # keeps the current stream busy
    U.mul_(1.0)
    p = U.data_ptr()
    del U
    with torch.cuda.stream(side):
        other = torch.empty((E, R, C), dtype=torch.bfloat16, device=DEV)
    assert other.data_ptr() != p
    torch.cuda.synchronize()
