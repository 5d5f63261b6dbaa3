"""A gradient at the logits that shares some of the logits' memory without being them is refused; one
that lies between their rows, or is them, is right."""
import ctypes

import pytest
import torch

BF16, F32, EINVAL = 3, 1, -1
AT = 1 << 20
D = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def lib():
    from loss_scaling_master_gb300 import build as B
    B.build()
    from loss_scaling_master_gb300 import ops
    return ops._load()


def shares(rows, cols, ld, dld, off):
    """By looking at every element."""
    z = {r * ld + c for r in range(rows) for c in range(cols)}
    return any(off + r * dld + c in z for r in range(rows) for c in range(cols))


# rows, cols, stride of z, of dz, elements from z's start to dz's
SHARED = [(4, 8, 8, 8, 1), (4, 8, 8, 8, -1), (4, 8, 8, 8, 8), (4, 8, 8, 8, 31), (4, 8, 8, 8, -31), (1, 8, 8, 8, 7),
          (1, 8, 20, 9, -7), (4, 8, 20, 20, 7), (4, 8, 20, 20, 13), (4, 8, 20, 20, 53), (4, 8, 20, 20, 60),
          (4, 8, 20, 20, -13), (4, 8, 20, 8, 4), (4, 8, 8, 20, 3), (3, 5, 5, 7, 10)]


@pytest.mark.parametrize("dt,size", [(BF16, 2), (F32, 4)])
@pytest.mark.parametrize("rows,cols,ld,dld,off", SHARED)
def test_shared_elements_are_refused(lib, dt, size, rows, cols, ld, dld, off):
    assert shares(rows, cols, ld, dld, off)
    z, dz = ctypes.c_void_p(AT), ctypes.c_void_p(AT + off * size)    # never dereferenced: refused
    assert lib.amp_token_logprobs_backward(D, z, dt, rows, cols, ld, D, D, D, D, D, dz, dld, None) == EINVAL
    assert b"overlaps" in lib.amp_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_between_one_another(lib, dtype):
    """Column slices of one buffer, on either side, the last row's ends meeting; ranges that touch."""
    import loss_scaling_master_gb300 as G
    buf = torch.randn(5, 100, device="cuda").to(dtype)
    t = torch.tensor([3, 0, -1, 49, 7], device="cuda")
    for left, right in (((0, 50), (50, 100)), ((50, 100), (0, 50)), ((0, 33), (40, 73)), ((67, 100), (0, 33))):
        b = buf.clone()
        z, dz = b[:, slice(*left)], b[:, slice(*right)]
        tt = t.clamp(max=z.shape[1] - 1)
        logp, stats, dlogp = torch.empty(5, device="cuda"), torch.empty(5, 2, device="cuda"), torch.ones(5, device="cuda")
        G.amp_token_logprobs_forward(z, tt, logp, stats=stats)
        apart = torch.empty(5, z.shape[1], dtype=dtype, device="cuda")
        G.amp_token_logprobs_backward(dlogp, z, tt, stats, apart)
        G.amp_token_logprobs_backward(dlogp, z, tt, stats, dz)
        assert torch.equal(dz, apart)
        b[:, slice(*right)] = buf[:, slice(*right)]
        assert torch.equal(b, buf)                      # and nothing else was written
    flat = torch.randn(10, 50, device="cuda").to(dtype)
    z, dz = flat[5:], flat[:5]
    want = torch.empty_like(dz)
    G.amp_token_logprobs_forward(z, t, logp, stats=stats)
    G.amp_token_logprobs_backward(dlogp, z, t, stats, want)
    G.amp_token_logprobs_backward(dlogp, z, t, stats, dz)
    assert torch.equal(dz, want)
