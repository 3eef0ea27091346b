"""The scratch of a matrix product that runs no backward."""
import os

import pytest
import torch

# T, K, N, fp32 or bf16: few rows, the tiles with and without shares, odd widths on them and off them, the general kernel
SIZES = [(1, 2048, 768, 1), (4, 300, 9, 0), (3, 70, 7, 0), (16, 2048, 768, 1), (40, 4096, 64, 1), (300, 777, 1555, 1),
         (1000, 1001, 520, 1), (1000, 520, 1001, 1), (60, 301, 129, 1), (1003, 769, 333, 0), (300, 4000, 64, 0), (16384, 1536, 4096, 1)]


def _shape(size, act):
    from combine_top_router_amd import lib as L
    if not os.path.exists(L.lib_path()):
        pytest.skip("libmoe.so not built")
    T, K, N, dtype = size
    return L, L.MoeLinearShape(T, K, N, dtype, act)


@pytest.mark.parametrize("act", [0, 1, 3])
@pytest.mark.parametrize("size", SIZES + [(0, 8, 8, 1), (2 ** 31 - 1, 1, 1, 0), (2 ** 31 - 1, 1 << 20, 1 << 20, 1)],
                         ids=lambda s: "x".join(map(str, s)))
def test_forward_scratch_is_a_part(size, act):
    L, s = _shape(size, act)
    n = L.moe_linear_fwd_scratch_bytes(s)
    assert 0 < n <= L.moe_linear_scratch_bytes(s)


def test_forward_scratch_has_no_gradients():
    L, s = _shape((16384, 1536, 4096, 1), 2)
    assert L.moe_linear_fwd_scratch_bytes(s) < 16384 * 4096 * 2   # less than dz alone
    from combine_top_router_amd import Linear
    op = Linear(64, 128, 256, act=2, train=False, device="cpu")
    assert op.scratch.numel() == L.moe_linear_fwd_scratch_bytes(op.shape) < Linear(64, 128, 256, act=2, device="cpu").scratch.numel()
    with pytest.raises(L.MoeError) as e:
        L.moe_linear_fwd_scratch_bytes(L.MoeLinearShape(4, 0, 4, 1, 0))
    assert e.value.code == L.MOE_EINVAL


@pytest.mark.gpu
@pytest.mark.parametrize("act", [1, 2])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_forward_stays_in_its_scratch(size, act):
    """The same y and z as with all the scratch, and nothing behind it is written; odd addresses take the general kernel."""
    L, s = _shape(size, act)
    T, K, N, dtype = size
    dt = torch.bfloat16 if dtype else torch.float32
    g = torch.Generator().manual_seed(T + K)
    n, whole = L.moe_linear_fwd_scratch_bytes(s), L.moe_linear_scratch_bytes(s)
    for off in (0, 1):
        def at(*d):
            m = torch.Size(d).numel()
            return (torch.randn(m + off, generator=g) / (K ** 0.5 if d == (K, N) else 1.0)).to(dt).cuda()[off:].view(d)

        x, w, b, res = at(T, K), at(K, N), at(N), at(T, N)
        out = []
        for room in (n, whole):
            ws = torch.full((room + 4096,), 7, dtype=torch.uint8, device="cuda")
            y, z = (torch.zeros(T * N + off, dtype=dt, device="cuda")[off:] for _ in range(2))
            L.moe_linear_fwd(s, x.data_ptr(), w.data_ptr(), b.data_ptr(), res.data_ptr(), z.data_ptr(), y.data_ptr(), ws.data_ptr(),
                             torch.cuda.current_stream().cuda_stream)
            torch.cuda.synchronize()
            assert (ws[room:] == 7).all()
            out.append((y, z))
        assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
