"""The codes of the 8-bit moments to the bit: those of m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2 and
sqrt(v) in fp32, each product, sum and root rounded to nearest.  A code is decided by the last bits of such a
number, so a root that is off by one unit in the last place takes another code now and then, and the parameter
follows it from the next step on.  Here the same numbers are formed on the CPU, the root in fp64 and rounded
(torch's own of fp32 is off by a unit there, too)."""
import numpy as np
import pytest
import torch

from oracle import step as os_

pytestmark = pytest.mark.gpu


def _adamw(p, **kw):
    from combine_top_router_amd import AdamW, lib as L
    return AdamW([p], state=L.MOE_STATE_8BIT, **kw)


def _exponents(x):
    """The blocks' scale exponents: the smallest X with max |x| <= 448 2^X, 0 for zeros."""
    amax = x.abs().view(-1, 32).amax(1)
    mant, e = torch.frexp(amax)
    return torch.where(amax > 0, (e - 9 + (mant > 0.875).to(e.dtype)).clamp(-127, 127), 0)


def _codes(x, r16=None, keep=False):
    """(codes as values of their scale, exponents) of fp32 x >= 0 or of either sign."""
    e = _exponents(x)
    y = np.ldexp(x.double().abs().view(-1, 32).numpy(), -e.numpy()[:, None])
    q = os_.e4m3_grid(y, None if r16 is None else r16.reshape(-1, 32))
    if keep:
        q = np.where((y > 0) & (q == 0), 2.0 ** -9, q)
    return np.copysign(q, x.view(-1, 32).numpy()), e


def _got(codes, scale):
    return codes.cpu().view(torch.float8_e4m3fn).double().view(-1, 32).numpy(), scale.cpu().to(torch.int32) - 127


def test_root_of_squares():
    """Numbers halfway between two codes, squared exactly by beta2 = 0: the root is the number, and the code
    the even one of the two."""
    mids = torch.tensor([1 + (2 * i + 1) / 16 for i in range(8)])   # five significant bits
    rows = []
    for e in range(-60, 60):
        b = torch.cat([mids * 2.0 ** k for k in (0, 1, 2)] + [torch.tensor([1.0, 1.5, 7.0, 7.5, 5.0, 3.25, 2.0, 1.125])])
        rows.append(b * 2.0 ** e)
    g = torch.stack(rows).view(-1)
    op = _adamw(torch.zeros(g.numel(), device="cuda"), betas=(0.9, 0.0))
    op.step([g.cuda()], 1e-3)
    want, e = _codes(g, keep=True)
    got, x = _got(op.v, op.v_scale)
    assert torch.equal(x, e.to(torch.int32))
    assert np.array_equal(got, want), np.argwhere(got != want)[:4].tolist()


@pytest.mark.parametrize("stochastic", [False, True])
@pytest.mark.parametrize("g_dtype", [torch.float32, torch.bfloat16])
def test_codes_of_the_formula_in_fp32(g_dtype, stochastic):
    gen = torch.Generator().manual_seed(11)
    n, seed, steps = 1 << 20, 12345, 5
    op = _adamw(torch.zeros(n, device="cuda"), betas=(0.9, 0.95), stochastic=stochastic, seed=seed)
    b1, c1, b2, c2 = (torch.tensor(x) for x in (0.9, 1.0 - 0.9, 0.95, 1.0 - 0.95))
    m, v = torch.zeros(n), torch.zeros(n)
    for t in range(1, steps + 1):
        g = (1e-3 * (0.3 + torch.rand(n // 32, 1, generator=gen)) * torch.randn(n // 32, 32, generator=gen)).view(-1).to(g_dtype)
        op.step([g.cuda()], 1e-3)
        g = g.float()
        m = b1 * m + c1 * g
        s = torch.from_numpy(np.sqrt((b2 * v + c2 * (g * g)).double().numpy()).astype(np.float32))   # (53 bits are enough)
        r = os_.random_bits(seed, t, np.arange(n)) if stochastic else None
        for name, x, r16, codes, scale in (("m", m, None if r is None else r & np.uint64(0xFFFF), op.m, op.m_scale),
                                           ("v", s, None if r is None else r >> np.uint64(16), op.v, op.v_scale)):
            want, e = _codes(x, r16, keep=name == "v")
            got, have = _got(codes, scale)
            assert torch.equal(have, e.to(torch.int32)), (name, t)
            assert np.array_equal(got, want), (name, t, int((got != want).sum()))
            held = torch.from_numpy(np.ldexp(want, e.numpy()[:, None])).float().view(-1)   # exact
            if name == "m":
                m = held
            else:
                v = held * held
