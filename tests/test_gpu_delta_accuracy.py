"""The gated delta rule where its terms are far larger than its results, token
by token against the oracle (float64)."""
import pytest
import torch

from gpu_helpers import banner
from oracle import delta as OD

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROUND = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -12, torch.bfloat16: 2.0 ** -9}


def unit_rows(g, *shape):
    """Unit vectors that every type holds exactly: 64 entries of 1/8, signs at random."""
    place = torch.rand(shape, generator=g, device=DEV).argsort(dim=-1) < 64
    sign = torch.randint(0, 2, shape, generator=g, device=DEV) * 2 - 1
    return place * sign * 0.125


def norms(x):
    """2-norms of the heads of [batch, tokens, heads, columns]."""
    return x.square().sum((0, 1, 3)).sqrt()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("save", [False, True])
@pytest.mark.parametrize("size", [3e3, 3e4])
def test_output_where_a_token_reads_what_it_corrects(hip, dtype, save, size):
    """q = k, beta = 1, no gate: o_t is what S_t answers for the row just projected
    on, v_t of size 1, as a difference of two terms of the size of S^T k.

    A product of 24 bits is off by 2^-23 of its terms, and sums of 128 + 64 of them
    in fp32 by sqrt(192) 2^-24 = 8e-7 of the terms' size; with 16 bits they are off
    by 2.5e-6 and more.  The output's rounding comes on top."""
    banner(f"delta output {dtype} save {save} size {size}")
    g = torch.Generator(device=DEV).manual_seed(21)
    B, T, H, dk, dv = 2, 64, 3, 128, 48
    k = unit_rows(g, B, T, H, dk).to(dtype)
    v = torch.randn(B, T, H, dv, generator=g, device=DEV).to(dtype)
    one, zero = torch.ones(B, T, H, device=DEV), torch.zeros(B, T, H, device=DEV)
    state = size * torch.randn(B, H, dk, dv, generator=g, device=DEV)   # so is S^T k
    c = dict(q=k, k=k, v=v, beta=one, gate=zero, state=state)
    if save:
        o = hip.delta_rule(**{**c, "v": v.clone().requires_grad_()}, scale=1.0)[0].detach()
    else:
        with torch.no_grad():
            o = hip.delta_rule(**c, scale=1.0)[0]
    want = OD.rule(**c, scale=1.0)[0]
    terms = (state.double()[:, None] * k.double()[..., None]).sum(3)
    off, bound = norms(o.double() - want), ROUND[dtype] * norms(want) + 8e-7 * norms(terms)
    print("off", off.tolist(), "bound", bound.tolist())
    assert (off <= bound).all()
