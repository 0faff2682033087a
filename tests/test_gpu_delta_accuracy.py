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


def walk(q, k, v, beta, gate, grad_o, grad_state, scale):
    """Per head, the largest of ||S_t|| and |v_t|, and of ||dS_t|| and |dO_t|."""
    group = v.shape[2] // q.shape[2]
    q, k = (x.double().repeat_interleave(group, dim=2) for x in (q, k))
    v, beta, a, do = v.double(), beta.double(), gate.double().exp(), grad_o.double()
    top, dtop = v.norm(dim=-1).amax(1), do.norm(dim=-1).amax(1)
    S = torch.zeros_like(grad_state, dtype=torch.float64)
    dS = grad_state.double()
    for t in range(v.shape[1]):
        S = a[:, t, :, None, None] * S
        w = v[:, t] - (S * k[:, t, :, :, None]).sum(2)
        S = S + k[:, t, :, :, None] * (beta[:, t, :, None] * w)[:, :, None, :]
        top = torch.maximum(top, S.norm(dim=(2, 3)))
    for t in reversed(range(v.shape[1])):
        dS = dS + scale * q[:, t, :, :, None] * do[:, t, :, None, :]
        dtop = torch.maximum(dtop, dS.norm(dim=(2, 3)))
        dw = beta[:, t, :, None] * (dS * k[:, t, :, :, None]).sum(2)
        dS = a[:, t, :, None, None] * (dS - k[:, t, :, :, None] * dw[:, :, None, :])
    return top, dtop


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,Hk,Hv,dk,dv", [(60, 1, 2, 40, 48), (150, 2, 4, 128, 64), (130, 2, 2, 64, 33)])
def test_gate_gradients_of_strong_decays(hip, dtype, T, Hk, Hv, dk, dv):
    """Every token's own gradient where strong decays stand among weak ones.

    The gate's gradient is a_t <dS, S_(t-1)> (after and before the token): a_t times
    inner products of what the passes carry, each good to 1.5e-6 for a chunk, the
    two passes together twice that.  A difference of sums that lack a_t would be
    off by 1e-7 of their size, for a gate of -20 the gradient's size 50 times."""
    banner(f"gate gradients {dtype} {T} {Hk} {Hv} {dk} {dv}")
    g = torch.Generator(device=DEV).manual_seed(22)
    randn = lambda *s: torch.randn(s, generator=g, device=DEV)
    B, norm = 2, torch.nn.functional.normalize
    c = dict(q=norm(randn(B, T, Hk, dk), dim=-1).to(dtype), k=norm(randn(B, T, Hk, dk), dim=-1).to(dtype),
             v=randn(B, T, Hv, dv).to(dtype), beta=torch.sigmoid(randn(B, T, Hv)),
             gate=-0.1 * randn(B, T, Hv).abs())
    strong = torch.tensor([-8.0, -12.0, -16.0, -20.0], device=DEV)
    pick = torch.randint(0, 24, (B, T, Hv), generator=g, device=DEV)
    c["gate"] = torch.where(pick < 4, strong[pick.clamp(max=3)], c["gate"])
    c["gate"][0, :, 0] = -16.0          # and a head of strong decays alone
    go, gs = randn(B, T, Hv, dv).to(dtype), randn(B, Hv, dk, dv)
    gate = c["gate"].clone().requires_grad_()
    o, S = hip.delta_rule(**{**c, "gate": gate}, scale=1.0)
    (got,) = torch.autograd.grad([o, S], gate, [go, gs])
    want = OD.rule_adjoint(**c, grad_o=go, grad_state=gs, scale=1.0)["gate"]
    top, dtop = walk(**c, grad_o=go, grad_state=gs, scale=1.0)
    bound = 2 * 1.5e-6 * (T // 64 + 2) * c["gate"].double().exp() * (top * dtop)[:, None]
    off = (got.double() - want).abs()
    print("off / bound", float((off / bound).max()), "strong", float((off / bound)[pick < 4].max()))
    assert (off <= bound).all()
