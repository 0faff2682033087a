"""The gated delta rule's range of gates: growth within it, NaN beyond it for
any length, against the oracle (float64, token by token).

Within a chunk a run of gates may sum to 2.  Terms that grew by e^2 = 7.4 and
cancel again cost that factor in accuracy: 7.4 times the 1.5e-6 a chunk (and
one more) of the rule's products and sums, twice that for gradients."""
import math

import pytest
import torch

from gpu_helpers import banner
from oracle import delta as OD

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def inputs(T, seed, equal=True, B=2, Hk=2, Hv=4, dk=32, dv=40):
    g = torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device=DEV)
    k = randn(B, T, Hk, dk)
    if equal:           # tokens that correct each other entirely
        k = k[:, :1].expand(B, T, Hk, dk)
    k = torch.nn.functional.normalize(k, dim=-1).contiguous()
    return dict(q=k.clone() if equal else randn(B, T, Hk, dk), k=k, v=randn(B, T, Hv, dv),
                beta=torch.ones(B, T, Hv, device=DEV), gate=torch.zeros(B, T, Hv, device=DEV))


def rel(x, y):
    return float((x.double() - y.double()).norm() / y.double().norm())


def rule(hip, c, grad_o=None):
    if grad_o is None:
        with torch.no_grad():
            return hip.delta_rule(**c, scale=1.0)
    leaves = [c[n].clone().requires_grad_() for n in ("q", "k", "v", "beta", "gate")]
    o, S = hip.delta_rule(*leaves, scale=1.0)
    return o.detach(), S.detach(), torch.autograd.grad(o, leaves, grad_o)


@pytest.mark.parametrize("T", [9, 64, 150])
@pytest.mark.parametrize("equal", [True, False])
def test_growth_within_the_range(hip, T, equal):
    banner(f"growth within the range {T} {equal}")
    c = inputs(T, 31, equal)
    c["gate"][..., 0] = 1.98 / min(T, 64)       # one long run
    c["gate"][:, 2::7, 1] = 1.9                 # single tokens, with decays between them
    c["gate"][:, 3::7, 1] = -2.0
    c["gate"][:, ::2, 2] = -math.inf            # growth after the state was erased
    c["gate"][:, 1::2, 2] = 1.9
    go = torch.randn_like(c["v"])
    o, S, grads = rule(hip, c, go)
    wo, wS = OD.rule(**c, scale=1.0)
    want = OD.rule_adjoint(**c, grad_o=go, scale=1.0)
    tol = 7.4 * 1.5e-6 * (T // 64 + 2)
    assert rel(o, wo) <= tol and rel(S, wS) <= tol
    o, S = rule(hip, c)
    assert rel(o, wo) <= tol and rel(S, wS) <= tol
    for n, x in zip(("q", "k", "v", "beta"), grads):
        assert rel(x, want[n]) <= 2 * tol, n
    assert torch.isfinite(grads[4]).all()


@pytest.mark.parametrize("T", [9, 150])
@pytest.mark.parametrize("what", ["growth", "jump", "nan", "inf"])
def test_beyond_the_range_is_nan_for_any_length(hip, T, what):
    """Never a finite answer that the formulas do not give, whether a call is short
    or long; other heads and sequences as without it."""
    banner(f"beyond the range {T} {what}")
    for save in (False, True):
        c = inputs(T, 32)
        clean, clean_S = rule(hip, c, torch.ones_like(c["v"]))[:2] if save else rule(hip, c)
        at = T // 2 + 1
        if what == "growth":
            c["gate"][0, at - 3:, 1] = 1.0      # above 2 with the third of them
        else:
            c["gate"][0, at, 1] = {"jump": 2.5, "nan": math.nan, "inf": math.inf}[what]
        out = rule(hip, c, torch.ones_like(c["v"])) if save else rule(hip, c)
        o, S = out[:2]
        assert torch.isnan(o[0, at:, 1]).all() and torch.isnan(S[0, 1]).all()
        first = at // 64 * 64                   # chunks before it are as they were
        assert torch.equal(o[0, :first, 1], clean[0, :first, 1])
        assert torch.equal(o[1], clean[1]) and torch.equal(S[1], clean_S[1])
        for h in (0, 2, 3):
            assert torch.equal(o[0, :, h], clean[0, :, h]) and torch.equal(S[0, h], clean_S[0, h])
        if save:
            assert all(torch.isfinite(x[1]).all() for x in out[2])
            assert torch.isnan(out[2][4][0, at:, 1]).any()
            assert torch.isfinite(out[2][4][0][:, [0, 2, 3]]).all()


@pytest.mark.parametrize("gate", [1.0, 5.0, 40.0])
def test_single_tokens_take_any_gate(hip, gate):
    """One token with a gate above 0, as the formula stands: sums of 32 terms and a
    few roundings of 2^-24, under 1e-6 of the grown state's size."""
    c = inputs(1, 33, equal=False)
    c["gate"][:] = gate
    start = torch.randn(2, 4, 32, 40, device=DEV)
    S = start.clone()
    o = hip.delta_rule_step(*(c[n][:, 0] for n in ("q", "k", "v", "beta", "gate")), state=S,
                            scale=1.0)
    wo, wS = OD.rule(**c, state=start, scale=1.0)
    assert rel(o, wo[:, 0]) <= 1e-6 and rel(S, wS) <= 1e-6


@pytest.mark.parametrize("T", [9, 150])
@pytest.mark.parametrize("name", ["q", "k", "v", "beta"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_values_that_are_not_finite_stay_in_their_head(hip, T, name, bad):
    """They show in their token's answer, and reach no other sequence or head, no
    chunk before theirs, and from v no other column."""
    c = inputs(T, 34, equal=False)
    clean, clean_S, clean_g = rule(hip, c, torch.ones_like(c["v"]))
    at, head = T // 2 + 1, 1 if name in ("v", "beta") else 0
    c[name] = c[name].clone()
    if name == "beta":
        c[name][0, at, head] = bad
    else:
        c[name][0, at, head, 3] = bad
    o, S, grads = rule(hip, c, torch.ones_like(c["v"]))
    heads = [head] if name in ("v", "beta") else [0, 1]     # two value heads read a key head
    others = [h for h in range(4) if h not in heads]
    assert torch.equal(o[1], clean[1]) and torch.equal(S[1], clean_S[1])
    assert torch.equal(o[0][:, others], clean[0][:, others])
    assert torch.equal(S[0, others], clean_S[0, others])
    first = at // 64 * 64
    assert torch.equal(o[0, :first], clean[0, :first])
    hit = o[0, at][heads]
    if name == "v":
        assert not torch.isfinite(hit[:, 3]).any()
        rest = [i for i in range(40) if i != 3]
        assert torch.equal(o[0, :, head][:, rest], clean[0, :, head][:, rest])
        assert torch.equal(S[0, head][:, rest], clean_S[0, head][:, rest])
    else:
        assert not torch.isfinite(hit).any()
    for n, x, y in zip("qkvbg", grads, clean_g):
        assert torch.equal(x[1], y[1])
        if n in "vbg":
            assert torch.equal(x[0][:, others], y[0][:, others])
