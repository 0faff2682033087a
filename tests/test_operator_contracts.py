"""What the sequence and training operators refuse, and what autograd is told of
them: CPU tests of the checks, GPU tests of the rest."""
import pytest
import torch

DEV = "cuda:0"


def rule_inputs(device, B=2, T=70, Hk=1, Hv=2, dk=16, dv=24):
    g = torch.Generator().manual_seed(41)
    randn = lambda *s: torch.randn(s, generator=g).to(device)
    return dict(q=randn(B, T, Hk, dk), k=torch.nn.functional.normalize(randn(B, T, Hk, dk), dim=-1),
                v=randn(B, T, Hv, dv), beta=torch.sigmoid(randn(B, T, Hv)),
                gate=-randn(B, T, Hv).abs(), state=randn(B, Hv, dk, dv))


# -------------------------------------------- the autograd function's own checks

def test_function_refuses_host_tensors():
    from differentiable_sparse_linear_amd import DeltaRule
    with pytest.raises(ValueError, match="device tensor"):
        DeltaRule.apply(*rule_inputs("cpu").values(), 1.0, None)


@pytest.mark.gpu
def test_function_checks_what_the_call_checks(hip):
    """Refused before any kernel runs: they would read past the shorter arrays."""
    c = rule_inputs(DEV)
    for kw, text in [(dict(k=c["k"][:, :3]), "shape"), (dict(v=c["v"].half()), "dtype"),
                     (dict(q=c["q"].cpu()), "device"), (dict(beta=c["beta"][:1]), "shape"),
                     (dict(state=c["state"][..., :5]), "shape")]:
        with pytest.raises(ValueError, match=text):
            hip.DeltaRule.apply(*{**c, **kw}.values(), 1.0, None)
    short = torch.ones(1, device=DEV, dtype=torch.int32)
    with pytest.raises(ValueError, match="shape"):
        hip.DeltaRule.apply(*c.values(), 1.0, short)


@pytest.mark.gpu
def test_function_takes_strided_rows(hip):
    """Rows whose last dimension is not contiguous, and the default scale."""
    c = rule_inputs(DEV)
    wide = {n: c[n].repeat_interleave(2, dim=-1)[..., ::2].requires_grad_() for n in ("q", "k", "v")}
    assert not wide["v"].is_contiguous()
    leaves = {n: x.detach().requires_grad_() for n, x in c.items()}
    got = hip.DeltaRule.apply(*{**leaves, **wide}.values(), None, None)
    flat = {n: x.detach().clone().requires_grad_() for n, x in c.items()}
    want = hip.delta_rule(**flat)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ga = torch.autograd.grad(got[0].square().sum(), [wide["q"], wide["k"], wide["v"]])
    gb = torch.autograd.grad(want[0].square().sum(), [flat["q"], flat["k"], flat["v"]])
    assert all(torch.equal(a, b) for a, b in zip(ga, gb))
