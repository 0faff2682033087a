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


# ------------------------------------------------------ derivatives not given

@pytest.mark.gpu
def test_forward_mode_is_refused_not_dropped(hip):
    """A tangent is an error also with gradients off, where torch's own operations
    carry it on."""
    from torch.autograd import forward_ad
    c = rule_inputs(DEV)
    with forward_ad.dual_level():
        dual = {**c, "v": forward_ad.make_dual(c["v"], torch.ones_like(c["v"]))}
        for context in (torch.no_grad(), torch.enable_grad()):
            with context, pytest.raises(NotImplementedError):
                hip.delta_rule(**dual)
        one = {n: x[:, 0] if n != "state" else x.clone() for n, x in dual.items()}
        with torch.no_grad(), pytest.raises(ValueError, match="no derivatives"):
            hip.delta_rule_step(**one)
        with torch.no_grad():       # tensors without a tangent are answered
            o, S = hip.delta_rule(**c)
    wo, wS = hip.delta_rule(**c)
    assert torch.equal(o, wo) and torch.equal(S, wS)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["q", "k", "v", "beta", "gate", "state"])
def test_step_refuses_inputs_that_ask_for_gradients(hip, name):
    c = rule_inputs(DEV)
    one = {n: x[:, 0].clone() if n != "state" else x.clone() for n, x in c.items()}
    with torch.no_grad():
        want = hip.delta_rule_step(**{**one, "state": one["state"].clone()})
    asks = {**one, name: one[name].requires_grad_()}
    before = asks["state"].detach().clone()
    with pytest.raises(ValueError, match="no derivatives"):
        hip.delta_rule_step(**asks)
    assert torch.equal(asks["state"], before)
    with torch.no_grad():
        assert torch.equal(hip.delta_rule_step(**asks), want)


# ------------------------------------------- updates in place, as autograd sees them

@pytest.mark.gpu
def test_backward_across_an_optimizer_step_is_an_error(hip):
    """A graph that was kept across a step holds weights that are no longer there."""
    w = torch.nn.Parameter(torch.randn(8, 8, device=DEV))
    x = torch.randn(4, 8, device=DEV, requires_grad=True)
    opt = hip.AdamW([w], max_norm=1.0)
    loss = (x @ w).square().sum()
    loss.backward(retain_graph=True)
    opt.step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    opt.zero_grad()
    (x @ w).square().sum().backward()       # a new graph is as good as ever
    opt.step()


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["clip", "param", "moments", "master", "state", "out"])
def test_updates_raise_versions(hip, what):
    f = lambda *s, t=torch.float32: torch.ones(s, device=DEV, dtype=t)
    if what == "clip":
        xs = [f(5), f(3, t=torch.float64)]
        hip.clip_grad_norm_(xs, 1.0)
    elif what in ("param", "moments", "master"):
        p, g, m, v, w = [f(5, t=torch.bfloat16)], [f(5, t=torch.bfloat16)], [f(5)], [f(5)], [f(5)]
        seen = [x._version for x in g]
        hip.adamw_step_(p, g, m, v, 1, max_norm=1.0, masters=w)
        xs = {"param": p, "moments": m + v, "master": w}[what]
        assert [x._version for x in g] == seen      # gradients stay as they are
    else:
        c = rule_inputs(DEV)
        one = {n: x[:, 0].contiguous() if n != "state" else x.clone() for n, x in c.items()}
        out = torch.empty_like(one["v"])
        hip.delta_rule_step(**one, out=out)
        xs = [one["state"] if what == "state" else out]
    assert all(x._version == 1 for x in xs)


# ------------------------------------------------------ what a training pass keeps

@pytest.mark.parametrize("T,dk,dv", [(0, 64, 64), (1, 64, 64), (64, 128, 32), (65, 20, 33)])
def test_what_a_training_pass_keeps(T, dk, dv):
    """A state and 64 rows of W for each chunk and head, padded to whole tiles; no
    more than that (the state after the last chunk is an output)."""
    import ctypes
    import differentiable_sparse_linear_amd as sla
    from differentiable_sparse_linear_amd import delta as D
    s = D._Stride(1, 1, 1)
    args = D._Args(3, T, 1, 2, dk, dv, sla.SLA_F32, 1.0, 16, 16, 16, 16, 16, s, s, s, s, s, None)
    chunks = -(-T // 64)
    want = 3 * 2 * chunks * 4 * ((64 if dk <= 64 else 128) + 64) * (-(-dv // 32) * 32)
    assert sla.load().sla_delta_saved_bytes(ctypes.byref(args)) == want


@pytest.mark.gpu
def test_values_are_free_after_the_forward_pass(hip):
    """No gradient reads v: it may be written over, and is not held."""
    import gc
    import weakref
    c = rule_inputs(DEV)
    leaves = {n: x.clone().requires_grad_() for n, x in c.items()}
    want = torch.autograd.grad(hip.delta_rule(**leaves)[0].square().sum(), list(leaves.values()))
    v = leaves["v"] * 1.0
    o = hip.delta_rule(**{**leaves, "v": v})[0]
    with torch.no_grad():
        v.fill_(float("nan"))
    got = torch.autograd.grad(o.square().sum(), list(leaves.values()))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    v = c["v"].clone()
    kept = dict(leaves, v=v)
    o = hip.delta_rule(**kept)[0]
    held = weakref.ref(v)
    del v, kept
    gc.collect()
    assert held() is None
    o.sum().backward()


@pytest.mark.gpu
def test_raw_backward_without_values(hip):
    from differentiable_sparse_linear_amd import delta as D
    c = rule_inputs(DEV)
    q, k, v, beta, gate, state = c.values()
    o, last, saved = D._forward(q, k, v, beta, gate, state, 1.0, None, True)

    def back(args):
        out = [torch.empty_like(x) for x in (q, k, v, beta, gate)]
        work = D._bytes(D.sla_delta_workspace_bytes(args, backward=True), DEV)
        st = D.sla_delta_backward(args, saved, torch.ones_like(v), D._stride(v), None, *out, None,
                                  work, 0)
        return st, out

    torch.cuda.synchronize()
    args = D._make_args(q, k, v, beta, gate, 1.0, None)
    st, want = back(args)
    args.d_v = None
    other, got = back(args)
    torch.cuda.synchronize()
    assert st == other == hip.SLA_OK and all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------ the optimizer

def test_optimizer_refuses_host_parameters():
    from differentiable_sparse_linear_amd import AdamW
    p = torch.nn.Parameter(torch.ones(3))
    opt = AdamW([p], max_norm=1.0)
    opt.step()                      # nothing has a gradient
    p.grad = torch.ones(3)
    with pytest.raises(ValueError, match="device tensors"):
        opt.step()
    assert not opt.state and torch.equal(p.detach(), torch.ones(3))
