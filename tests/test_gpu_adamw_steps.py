"""What counts as a step of the optimizer class: steps that the device skips,
calls that fail, and captured calls."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
KINDS = [torch.float64, torch.float32, torch.bfloat16, torch.float16]
# A few more roundings of the correction's powers (under 100 of 2^-53) and of an
# update in the moments' type; masters are compared where there are some.
NEAR = {torch.float64: 1e-12, torch.float32: 1e-6}


def params(kind, seed=51):
    g = torch.Generator().manual_seed(seed)
    return [torch.nn.Parameter(torch.randn(n, generator=g).to(kind).to(DEV)) for n in (5, 3000, 70)]


def put_grads(ps, seed, bad=None):
    g = torch.Generator().manual_seed(seed)
    for p in ps:
        p.grad = torch.randn(p.shape, generator=g).to(p.dtype).to(DEV)
    if bad is not None:
        ps[1].grad[2222] = bad


def held(opt, ps):
    """Parameters (or their masters) and moments."""
    st = [opt.state[p] for p in ps]
    return [s["master"] if s["master"] is not None else p.detach() for s, p in zip(st, ps)] + [
        s[n] for s in st for n in ("exp_avg", "exp_avg_sq")]


def same(a, b, ps, qs):
    for x, y in zip(held(a, ps), held(b, qs)):
        assert torch.allclose(x, y, rtol=NEAR[x.dtype], atol=NEAR[x.dtype] * 1e-2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_skipped_steps_do_not_count(hip, kind, bad):
    """Bad gradients first, between and in a row: as an optimizer that never saw them."""
    ps, qs = params(kind), params(kind)
    kw = dict(lr=1e-2, betas=(0.9, 0.999), weight_decay=0.1, max_norm=3.0)
    a, b = hip.AdamW(ps, **kw), hip.AdamW(qs, **kw)
    for i, broken in enumerate([True, False, False, True, True, True, False, False]):
        put_grads(ps, i, bad if broken else None)
        before = [p.detach().clone() for p in ps]
        a.step()
        assert math.isfinite(float(a.param_groups[0]["last_norm"])) != broken
        if broken:
            assert all(torch.equal(x, y) for x, y in zip(ps, before))
            continue
        put_grads(qs, i)
        b.step()
        same(a, b, ps, qs)
        if i == 2:      # the counters are saved and restored with the rest
            saved = a.state_dict()
            a = hip.AdamW(ps, **kw)
            a.load_state_dict(saved)


def test_a_parameter_that_joins_after_a_skipped_step(hip):
    ps, qs = params(torch.float32), params(torch.float32)
    a, b = hip.AdamW(ps, max_norm=3.0), hip.AdamW(qs, max_norm=3.0)
    put_grads(ps, 0, math.nan)
    ps[0].grad = None
    a.step()
    for i in (1, 2):
        put_grads(ps, i)
        put_grads(qs, i)
        a.step()
        b.step()
        same(a, b, ps, qs)
    a.param_groups[0]["max_norm"] = b.param_groups[0]["max_norm"] = None
    put_grads(ps, 3)        # what was skipped is still not counted
    put_grads(qs, 3)
    a.step()
    b.step()
    same(a, b, ps, qs)


def test_a_call_that_fails_does_not_count(hip):
    ps, qs = params(torch.float32), params(torch.float32)
    a, b = hip.AdamW(ps, max_norm=3.0), hip.AdamW(qs, max_norm=3.0)
    put_grads(ps, 0)
    a.param_groups[0]["max_norm"] = -1.0
    with pytest.raises(ValueError):
        a.step()
    a.param_groups[0]["max_norm"] = 3.0
    put_grads(qs, 0)
    a.step()
    b.step()
    assert all(torch.equal(x, y) for x, y in zip(held(a, ps), held(b, qs)))


def test_capture_is_refused(hip):
    ps = params(torch.float32)
    opt = hip.AdamW(ps)
    put_grads(ps, 0)
    opt.step()
    x = torch.zeros(4, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.add_(1)
        with pytest.raises(RuntimeError, match="captured"):
            opt.step()
    assert all(opt.state[p]["step"] == 1 for p in ps)


def test_counters_are_checked(hip):
    x = [torch.ones(4, device=DEV)]
    step = lambda c: hip.adamw_step_([x[0].clone()], x, [x[0].clone()], [x[0].clone()], 1,
                                     max_norm=1.0, skipped=c)
    for bad in ([], [torch.zeros((), device=DEV)], [torch.zeros(2, device=DEV, dtype=torch.int64)],
                [torch.zeros((), dtype=torch.int64)]):
        with pytest.raises(ValueError):
            step(bad)
    step([None])
    step([torch.zeros((), device=DEV, dtype=torch.int64)])


def test_state_dict_holds_no_answers(hip):
    """The norm stays with the optimizer; what is saved is numbers and the tensors
    of the state, and the optimizer that saved goes on as it was."""
    ps = params(torch.float32)
    opt = hip.AdamW(ps, max_norm=3.0)
    put_grads(ps, 0)
    opt.step()
    norm = opt.param_groups[0]["last_norm"]
    saved = opt.state_dict()
    assert not any(isinstance(x, torch.Tensor) for g in saved["param_groups"] for x in g.values())
    assert opt.param_groups[0]["last_norm"] is norm
    other = hip.AdamW(params(torch.float32), max_norm=1.0)
    other.load_state_dict(saved)
    assert other.param_groups[0]["max_norm"] == 3.0 and "last_norm" not in other.param_groups[0]
