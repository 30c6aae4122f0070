"""moe_route_backward against the plain 64-bit formula and against differences
of moe_route."""
import pytest
import torch

import _block as B
import _gpu as G

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1, 1, 0.0, False), (1, 256, 8, 0.0, False), (7, 5, 3, 0.4, False),
          (9, 1024, 32, 0.2, False), (33, 61, 6, 0.0, False), (257, 896, 16, 0.1, False),
          (300, 8, 8, 0.2, True), (5000, 256, 8, 0.05, False), (64, 130, 2, 0.9, False)]


def problem(T, E, k, sigmoid):
    m = G.lib()
    return m.make_problem(T, 128, 128, E, k, flags=m.F_SIGMOID_ROUTING if sigmoid else 0)


def backward(p, logits, idx, w, dw):
    m = G.lib()
    out = torch.full((p.T, p.E), 7.0, device="cuda")
    d = lambda v: None if v is None else v.cuda()
    m.moe_route_backward(p, d(logits), d(idx), d(w), d(dw), out)
    return out


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("sigmoid", [False, True])
def test_against_the_formula(shape, sigmoid):
    T, E, k, masked, repeat = shape
    g = torch.Generator().manual_seed(T + E)
    idx = B.routing(T, E, k, g, masked, repeat)
    logits = 3.0 * torch.randn(T, E, generator=g)
    w = B.route_weights(logits, idx, sigmoid).float()
    dw = torch.randn(T, k, generator=g)
    # what masked slots hold must not matter
    w_in, dw_in = w.clone(), dw.clone()
    w_in[idx < 0], dw_in[idx < 0] = float("nan"), float("inf")
    out = backward(problem(T, E, k, sigmoid), logits if sigmoid else None, idx, w_in, dw_in)
    assert G.lib().moe_get_last_error() == 0
    ref, mag = B.route_backward(logits, idx, w, dw, sigmoid)
    # c: k products and sums; the difference; the factor (exp 2 units, three products, a quotient)
    # and, with sigmoid, the sum of k scores; slots of one expert add up
    tiny = 2.0 ** -126
    B.within(out, ref, (3 * k + 24) * B.U * mag + tiny, "dlogits")


def test_far_logits_with_sigmoid():
    # scores near 0 and 1 keep their small derivative: neither overflows nor cancels
    T, E, k = 4, 6, 2
    logits = torch.tensor([[30.0, 25.0], [-30.0, -40.0], [80.0, -80.0], [0.0, 60.0]])
    logits = torch.cat((logits, torch.zeros(T, E - k)), 1)
    idx = torch.tensor([[0, 1]] * T, dtype=torch.int32)
    w = B.route_weights(logits, idx, True).float()
    dw = torch.tensor([[1.0, -2.0]] * T)
    out = backward(problem(T, E, k, True), logits, idx, w, dw)
    ref, mag = B.route_backward(logits, idx, w, dw, True)
    B.within(out, ref, (3 * k + 24) * B.U * mag + 2.0 ** -126, "dlogits")


@pytest.mark.parametrize("bad", [-2, 8, 2 ** 31 - 1])
def test_indices_out_of_range_are_reported(bad):
    T, E, k = 10, 8, 2
    g = torch.Generator().manual_seed(1)
    idx = B.routing(T, E, k, g)
    idx[4, 1] = bad
    w, dw = torch.rand(T, k, generator=g), torch.randn(T, k, generator=g)
    out = backward(problem(T, E, k, False), None, idx, w, dw)
    assert G.lib().moe_get_last_error() == 1
    idx[4, 1] = -1
    ref, mag = B.route_backward(torch.zeros(T, E), idx, w, dw, False)
    B.within(out, ref, (3 * k + 24) * B.U * mag, "dlogits")


@pytest.mark.parametrize("sigmoid", [False, True])
def test_against_differences_of_moe_route(sigmoid):
    m = G.lib()
    T, E, k, step = 40, 32, 4, 2.0 ** -7
    g = torch.Generator().manual_seed(2)
    # logits a whole step and more apart: the selection holds under the difference
    logits = torch.stack([torch.randperm(E, generator=g) for _ in range(T)]).float() * 0.125
    d = torch.rand(T, E, generator=g) * 2 - 1
    dw = torch.randn(T, k, generator=g)
    p = problem(T, E, k, sigmoid)

    def route(l):
        idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
        w = torch.empty(T, k, device="cuda")
        m.moe_route(p, l.cuda(), None, idx, w)
        return idx.cpu(), w.cpu()

    idx, w = route(logits)
    up, down = logits + step * d, logits - step * d
    (iu, wu), (il, wl) = route(up), route(down)
    # each token's chosen experts stay; a slot may hold another of them
    assert torch.equal(iu.sort(1).values, idx.sort(1).values) and torch.equal(il.sort(1).values, idx.sort(1).values)
    by_expert = lambda i, v: torch.zeros(T, E, dtype=torch.float64).scatter(1, i.long(), v.double())
    dense = by_expert(idx, dw)
    got = ((by_expert(iu, wu) - by_expert(il, wl)) * dense).sum() / (2 * step)
    out = backward(p, logits, idx, w, dw).cpu().double()
    wx = lambda l: (B.route_weights(l, idx, sigmoid) * dw.double()).sum()
    truncation = abs((wx(up) - wx(down)) / (2 * step)
                     - (B.route_backward(logits, idx, B.route_weights(logits, idx, sigmoid), dw, sigmoid)[0]
                        * d).sum())
    # the weights' own rounding, (k + 10) units each, over the step
    rounding = ((k + 10) * B.U * (wu + wl).double() * dw.abs().double()).sum() / (2 * step)
    mag = B.route_backward(logits, idx, w, dw, sigmoid)[1]
    assert abs(got - (out * d).sum()) <= truncation + rounding + (3 * k + 24) * B.U * mag.sum()


def test_empty_batch():
    m = G.lib()
    e = lambda *s: torch.empty(*s, device="cuda")
    m.moe_route_backward(problem(0, 8, 2, False), None, torch.empty(0, 2, dtype=torch.int32, device="cuda"),
                         e(0, 2), e(0, 2), e(0, 8))
    assert m.moe_get_last_error() == 0


@pytest.mark.parametrize("sigmoid", [False, True])
def test_nan_of_a_chosen_logit_stays(sigmoid):
    # the weights of its token have no gradient, which must show; other tokens, masked slots
    # and logits that were not chosen are as without it
    T, E, k = 12, 10, 3
    g = torch.Generator().manual_seed(4)
    idx = B.routing(T, E, k, g)
    idx[5, 2] = -1
    logits = torch.randn(T, E, generator=g)
    w, dw = B.route_weights(logits, idx, sigmoid).float(), torch.randn(T, k, generator=g)
    p = problem(T, E, k, sigmoid)
    want = backward(p, logits, idx, w, dw).cpu()
    chosen = idx.clamp(min=0).long()
    bad = logits.clone()
    for t in (0, 5):
        bad[t, chosen[t, 1]] = float("nan")
    other = next(e for e in range(E) if e not in chosen[7].tolist())
    bad[7, other] = float("nan")  # not chosen
    w = B.route_weights(bad, idx, sigmoid).float()
    out = backward(p, bad, idx, w, dw).cpu()
    assert G.lib().moe_get_last_error() == 0
    keep = [t for t in range(T) if t not in (0, 5)]
    assert torch.equal(out[keep], want[keep])
    for t in (0, 5):
        live = torch.zeros(E, dtype=torch.bool)
        live[chosen[t][idx[t] >= 0]] = True
        assert out[t, live].isnan().all() and not out[t, ~live].any()


def test_scores_that_underflow_have_no_gradient():
    # sigmoid(-200) is zero in fp32, all of a token's scores are: zeros, not 0 / 0
    T, E, k = 3, 8, 2
    logits = torch.full((T, E), -200.0)
    idx = torch.tensor([[1, 6]] * T, dtype=torch.int32)
    w, dw = torch.full((T, k), 0.5), torch.tensor([[1.0, -2.0]] * T)
    assert not backward(problem(T, E, k, True), logits, idx, w, dw).any()
