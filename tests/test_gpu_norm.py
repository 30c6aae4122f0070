"""moe_add_rmsnorm and its gradient against plain 64-bit implementations, to the
bounds of _block.py."""
import pytest
import torch

import _block as B
import _gpu as G

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 8192), (2, 7), (3, 64), (5, 1001), (9, 250), (33, 3584), (64, 7168),
          (130, 1024), (257, 4104), (700, 96), (2, 33000), (1, 131072), (2049, 8)]
E4M3 = torch.float8_e4m3fn


def gen(seed=0):
    return torch.Generator().manual_seed(seed)


def new(*shape, dtype=torch.float32):
    t = torch.empty(*shape, dtype=dtype, device="cuda")
    t.view(torch.uint8).fill_(0x5A)
    return t


def dev(t):
    return None if t is None else t.cuda()


def inputs(T, H, t, residual, seed=0):
    g = gen(seed + T + H)
    channel = torch.exp(0.7 * torch.randn(H, generator=g))
    x = torch.randn(T, H, generator=g).to(t)
    r = (2.0 * torch.randn(T, H, generator=g) * channel).to(t) if residual else None
    return x, r, (1.0 + 0.2 * torch.randn(H, generator=g)).to(t)


def forward(n, x, r, gamma, h=True, y=True, q=True):
    m = G.lib()
    T, H = x.shape
    out = (new(T, H, dtype=x.dtype) if h else None, new(T, H, dtype=x.dtype) if y else None,
           new(T, H, dtype=E4M3) if q else None, new(T) if q else None)
    m.moe_add_rmsnorm(n, dev(x), dev(r), dev(gamma), *out)
    assert m.moe_get_last_error() == 0
    return out


def check_forward(out, x, r, gamma, eps=B.EPS):
    t, H = x.dtype, x.shape[1]
    h, y, _ = B.norm(x, r, gamma, eps)
    # m: half the error of the mean square, the root (2 units) and the sum; two products
    c = (B.chain(H) / 2 + 12) * B.U
    if out[0] is not None:
        B.within(out[0], h, B.store(t, h) + B.U * h.abs(), "h")
    if out[1] is not None:
        B.within(out[1], y, B.store(t, y) + c * y.abs(), "y")
    if out[2] is not None:
        amax = y.abs().amax(1)
        s = torch.where(amax > 0, amax / 448.0, 1.0)
        B.within(out[3], s, (c + 2 * B.U) * s, "q_scale")
        got = out[2].cpu().double() * out[3].cpu().double()[:, None]
        # half a step of e4m3: 2^-4 of a normal value, 2^-10 below 2^-6 (in units of the scale)
        B.within(got, y, (2.0 ** -4 + 2 * c) * y.abs() + 2.0 ** -10 * s[:, None] * (1 + c), "q")
        # the largest magnitude of a row is coded as 448
        live = amax > 0
        assert (out[2].cpu().float().abs().amax(1)[live] == 448.0).all()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
def test_forward(shape, dtype, residual):
    T, H = shape
    t, m = B.DTYPES[dtype], G.lib()
    x, r, gamma = inputs(T, H, t, residual)
    check_forward(forward(m.make_norm(T, H, t), x, r, gamma), x, r, gamma)


@pytest.mark.parametrize("h,y,q", [(0, 1, 0), (1, 1, 0), (0, 0, 1), (1, 0, 1), (0, 1, 1)])
@pytest.mark.parametrize("shape", [(7, 512), (7, 513)], ids=str)
def test_chosen_outputs(h, y, q, shape):
    # outputs that are left out change nothing in the others
    T, H = shape
    m, t = G.lib(), torch.bfloat16
    x, r, gamma = inputs(T, H, t, True)
    n = m.make_norm(T, H, t, eps=1e-5)
    out = forward(n, x, r, gamma, h, y, q)
    check_forward(out, x, r, gamma, eps=n.eps)
    every = forward(n, x, r, gamma)
    for a, b in zip(out, every):
        if a is not None:
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_rows_of_zeros_and_tiny_values():
    m = G.lib()
    T, H = 4, 256
    x = torch.zeros(T, H)
    x[1, 3] = 1e-30
    x[2] = 1e-12
    gamma = torch.ones(H)
    n = m.make_norm(T, H, torch.float32)
    out = forward(n, x, None, gamma)
    h, y, q, s = (v.cpu() for v in out)
    assert not y[0].any() and not q[0].float().any() and s[0] == 1.0
    check_forward(tuple(v[1:] for v in (h, y, q, s)), x[1:], None, gamma, eps=n.eps)
    # without eps a row of zeros has no norm: NaN, in every output
    out = forward(m.make_norm(1, H, torch.float32, eps=0.0), x[:1], None, gamma)
    assert out[1].isnan().all() and out[3].isnan().all() and out[2].float().isnan().all()


@pytest.mark.parametrize("H", [64, 65, 8192])
def test_infinities_and_nan_stay_in_their_row(H):
    m, t = G.lib(), torch.bfloat16
    x, r, gamma = inputs(5, H, t, True)
    x[1, 3], x[3, H - 1] = float("nan"), float("inf")
    n = m.make_norm(5, H, t)
    h, y, q, s = forward(n, x, r, gamma)
    assert h[1, 3].isnan() and h[3, H - 1] == float("inf")
    assert y[1].isnan().all() and s[1].isnan() and s[3].isnan() and y[3, H - 1].isnan()
    for v in (q[1], q[3]):
        assert v.float().isnan().all()
    keep = [0, 2, 4]
    check_forward(tuple(v[keep] for v in (h, y, q.view(torch.uint8), s))[:2] + (
        q.view(torch.uint8)[keep].view(E4M3), s[keep]), x[keep], r[keep], gamma)


def backward(n, h, gamma, dy, dh, dgamma=True):
    m = G.lib()
    T, H = h.shape
    dx, dg = new(T, H, dtype=h.dtype), new(H) if dgamma else None
    ws = new(m.moe_norm_workspace_bytes(n), dtype=torch.uint8) if dgamma else None
    m.moe_add_rmsnorm_backward(n, dev(h), dev(gamma), dev(dy), dev(dh), dx, dg, ws)
    assert m.moe_get_last_error() == 0
    return dx, dg


def check_backward(dx, dg, h, gamma, dy, dh):
    T, H = h.shape
    t = h.dtype
    ref, mag, rg, gmag = B.norm_backward(h, gamma, dy, dh)
    c = (2 * B.chain(H) + 24) * B.U
    B.within(dx, ref, B.store(t, ref) + c * mag, "dx")
    if dg is not None:
        B.within(dg, rg, (T * B.U + c) * gmag, "dgamma")


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("with_dh", [False, True])
def test_backward(shape, dtype, with_dh):
    T, H = shape
    t, m = B.DTYPES[dtype], G.lib()
    _, h, gamma = inputs(T, H, t, True, seed=1)
    g = gen(T)
    dy = torch.randn(T, H, generator=g).to(t)
    dh = torch.randn(T, H, generator=g).to(t) if with_dh else None
    n = m.make_norm(T, H, t)
    dx, dg = backward(n, h, gamma, dy, dh)
    check_backward(dx, dg, h, gamma, dy, dh)
    alone, none = backward(n, h, gamma, dy, dh, dgamma=False)
    assert none is None and torch.equal(alone, dx)


@pytest.mark.parametrize("H", [2, 3, 5, 8, 9, 15, 17, 23, 33, 127, 1023, 1031, 4098, 8191, 8193, 12289])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [1, 7, 500])
def test_widths_that_are_no_multiple_of_a_vector(H, dtype, T):
    # rows start and end inside vectors, each at a place of its own, and the buffers end with
    # the last row; 500 rows are several per block
    t, m = B.DTYPES[dtype], G.lib()
    x, r, gamma = inputs(T, H, t, True, seed=4)
    n = m.make_norm(T, H, t)
    check_forward(forward(n, x, r, gamma), x, r, gamma)
    dx, dg = backward(n, r, gamma, x, x)
    check_backward(dx, dg, r, gamma, x, x)


@pytest.mark.parametrize("H", [9, 1001])
def test_neighbouring_rows_stay_apart(H):
    # a row's vectors hold elements of its neighbours: their infinities and NaNs must not matter
    T, t, m = 400, torch.bfloat16, G.lib()
    x, r, gamma = inputs(T, H, t, True)
    bad = torch.arange(T) % 2 == 1
    x[bad] = float("nan")
    n = m.make_norm(T, H, t)
    h, y, q, s = forward(n, x, r, gamma)
    codes = q.view(torch.uint8)[~bad].view(E4M3)
    check_forward((h[~bad], y[~bad], codes, s[~bad]), x[~bad], r[~bad], gamma)
    dx, _ = backward(n, x, gamma, r, r, dgamma=False)
    check_backward(dx[~bad], None, x[~bad], gamma, r[~bad], r[~bad])
    dx, _ = backward(n, r, gamma, x, None, dgamma=False)
    check_backward(dx[~bad], None, r[~bad], gamma, x[~bad], None)


def test_backward_against_differences_of_the_forward():
    m = G.lib()
    T, H, step = 6, 192, 2.0 ** -6
    x, r, gamma = inputs(T, H, torch.float32, True, seed=2)
    g = gen(3)
    c, d = torch.randn(T, H, generator=g), torch.randn(T, H, generator=g)
    n = m.make_norm(T, H, torch.float32)
    h = x + r
    dx, dg = backward(n, h, gamma, c, None)
    loss = lambda v, w: (forward(n, v, None, w, h=False, q=False)[1].cpu().double() * c.double()).sum()
    exact = lambda v, w: (B.norm(v, None, w)[1] * c.double()).sum()
    e = torch.randn(H, generator=g)
    for (v1, w1), (v0, w0), grad in (((h + step * d, gamma), (h - step * d, gamma), (dx.cpu().double() * d).sum()),
                                     ((h, gamma + step * e), (h, gamma - step * e), (dg.cpu().double() * e).sum())):
        got = (loss(v1, w1) - loss(v0, w0)) / (2 * step)
        want = (exact(v1, w1) - exact(v0, w0)) / (2 * step)
        # what differs from the 64-bit difference is the forward's rounding; the rest of the way
        # to the gradient is the difference's own truncation
        y = B.norm(v1, None, w1)[1]
        rounding = 2 * ((B.chain(H) / 2 + 13) * B.U * y.abs() * c.abs()).sum() / (2 * step)
        assert abs(got - want) <= rounding
        ref = B.norm_backward(h, gamma, c, None)
        true = (ref[0] * d).sum() if grad is not None and v1 is not h else (ref[2] * e).sum()
        assert abs(grad - got) <= abs(want - true) + rounding + (2 * B.chain(H) + 24 + T) * B.U * (
            (ref[1] * d.abs()).sum() if v1 is not h else (ref[3] * e.abs()).sum())


@pytest.mark.parametrize("off", [1, 4])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_misaligned_buffers(off, dtype):
    T, H = 11, 512
    m, t = G.lib(), B.DTYPES[dtype]
    x, r, gamma = inputs(T, H, t, True)

    def at(v):
        flat = torch.empty(v.numel() + off, dtype=v.dtype, device="cuda")
        flat[off:].copy_(v.reshape(-1))
        return flat[off:].view(v.shape)

    n = m.make_norm(T, H, t)
    out = [at(torch.zeros(T, H, dtype=t)) for _ in range(2)] + [
        at(torch.zeros(T, H, dtype=torch.uint8)).view(E4M3), new(T)]
    m.moe_add_rmsnorm(n, at(x), at(r), at(gamma), *out)
    check_forward([out[0].clone(), out[1].clone(), out[2].view(torch.uint8).clone().view(E4M3), out[3]],
                  x, r, gamma)
    dx, dg = at(torch.zeros(T, H, dtype=t)), new(H)
    ws = new(m.moe_norm_workspace_bytes(n), dtype=torch.uint8)
    m.moe_add_rmsnorm_backward(n, at(r), at(gamma), at(x), None, dx, dg, ws)
    assert m.moe_get_last_error() == 0
    check_backward(dx.clone(), dg, r, gamma, x, None)


@pytest.mark.parametrize("T,H", [(3000, 512), (700, 8192), (1300, 129)])
def test_many_rows_and_repeats(T, H):
    # more rows than blocks: the sums of dgamma go over several rows each
    m, t = G.lib(), torch.bfloat16
    _, h, gamma = inputs(T, H, t, True)
    dy = torch.randn(T, H, generator=gen(1)).to(t)
    n = m.make_norm(T, H, t)
    dx, dg = backward(n, h, gamma, dy, dy)
    check_backward(dx, dg, h, gamma, dy, dy)
    for _ in range(2):
        again = backward(n, h, gamma, dy, dy)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dg)


@pytest.mark.parametrize("H", [8192, 8191])
def test_rows_past_32_bits(H):
    T = 280000  # 2.3 G elements
    m, t = G.lib(), torch.bfloat16
    x = torch.randn(T, H, device="cuda", dtype=t, generator=torch.Generator("cuda").manual_seed(0))
    gamma = torch.randn(H, generator=gen(1)).to(t).cuda()
    y = new(T, H, dtype=t)
    n = m.make_norm(T, H, t)
    m.moe_add_rmsnorm(n, x, None, gamma, None, y, None, None)
    dx = new(T, H, dtype=t)
    m.moe_add_rmsnorm_backward(n, x, gamma, x, None, dx, None, None)
    assert m.moe_get_last_error() == 0
    keep = [0, 1, T // 2, 262143, 262144, 262145, T - 1]
    xs = x[keep].cpu()
    check_forward((None, y[keep], None, None), xs, None, gamma.cpu())
    check_backward(dx[keep], None, xs, gamma.cpu(), xs, None)


def test_empty_batch():
    m = G.lib()
    n = m.make_norm(0, 64, torch.float32)
    e = lambda *s: torch.empty(*s, device="cuda")
    m.moe_add_rmsnorm(n, e(0, 64), None, e(64), None, e(0, 64), None, None)
    dg = new(64)
    m.moe_add_rmsnorm_backward(n, e(0, 64), e(64), e(0, 64), None, e(0, 64), dg, None)
    assert m.moe_get_last_error() == 0 and not dg.any()


def test_graph_replay_on_another_stream():
    T, H = 40, 1024
    m, t = G.lib(), torch.bfloat16
    x, r, gamma = (v.cuda() for v in inputs(T, H, t, True))
    n = m.make_norm(T, H, t)
    out = [new(T, H, dtype=t), new(T, H, dtype=t), new(T, H, dtype=E4M3), new(T)]
    dx, dg = new(T, H, dtype=t), new(H)
    ws = new(m.moe_norm_workspace_bytes(n), dtype=torch.uint8)

    def step():
        m.moe_add_rmsnorm(n, x, r, gamma, *out)
        m.moe_add_rmsnorm_backward(n, out[0], gamma, out[1], x, dx, dg, ws)

    step()
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for seed in (5, 6):
        nx, nr, _ = inputs(T, H, t, True, seed=seed)
        x.copy_(nx)
        r.copy_(nr)
        graph.replay()
        torch.cuda.synchronize()
        check_forward(out, nx, nr, gamma.cpu())
        check_backward(dx, dg, out[0].cpu(), gamma.cpu(), out[1].cpu(), nx)
    assert m.moe_get_last_error() == 0


@pytest.mark.parametrize("T,H", [(2048, 4096), (300, 4096), (1500, 4097), (64, 65536), (64, 65537)])
def test_codes_are_the_rounded_quotients(T, H):
    # fp32 rows: y as stored is what is quantised, so a code is y / q_scale, rounded to fp32 and
    # then to e4m3, and nothing else
    m = G.lib()
    x, _, gamma = inputs(T, H, torch.float32, False, seed=6)
    _, y, q, s = forward(m.make_norm(T, H, torch.float32), x, None, gamma, h=False)
    want = (y.cpu() / s.cpu()[:, None]).to(E4M3)
    off = (q.cpu().view(torch.uint8) != want.view(torch.uint8)).sum().item()
    assert off == 0, f"{off} of {T * H} codes differ"


@pytest.mark.parametrize("T,H", [(60, 512), (700, 512), (60, 509)])
def test_codes_at_the_midpoints(T, H):
    # rows of the midpoints between neighbouring codes, both signs, with 448 as the largest: every
    # quotient is a tie or a rounding away from one
    m = G.lib()
    codes = torch.arange(127, dtype=torch.uint8).view(E4M3).float()
    mid = (codes[1:] + codes[:-1]) / 2
    g = gen(8)
    x = mid[torch.randint(0, 126, (T, H), generator=g)] * (torch.randint(0, 2, (T, H), generator=g) * 2 - 1)
    x[:, 7] = 448.0
    x *= torch.exp2(torch.randint(-20, 20, (T, 1), generator=g).float())
    gamma = torch.full((H,), 1.25)
    _, y, q, s = forward(m.make_norm(T, H, torch.float32), x, None, gamma, h=False)
    want = (y.cpu() / s.cpu()[:, None]).to(E4M3)
    off = (q.cpu().view(torch.uint8) != want.view(torch.uint8)).sum().item()
    assert off == 0, f"{off} of {T * H} codes differ"


@pytest.mark.parametrize("H", [256, 257, 16389])
def test_scales_below_the_smallest_number(H):
    # a row whose largest |y| is so small that |y| / 448 rounds to zero is a row of zeros in
    # eight bits: scale 1, as for zeros themselves; a scale of a few of the smallest numbers stays
    m = G.lib()
    x = torch.ones(4, H)
    x[0] = 0.0
    x[2, 1:] = 0.0  # m = sqrt(H)
    gamma = torch.full((H,), 1e-44)
    n = m.make_norm(4, H, torch.float32)
    _, y, q, s = (None if v is None else v.cpu() for v in forward(n, x, None, gamma, h=False))
    assert y[1].ne(0).all() and s[:2].eq(1.0).all() and s[3] == 1.0
    assert not q[:2].float().any() and not q[3].float().any()
    gamma = torch.full((H,), 1e-42)
    _, y, q, s = (v.cpu() for v in forward(n, x, None, gamma))
    assert s[0] == 1.0 and 0.0 < s[1] < 1e-44 and not q[0].float().any()
    assert torch.equal(q[1:].view(torch.uint8), (y[1:] / s[1:, None]).clamp(max=448.0).to(E4M3).view(torch.uint8))


@pytest.mark.parametrize("dtype,T,H", [("bf16", 3, 512), ("bf16", 700, 512), ("bf16", 5, 1001), ("f32", 700, 1001),
                                       ("f32", 4, 33000), ("bf16", 4, 131072), ("f32", 3, 16389), ("f16", 3, 32777)])
@pytest.mark.parametrize("quant", [False, True])
def test_in_place(dtype, T, H, quant):
    # the sum in place of the residual and y in place of x, in every kernel of the forward
    t, m = B.DTYPES[dtype], G.lib()
    x, r, gamma = inputs(T, H, t, True, seed=7)
    n = m.make_norm(T, H, t)
    want = forward(n, x, r, gamma, q=quant)
    xd, rd = x.cuda(), r.cuda()
    q, s = (new(T, H, dtype=E4M3), new(T)) if quant else (None, None)
    m.moe_add_rmsnorm(n, xd, rd, gamma.cuda(), rd, xd, q, s)
    assert m.moe_get_last_error() == 0
    assert torch.equal(rd, want[0]) and torch.equal(xd, want[1])
    if quant:
        assert torch.equal(q.view(torch.uint8), want[2].view(torch.uint8)) and torch.equal(s, want[3])


def test_rows_up_to_the_limit_of_their_count():
    # T = 2^31 - 1: the grids' and the steps' sizes go past 32 bits on their way
    T, m, t = 2 ** 31 - 1, G.lib(), torch.bfloat16
    n = m.make_norm(T, 1, t)
    at = torch.tensor([0, 1, 2 ** 30, T - 17, T - 16, T - 9, T - 8, T - 2, T - 1], device="cuda")
    x = torch.full((T, 1), -2.0, dtype=t, device="cuda")
    x[at] = 3.0
    y = torch.zeros_like(x)
    gamma = torch.ones(1, dtype=t, device="cuda")
    m.moe_add_rmsnorm(n, x, None, gamma, None, y, None, None)
    assert m.moe_get_last_error() == 0
    # x / |x|, less 2^-23
    assert (y[at] == 1.0).all() and int((y == -1.0).sum()) == T - len(at)
    # rows of one element: m (gamma dy) (1 - (h m)^2), 2^-22 of dy at most, rounds off beside dh
    dx, dg = torch.zeros_like(x), new(1)
    ws = new(m.moe_norm_workspace_bytes(n), dtype=torch.uint8)
    m.moe_add_rmsnorm_backward(n, x, gamma, x, x, dx, dg, ws)
    assert m.moe_get_last_error() == 0
    assert torch.equal(dx, x)
    # dgamma: T terms of about 2, summed over T / 2432 rows by a thread and then over those
    want = 2.0 * (T - len(at)) + 3.0 * len(at)
    assert abs(dg.item() - want) <= (T / 2432 + 256 + 24) * B.U * want


@pytest.mark.parametrize("T", [2, 3, 5, 8])
@pytest.mark.parametrize("H", [40, 1000, 7185])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_of_one_cluster(T, H, dtype):
    # blocks that add each other's sums of dgamma: the last round of each loop before the
    # cluster's barrier takes part of a warp only
    t, m = B.DTYPES[dtype], G.lib()
    x, h, gamma = inputs(T, H, t, True, seed=9)
    n = m.make_norm(T, H, t)
    dx, dg = backward(n, h, gamma, x, x)
    check_backward(dx, dg, h, gamma, x, x)
    for _ in range(10):
        again = backward(n, h, gamma, x, x)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dg)


@pytest.mark.parametrize("T,H", [(7, 250), (700, 250), (700, 1031), (7, 8192), (350, 8193), (3, 33000)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_misaligned_buffers_in_every_variant(T, H, dtype):
    # one value and eight a thread, several rows and one a block, rows read again for each pass
    m, t = G.lib(), B.DTYPES[dtype]
    x, r, gamma = inputs(T, H, t, True, seed=10)

    def at(v):
        flat = torch.empty(v.numel() + 1, dtype=v.dtype, device="cuda")
        flat[1:].copy_(v.reshape(-1))
        return flat[1:].view(v.shape)

    n = m.make_norm(T, H, t)
    out = [at(torch.zeros(T, H, dtype=t)) for _ in range(2)] + [
        at(torch.zeros(T, H, dtype=torch.uint8)).view(E4M3), new(T)]
    m.moe_add_rmsnorm(n, at(x), at(r), at(gamma), *out)
    check_forward([out[0].clone(), out[1].clone(), out[2].view(torch.uint8).clone().view(E4M3), out[3]], x, r, gamma)
    ws = new(m.moe_norm_workspace_bytes(n), dtype=torch.uint8)
    for dh in (x, None):
        dx, dg = at(torch.zeros(T, H, dtype=t)), new(H)
        m.moe_add_rmsnorm_backward(n, at(r), at(gamma), at(x), None if dh is None else at(dh), dx, dg, ws)
        assert m.moe_get_last_error() == 0
        check_backward(dx.clone(), dg, r, gamma, x, dh)


@pytest.mark.parametrize("dtype,H", [("f32", 16387), ("f32", 16389), ("f32", 8193), ("bf16", 32771), ("f16", 32777),
                                     ("bf16", 16387), ("f16", 12289)])
@pytest.mark.parametrize("T", [2, 200])
def test_widest_shifted_rows(dtype, H, T):
    # the last widths in registers and the first that are read again, forward and backward
    m, t = G.lib(), B.DTYPES[dtype]
    x, r, gamma = inputs(T, H, t, True, seed=11)
    n = m.make_norm(T, H, t)
    check_forward(forward(n, x, r, gamma), x, r, gamma)
    dx, dg = backward(n, r, gamma, x, x)
    check_backward(dx, dg, r, gamma, x, x)
