"""moe_dispatch, moe_combine and their gradients against plain 64-bit
implementations, at the sizes, masks, types and alignments where they can go
wrong.  Orders and moved rows are compared exactly; sums to the bounds of
_block.py."""
import pytest
import torch

import _block as B
import _gpu as G

pytestmark = pytest.mark.gpu

# T, H, E, k, share masked, a token may repeat an expert.  Widths: one, odd, even
# but not of 16 bytes, 16-byte rows, more than a block's vectors; batches: one
# token, odd ones, one and several steps of 1024 slots, one chunk and many
SHAPES = [
    (1, 8192, 256, 8, 0.0, False),
    (1, 64, 4, 1, 0.0, False),
    (2, 1, 1, 1, 0.5, False),
    (3, 7, 5, 3, 0.3, False),
    (31, 1001, 61, 6, 0.2, False),
    (33, 4104, 16, 2, 0.0, False),
    (64, 250, 8, 2, 0.0, False),
    (257, 72, 896, 16, 0.1, False),
    (130, 8192, 256, 8, 0.25, False),
    (700, 136, 1024, 32, 0.1, False),
    (100, 20, 3, 32, 0.2, True),
    (1025, 8, 2, 1, 0.4, True),
    (4099, 16, 256, 8, 0.05, False),
    (40000, 1, 130, 7, 0.1, False),
]


def gen(seed=0):
    return torch.Generator().manual_seed(seed)


def new(*shape, dtype=torch.float32, fill=None):
    """A device buffer that starts with other values than any output's."""
    t = torch.empty(*shape, dtype=dtype, device="cuda")
    t.view(torch.uint8).fill_(0x5A if fill is None else fill)
    return t


def dispatched(r, idx, x, x_scale=None):
    """moe_dispatch's outputs on the device, by name."""
    m = G.lib()
    T, k = idx.shape
    H = x.shape[1]
    out = dict(counts=new(r.E, dtype=torch.int32), offsets=new(r.E + 1, dtype=torch.int32),
               perm=new(T, k, dtype=torch.int32), src_row=new(T * k, dtype=torch.int32),
               x_rows=new(T * k, H, dtype=x.dtype),
               scale_rows=None if x_scale is None else new(T * k))
    ws = new(m.moe_rows_workspace_bytes(r), dtype=torch.uint8)
    m.moe_dispatch(r, idx, x, x_scale, *out.values(), ws)
    return out


def offset_copy(t, elements):
    """The same values in a buffer that starts `elements` elements past an allocation."""
    flat = torch.empty(t.numel() + elements, dtype=t.dtype, device=t.device)
    v = flat[elements:].view(t.shape)
    v.copy_(t)
    return v


def check_order(out, idx, E):
    for name, want in zip(("counts", "offsets", "perm", "src_row"), B.order(idx, E)):
        assert torch.equal(out[name].cpu(), want), name


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32", "e4m3"])
def test_dispatch(shape, dtype):
    T, H, E, k, masked, repeat = shape
    g = gen(T + H)
    m = G.lib()
    idx = B.routing(T, E, k, g, masked, repeat)
    if dtype == "e4m3":
        t = torch.float8_e4m3fn
        x = torch.randint(0, 255, (T, H), generator=g, dtype=torch.uint8).cuda().view(t)
    else:
        t = B.DTYPES[dtype]
        x = torch.randn(T, H, generator=g).to(t).cuda()
    scale = torch.rand(T, generator=g).cuda() if dtype in ("e4m3", "f32") else None
    out = dispatched(m.make_rows(T, H, E, k, t), idx.cuda(), x, scale)
    assert m.moe_get_last_error() == 0
    check_order(out, idx, E)
    src = B.order(idx, E)[3].long()
    bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()]
    want = x.view(bits).cpu()[src.clamp(min=0)]
    want[src < 0] = 0
    assert torch.equal(out["x_rows"].view(bits).cpu(), want)
    if scale is not None:
        want = scale.cpu()[src.clamp(min=0)]
        want[src < 0] = 0
        assert torch.equal(out["scale_rows"].cpu(), want)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("add", [False, True])
def test_combine_and_dispatch_backward(shape, dtype, add):
    T, H, E, k, masked, repeat = shape
    g, t, m = gen(T + 3 * H), B.DTYPES[dtype], G.lib()
    idx = B.routing(T, E, k, g, masked, repeat)
    perm = B.order(idx, E)[2]
    rows = torch.randn(T * k, H, generator=g).to(t)
    w = torch.rand(T, k, generator=g)
    extra = torch.randn(T, H, generator=g).to(t) if add else None
    # what masked slots point away from, and their weights, must not matter
    live = torch.zeros(T * k, dtype=torch.bool)
    live[perm[perm >= 0].long()] = True
    rows[~live] = float("nan")
    w[perm < 0] = float("inf")
    r = m.make_rows(T, H, E, k, t)
    dev = lambda v: None if v is None else v.cuda()
    for weights in (w, None):
        out = new(T, H, dtype=t)
        if weights is None:
            m.moe_dispatch_backward(r, dev(rows), dev(perm), dev(extra), out)
        else:
            m.moe_combine(r, dev(rows), dev(perm), dev(w), dev(extra), out)
        assert m.moe_get_last_error() == 0
        ref, mag = B.combine(rows, perm, weights, extra)
        B.within(out, ref, B.store(t, ref) + (k + 2) * B.U * mag, f"weights {weights is not None}")


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_combine_backward(shape, dtype):
    T, H, E, k, masked, repeat = shape
    g, t, m = gen(T + 5 * H), B.DTYPES[dtype], G.lib()
    idx = B.routing(T, E, k, g, masked, repeat)
    _, offsets, perm, _ = B.order(idx, E)
    rows, dout = torch.randn(T * k, H, generator=g).to(t), torch.randn(T, H, generator=g).to(t)
    w = torch.rand(T, k, generator=g)
    rows[int(offsets[E]):] = float("nan")
    w[perm < 0] = float("nan")
    drows, dw = new(T * k, H, dtype=t), new(T, k)
    m.moe_combine_backward(m.make_rows(T, H, E, k, t), dout.cuda(), rows.cuda(), perm.cuda(),
                           offsets.cuda(), w.cuda(), drows, dw)
    assert m.moe_get_last_error() == 0
    ref, rw, mag = B.combine_backward(dout, rows, perm, w)
    B.within(drows, ref, B.store(t, ref) + B.U * ref.abs(), "drows")  # one product, rounded twice
    B.within(dw, rw, (B.chain(H) + 2) * B.U * mag, "dw")


WIDTHS = [2, 3, 5, 8, 9, 15, 16, 17, 23, 31, 33, 127, 129, 1023, 1025, 1031, 2049, 8191]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32", "e4m3"])
@pytest.mark.parametrize("T,k", [(19, 3), (700, 9)])
def test_widths_that_are_no_multiple_of_a_vector(H, dtype, T, k):
    # rows start and end inside vectors, each at a place of its own; the neighbours' elements
    # are NaN where a row is not routed, and the buffers end with the last row
    E, g, m = 17, gen(H), G.lib()
    idx = B.routing(T, E, k, g, 0.2)
    _, offsets, perm, src = B.order(idx, E)
    if dtype == "e4m3":
        t = torch.float8_e4m3fn
        x = torch.randint(0, 255, (T, H), generator=g, dtype=torch.uint8).cuda().view(t)
    else:
        t = B.DTYPES[dtype]
        x = torch.randn(T, H, generator=g).to(t).cuda()
    r = m.make_rows(T, H, E, k, t)
    scale = torch.rand(T, generator=g).cuda()
    out = dispatched(r, idx.cuda(), x, scale)
    check_order(out, idx, E)
    bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()]
    want = x.view(bits).cpu()[src.long().clamp(min=0)]
    want[src < 0] = 0
    assert torch.equal(out["x_rows"].view(bits).cpu(), want)
    if dtype == "e4m3":
        assert m.moe_get_last_error() == 0
        return
    rows = torch.randn(T * k, H, generator=g).to(t)
    rows[int(offsets[E]):] = float("nan")
    w, dout = torch.rand(T, k, generator=g), torch.randn(T, H, generator=g).to(t)
    res, drows, dw = new(T, H, dtype=t), new(T * k, H, dtype=t), new(T, k)
    m.moe_combine(r, rows.cuda(), perm.cuda(), w.cuda(), dout.cuda(), res)
    m.moe_combine_backward(r, dout.cuda(), rows.cuda(), perm.cuda(), offsets.cuda(), w.cuda(), drows, dw)
    assert m.moe_get_last_error() == 0
    ref, mag = B.combine(rows, perm, w, dout)
    B.within(res, ref, B.store(t, ref) + (k + 2) * B.U * mag, "out")
    ref, rw, mag = B.combine_backward(dout, rows, perm, w)
    B.within(drows, ref, B.store(t, ref) + B.U * ref.abs(), "drows")
    B.within(dw, rw, (B.chain(H) + 2) * B.U * mag, "dw")


@pytest.mark.parametrize("H", [1001, 1024, 8192, 8191])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_rows_give_infinite_weight_gradients(H, dtype):
    # an infinity at a row's last or first element reaches its own dot product only, and as
    # an infinity
    T, E, k, t, m = 40, 5, 2, B.DTYPES[dtype], G.lib()
    idx = B.routing(T, E, k, gen(20))
    _, offsets, perm, _ = B.order(idx, E)
    rows = torch.ones(T * k, H, dtype=t)
    rows[perm[3, 1].long(), H - 1] = float("inf")
    rows[perm[7, 0].long(), 0] = -float("inf")
    dout = torch.full((T, H), 0.5, dtype=t)
    drows, dw = new(T * k, H, dtype=t), new(T, k)
    m.moe_combine_backward(m.make_rows(T, H, E, k, t), dout.cuda(), rows.cuda(), perm.cuda(), offsets.cuda(),
                           torch.ones(T, k, device="cuda"), drows, dw)
    assert m.moe_get_last_error() == 0
    want = torch.full((T, k), 0.5 * H)
    want[3, 1], want[7, 0] = float("inf"), -float("inf")
    assert torch.equal(dw.cpu(), want)
    assert torch.equal(drows.cpu(), torch.full((T * k, H), 0.5, dtype=t))


@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("off", [1, 2, 4])
def test_misaligned_rows(dtype, off):
    # rows of whole 16-byte vectors whose buffers do not start on one
    T, H, E, k = 37, 256, 9, 3
    g, m = gen(off), G.lib()
    idx = B.routing(T, E, k, g, 0.1)
    if dtype == "e4m3":
        t = torch.float8_e4m3fn
        x = torch.randint(0, 255, (T, H), generator=g, dtype=torch.uint8).cuda().view(t)
    else:
        t = B.DTYPES[dtype]
        x = torch.randn(T, H, generator=g).to(t).cuda()
    r = m.make_rows(T, H, E, k, t)
    scale = torch.rand(T, generator=g).cuda()
    raw = lambda v: v.view(torch.uint8).cpu()
    aligned = dispatched(r, idx.cuda(), x, scale)
    moved = dispatched(r, idx.cuda(), offset_copy(x.view(torch.uint8), off * x.element_size()).view(t)
                       if dtype == "e4m3" else offset_copy(x, off), scale)
    for name in aligned:
        assert torch.equal(raw(aligned[name]), raw(moved[name])), name
    if dtype == "e4m3":
        return
    rows, perm, w = aligned["x_rows"], aligned["perm"], torch.rand(T, k, generator=g).cuda()
    res = []
    for mv in (lambda v: v, lambda v: offset_copy(v, off)):
        out, drows, dw = mv(new(T, H, dtype=t)), mv(new(T * k, H, dtype=t)), new(T, k)
        m.moe_combine(r, mv(rows), perm, w, mv(x), out)
        m.moe_combine_backward(r, mv(x), mv(rows), perm, aligned["offsets"], w, drows, dw)
        res.append((out.clone(), drows.clone(), dw.cpu()))
    assert m.moe_get_last_error() == 0
    assert torch.equal(raw(res[0][0]), raw(res[1][0])) and torch.equal(raw(res[0][1]), raw(res[1][1]))
    mag = B.combine_backward(x.cpu(), rows.cpu(), perm.cpu(), w.cpu())[2]
    B.within(res[0][2], res[1][2], 2 * (B.chain(H) + 2) * B.U * mag, "dw")


@pytest.mark.parametrize("bad", [-2, 8, 2 ** 31 - 1, -2 ** 31])
def test_indices_out_of_range_are_reported_and_masked(bad):
    T, H, E, k = 20, 64, 8, 2
    m = G.lib()
    idx = B.routing(T, E, k, gen(1))
    idx[3, 1] = idx[19, 0] = bad
    x = torch.randn(T, H, generator=gen(2)).cuda()
    r = m.make_rows(T, H, E, k, torch.float32)
    out = dispatched(r, idx.cuda(), x)
    assert m.moe_get_last_error() == 1  # MOE_ERR_INVALID_ARG
    masked = torch.where((idx < 0) | (idx >= E), -1, idx)
    check_order(out, masked, E)
    # a permutation that points outside the rows
    perm = out["perm"].clone()
    perm[0, 0] = T * k
    perm[1, 1] = -5
    w = torch.rand(T, k, generator=gen(3))
    res, drows, dw = new(T, H), new(T * k, H, fill=0), new(T, k)
    m.moe_combine(r, out["x_rows"], perm, w.cuda(), None, res)
    assert m.moe_get_last_error() == 1
    m.moe_combine_backward(r, x, out["x_rows"], perm, out["offsets"], w.cuda(), drows, dw)
    assert m.moe_get_last_error() == 1
    fixed = perm.cpu()
    fixed[(fixed < 0) | (fixed >= T * k)] = -1
    ref, mag = B.combine(out["x_rows"].cpu(), fixed, w, None)
    B.within(res, ref, (k + 2) * B.U * mag, "out")
    ref, rw, mag = B.combine_backward(x.cpu(), out["x_rows"].cpu(), fixed, w)
    B.within(drows, ref, B.U * ref.abs(), "drows")
    B.within(dw, rw, (B.chain(H) + 2) * B.U * mag, "dw")
    assert m.moe_get_last_error() == 0


def test_offsets_outside_the_rows_are_clamped():
    # offsets a caller got wrong: no row outside [0, R) is written
    T, H, E, k = 5, 32, 4, 2
    m = G.lib()
    idx = B.routing(T, E, k, gen(4))
    perm = B.order(idx, E)[2].cuda()
    g, rows, w = (torch.randn(*s, generator=gen(5)).cuda() for s in ((T, H), (T * k, H), (T, k)))
    for last in (-7, T * k + 9):
        offsets = torch.zeros(E + 1, dtype=torch.int32)
        offsets[E] = last
        buf = new(T * k + 8, H, fill=0)
        m.moe_combine_backward(m.make_rows(T, H, E, k, torch.float32), g, rows, perm, offsets.cuda(),
                               w, buf[4:-4], new(T, k))
        assert m.moe_get_last_error() == 0
        assert not buf[:4].any() and not buf[-4:].any()


def test_every_slot_masked():
    T, H, E, k = 70, 40, 6, 4
    m = G.lib()
    idx = torch.full((T, k), -1, dtype=torch.int32)
    x = torch.randn(T, H, generator=gen(6)).cuda()
    r = m.make_rows(T, H, E, k, torch.float32)
    out = dispatched(r, idx.cuda(), x, torch.ones(T, device="cuda"))
    check_order(out, idx, E)
    assert not out["x_rows"].any() and not out["scale_rows"].any()
    nan = torch.full((T * k, H), float("nan"), device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    res, drows, dw = new(T, H), new(T * k, H), new(T, k)
    m.moe_combine(r, nan, out["perm"], w, None, res)
    m.moe_combine_backward(r, x, nan, out["perm"], out["offsets"], w, drows, dw)
    assert m.moe_get_last_error() == 0
    assert not res.any() and not drows.any() and not dw.any()
    m.moe_combine(r, nan, out["perm"], w, x, res)
    assert torch.equal(res, x)


def test_infinities_and_nan_in_live_rows_stay():
    T, H, E, k = 9, 24, 5, 2
    m = G.lib()
    idx = B.routing(T, E, k, gen(7))
    r = m.make_rows(T, H, E, k, torch.bfloat16)
    x = torch.randn(T, H, generator=gen(8)).to(torch.bfloat16)
    x[2, 3], x[4, 5] = float("inf"), float("nan")
    out = dispatched(r, idx.cuda(), x.cuda())
    res = new(T, H, dtype=torch.bfloat16)
    m.moe_combine(r, out["x_rows"], out["perm"], torch.full((T, k), 0.5, device="cuda"), None, res)
    res = res.cpu().float()
    assert res[2, 3] == float("inf") and res[4, 5].isnan()
    fine = torch.ones(T, H, dtype=torch.bool)
    fine[2, 3] = fine[4, 5] = False
    assert torch.equal(res[fine], x.float()[fine])


@pytest.mark.parametrize("H", [8192, 8191])
def test_large_rows_past_32_bits(H):
    # 2.6 G elements: places and row offsets beyond 2^31 elements and 2^32 bytes
    T, E, k = 40000, 64, 8
    m, t = G.lib(), torch.bfloat16
    idx = torch.rand(T, E, device="cuda", generator=torch.Generator("cuda").manual_seed(0)).topk(k, 1)
    idx = idx.indices.to(torch.int32)
    x = torch.randn(T, H, device="cuda", dtype=t, generator=torch.Generator("cuda").manual_seed(1))
    r = m.make_rows(T, H, E, k, t)
    out = dispatched(r, idx, x)
    check_order(out, idx.cpu(), E)
    src = out["src_row"].long()
    for a in range(0, T * k, 40000):
        assert torch.equal(out["x_rows"][a:a + 40000], x[src[a:a + 40000]])
    w = torch.full((T, k), 0.125, device="cuda")
    res = new(T, H, dtype=t)
    m.moe_combine(r, out["x_rows"], out["perm"], w, None, res)
    assert torch.equal(res, x)  # eight times an eighth: exact
    drows, dw = new(T * k, H, dtype=t), new(T, k)
    m.moe_combine_backward(r, x, out["x_rows"], out["perm"], out["offsets"], w, drows, dw)
    for a in range(0, T * k, 40000):
        assert torch.equal(drows[a:a + 40000], out["x_rows"][a:a + 40000] * 0.125)
    mag = (x.double() ** 2).sum(1, keepdim=True).cpu()
    B.within(dw, mag.expand(T, k), (B.chain(H) + 2) * B.U * mag, "dw")
    assert m.moe_get_last_error() == 0


def test_many_slots():
    # several steps of 1024 slots in each chunk
    T, E, k = 260000, 200, 8
    m = G.lib()
    g = gen(9)
    idx = torch.randint(-1, E, (T, k), generator=g, dtype=torch.int32)
    x = torch.randn(T, 1, generator=g).cuda()
    out = dispatched(m.make_rows(T, 1, E, k, torch.float32), idx.cuda(), x)
    assert m.moe_get_last_error() == 0
    check_order(out, idx, E)


@pytest.mark.parametrize("T,k", [(2048, 1), (2049, 1), (1024, 8), (8193, 1), (5400, 3), (16384, 1), (16385, 1),
                                 (131072, 1), (131073, 1)])
@pytest.mark.parametrize("E", [1, 257, 1024])
def test_orders_around_the_variants_limits(T, k, E):
    # one launch, one cluster of blocks with one and two steps, chunks of one step and of two
    m, g = G.lib(), gen(T + E)
    idx = B.routing(T, E, k, g, 0.1, repeat=True)
    x = torch.randn(T, 4, generator=g).cuda()
    out = dispatched(m.make_rows(T, 4, E, k, torch.float32), idx.cuda(), x)
    assert m.moe_get_last_error() == 0
    check_order(out, idx, E)
    src = out["src_row"].long()
    want = torch.where(src[:, None] < 0, 0.0, x[src.clamp(min=0)])
    assert torch.equal(out["x_rows"], want)


def test_repeats_bit_for_bit():
    T, H, E, k = 333, 520, 40, 8
    m, t = G.lib(), torch.bfloat16
    g = gen(10)
    idx = B.routing(T, E, k, g, 0.1).cuda()
    x, w = torch.randn(T, H, generator=g).to(t).cuda(), torch.rand(T, k, generator=g).cuda()
    r = m.make_rows(T, H, E, k, t)
    out = dispatched(r, idx, x)
    res = []
    for _ in range(3):
        y, drows, dw = new(T, H, dtype=t), new(T * k, H, dtype=t), new(T, k)
        m.moe_combine(r, out["x_rows"], out["perm"], w, x, y)
        m.moe_combine_backward(r, x, out["x_rows"], out["perm"], out["offsets"], w, drows, dw)
        res.append((y, drows, dw))
    for again in res[1:]:
        assert all(torch.equal(a, b) for a, b in zip(res[0], again))


def test_empty_batch():
    m = G.lib()
    r = m.make_rows(0, 64, 5, 2, torch.bfloat16)
    counts, offsets = new(5, dtype=torch.int32), new(6, dtype=torch.int32)
    e = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="cuda")
    i32 = torch.int32
    ws = new(m.moe_rows_workspace_bytes(r), dtype=torch.uint8)
    m.moe_dispatch(r, e(0, 2, dtype=i32), e(0, 64), None, counts, offsets, e(0, 2, dtype=i32),
                   e(0, dtype=i32), e(0, 64), None, ws)
    m.moe_combine(r, e(0, 64), e(0, 2, dtype=i32), e(0, 2, dtype=torch.float32), None, e(0, 64))
    assert m.moe_get_last_error() == 0
    assert not counts.any() and not offsets.any()


def test_graph_replay_on_another_stream():
    # captured on a stream of its own, replayed with new routing in the same buffers
    T, H, E, k = 50, 512, 32, 4
    m, t = G.lib(), torch.bfloat16
    r = m.make_rows(T, H, E, k, t)
    idx, x = B.routing(T, E, k, gen(11), 0.1).cuda(), torch.randn(T, H, device="cuda").to(t)
    w = torch.rand(T, k, device="cuda")
    first = dispatched(r, idx, x)  # sets the kernels up on this device
    ws = new(m.moe_rows_workspace_bytes(r), dtype=torch.uint8)
    out = {n: None if v is None else torch.empty_like(v) for n, v in first.items()}
    y, drows, dw = new(T, H, dtype=t), new(T * k, H, dtype=t), new(T, k)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        m.moe_dispatch(r, idx, x, None, *out.values(), ws)
        m.moe_combine(r, out["x_rows"], out["perm"], w, x, y)
        m.moe_combine_backward(r, x, out["x_rows"], out["perm"], out["offsets"], w, drows, dw)
    for seed in (12, 13):
        idx.copy_(B.routing(T, E, k, gen(seed), 0.3))
        x.copy_(torch.randn(T, H, generator=gen(seed)))
        graph.replay()
        torch.cuda.synchronize()
        want = dispatched(r, idx, x)
        check_order(out, idx.cpu(), E)
        assert torch.equal(out["x_rows"], want["x_rows"])
        ref, mag = B.combine(out["x_rows"].cpu(), out["perm"].cpu(), w.cpu(), x.cpu())
        B.within(y, ref, B.store(t, ref) + (k + 2) * B.U * mag, "y")
        ref, rw, mag = B.combine_backward(x.cpu(), out["x_rows"].cpu(), out["perm"].cpu(), w.cpu())
        B.within(drows, ref, B.store(t, ref) + B.U * ref.abs(), "drows")
        B.within(dw, rw, (B.chain(H) + 2) * B.U * mag, "dw")
    assert m.moe_get_last_error() == 0


def test_dispatched_codes_match_moe_permute():
    # the 8-bit form gives moe_expert_ffn exactly what moe_permute gives it
    T, H, E, k = 96, 512, 16, 4
    m = G.lib()
    idx = B.routing(T, E, k, gen(14)).cuda()
    x = torch.randn(T, H, generator=gen(15)).to(torch.bfloat16).cuda()
    p = m.make_problem(T, H, 128, E, k)
    i32 = torch.int32
    counts, offsets, perm, src = new(E, dtype=i32), new(E + 1, dtype=i32), new(T, k, dtype=i32), new(T * k, dtype=i32)
    xq, xs = new(T * k, H, dtype=torch.uint8), new(T * k)
    m.moe_permute(p, idx, x, counts, offsets, perm, src, xq, xs, G.workspace(p))
    # one token's codes: those of the row of its first slot
    codes, scale = xq[perm[:, 0].long()], xs[perm[:, 0].long()]
    out = dispatched(m.make_rows(T, H, E, k, torch.float8_e4m3fn), idx, codes, scale)
    for name, want in (("counts", counts), ("offsets", offsets), ("perm", perm), ("src_row", src),
                       ("x_rows", xq), ("scale_rows", xs)):
        assert torch.equal(out[name], want), name


@pytest.mark.parametrize("k", [1, 2, 3, 4])
@pytest.mark.parametrize("H", [8192, 2880, 8191, 4001])
@pytest.mark.parametrize("T,dtype", [(200, "bf16"), (200, "f32"), (700, "f16")])
def test_combine_backward_of_few_slots(T, dtype, H, k):
    # more tokens than multiprocessors and up to four slots: rows of several steps of a ring of
    # three stages, in whole vectors and in vectors of their own, with masked slots
    g, t, m, E = gen(T + H + k), B.DTYPES[dtype], G.lib(), 16
    idx = B.routing(T, E, k, g, 0.2)
    _, offsets, perm, _ = B.order(idx, E)
    rows, dout = torch.randn(T * k, H, generator=g).to(t), torch.randn(T, H, generator=g).to(t)
    w = torch.rand(T, k, generator=g)
    rows[int(offsets[E]):] = float("nan")
    w[perm < 0] = float("nan")
    drows, dw = new(T * k, H, dtype=t), new(T, k)
    m.moe_combine_backward(m.make_rows(T, H, E, k, t), dout.cuda(), rows.cuda(), perm.cuda(), offsets.cuda(),
                           w.cuda(), drows, dw)
    assert m.moe_get_last_error() == 0
    ref, rw, mag = B.combine_backward(dout, rows, perm, w)
    B.within(drows, ref, B.store(t, ref) + B.U * ref.abs(), "drows")
    B.within(dw, rw, (B.chain(H) + 2) * B.U * mag, "dw")


# buffers off 16-byte boundaries: a warp or a block per token, one and several steps of a row,
# groups of slots, the four-slot form, one launch and more, several blocks of columns
@pytest.mark.parametrize("T,H,k", [(5, 8193, 9), (19, 1031, 3), (700, 100, 9), (700, 100, 2), (700, 250, 9),
                                   (700, 1031, 2), (700, 8193, 2), (300, 8193, 9), (5000, 250, 2), (5000, 100, 9)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_misaligned_buffers_in_every_variant(T, H, k, dtype):
    g, t, m, E = gen(T + H + k), B.DTYPES[dtype], G.lib(), 24
    idx = B.routing(T, E, k, g, 0.2)
    _, offsets, perm, src = B.order(idx, E)
    x, rows = torch.randn(T, H, generator=g).to(t), torch.randn(T * k, H, generator=g).to(t)
    rows[int(offsets[E]):] = float("nan")
    w = torch.rand(T, k, generator=g)
    at = lambda v, off=1: offset_copy(v.cuda(), off)
    r = m.make_rows(T, H, E, k, t)
    bits = {2: torch.int16, 4: torch.int32}[x.element_size()]
    want = x.view(bits)[src.long().clamp(min=0)]
    want[src < 0] = 0
    for off in (1, 2, 4):
        out = dispatched(r, idx.cuda(), at(x, off))
        check_order(out, idx, E)
        assert torch.equal(out["x_rows"].view(bits).cpu(), want), off
    res, drows, dw = at(torch.zeros(T, H, dtype=t)), at(torch.zeros(T * k, H, dtype=t)), new(T, k)
    for extra in (x, None):
        m.moe_combine(r, at(rows), perm.cuda(), w.cuda(), None if extra is None else at(extra), res)
        ref, mag = B.combine(rows, perm, w, extra)
        B.within(res.clone(), ref, B.store(t, ref) + (k + 2) * B.U * mag, "out")
    m.moe_combine_backward(r, at(x), at(rows), perm.cuda(), offsets.cuda(), w.cuda(), drows, dw)
    assert m.moe_get_last_error() == 0
    ref, rw, mag = B.combine_backward(x, rows, perm, w)
    B.within(drows.clone(), ref, B.store(t, ref) + B.U * ref.abs(), "drows")
    B.within(dw, rw, (B.chain(H) + 2) * B.U * mag, "dw")


@pytest.mark.parametrize("T,H,k", [(37, 1031, 3), (300, 250, 9), (700, 8192, 2), (700, 1031, 9), (5000, 250, 4)])
@pytest.mark.parametrize("off", [1, 2, 4, 8])
def test_misaligned_codes_in_every_unit(T, H, k, off):
    # 8-bit rows in units of one to eight bytes, in one launch and in more
    g, m, E, t = gen(T + H + off), G.lib(), 24, torch.float8_e4m3fn
    idx = B.routing(T, E, k, g, 0.2)
    src = B.order(idx, E)[3].long()
    x = torch.randint(0, 255, (T, H), generator=g, dtype=torch.uint8)
    scale = torch.rand(T, generator=g)
    out = dispatched(m.make_rows(T, H, E, k, t), idx.cuda(), offset_copy(x.cuda(), off).view(t), scale.cuda())
    assert m.moe_get_last_error() == 0
    check_order(out, idx, E)
    want, want_scale = x[src.clamp(min=0)], scale[src.clamp(min=0)]
    want[src < 0], want_scale[src < 0] = 0, 0
    assert torch.equal(out["x_rows"].view(torch.uint8).cpu(), want)
    assert torch.equal(out["scale_rows"].cpu(), want_scale)
