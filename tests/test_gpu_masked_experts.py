"""Batches with masked slots through the experts: moe_add_rmsnorm's codes, moe_dispatch,
moe_expert_ffn on fewer than R rows and moe_combine, and the serving step of
examples/moe_block.py against the CPU oracle."""
import os
import sys

import numpy as np
import pytest
import torch

import _block as B
import _gpu as G
import moe_inputs as mi

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

FP8 = mi.MoEConfig("masked_fp8", T=300, H=512, I=256, E=16, k=4)
BLOCK = FP8.with_(name="masked_fp8_block", wfmt="fp8_block")
MX = FP8.with_(name="masked_mxfp4", wfmt="mxfp4")
E4M3 = torch.float8_e4m3fn


def fill(*shape, dtype=torch.float32):
    """A device buffer of bytes 0xFF: NaN in every float type."""
    t = torch.empty(*shape, dtype=dtype, device="cuda")
    t.view(torch.uint8).fill_(0xFF)
    return t


# FP8: tiles of 128 rows, SM pairs (256, with and without small tiles), their single-SM form;
# MXFP4: single-SM kernels, and SM pairs on packed weights
FORMS = [(FP8, dict(), False), (FP8, dict(tile_n=256), False), (FP8, dict(tile_n=256, pair_small=0), False),
         (FP8, dict(tile_n=256, gemm_1cta=1), False), (BLOCK, dict(), False), (MX, dict(), False), (MX, dict(), True)]


@pytest.mark.parametrize("masked", [0.0, 0.4, 0.98, 1.0])
@pytest.mark.parametrize("cfg,choices,packed", FORMS, ids=lambda v: getattr(v, "name", None) or str(v))
def test_masked_slots_through_the_experts(orc, tuning, cfg, choices, packed, masked):
    m = G.lib()
    tuning(**choices)
    T, H, E, k, R = cfg.T, cfg.H, cfg.E, cfg.k, cfg.T * cfg.k
    g = torch.Generator().manual_seed(17)
    idx = B.routing(T, E, k, g, masked)
    if masked == 1.0:
        idx[:] = -1
    x, h = (torch.randn(T, H, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    w = torch.rand(T, k, generator=g)
    w[idx < 0] = float("nan")
    q, q_scale = fill(T, H, dtype=E4M3), fill(T)
    gamma = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    m.moe_add_rmsnorm(m.make_norm(T, H, torch.bfloat16), x, None, gamma, None, None, q, q_scale)

    r = m.make_rows(T, H, E, k, E4M3)
    i32 = torch.int32
    counts, offsets, perm, src = fill(E, dtype=i32), fill(E + 1, dtype=i32), fill(T, k, dtype=i32), fill(R, dtype=i32)
    rows, scales = fill(R, H, dtype=E4M3), fill(R)
    m.moe_dispatch(r, idx.cuda(), q, q_scale, counts, offsets, perm, src, rows, scales,
                   fill(m.moe_rows_workspace_bytes(r), dtype=torch.uint8))
    assert torch.equal(perm.cpu(), B.order(idx, E)[2])

    inp = G.gpu_inputs(cfg)
    wt = G.pack(cfg, inp) if packed else inp
    p = G.problem(cfg, packed=packed)
    y = fill(R, H, dtype=torch.bfloat16)
    m.moe_expert_ffn(p, offsets, rows, scales, None, wt["w13"], wt["w13_scale"], wt["w2"], wt["w2_scale"], y,
                     fill(m.moe_workspace_bytes(p), dtype=torch.uint8))
    out = fill(T, H, dtype=torch.bfloat16)
    m.moe_combine(m.make_rows(T, H, E, k, torch.bfloat16), y, perm, w.cuda(), h, out)
    assert m.moe_get_last_error() == 0

    live = int(offsets[E])
    assert live == int((idx >= 0).sum())
    assert (y[live:].view(torch.uint8) == 0xFF).all()  # rows past the last routed one are not written
    if live:
        hw = G.host(inp)
        fmt = {"fp8": orc.FP8, "fp8_block": orc.FP8_BLOCK, "mxfp4": orc.MXFP4}[cfg.wfmt]
        codes = rows[:live].view(torch.uint8).cpu().numpy()
        ref = orc.expert_rows(fmt, offsets.cpu().numpy(), codes, scales[:live].cpu().numpy(),
                              np.ones(live, np.float32), hw["w13"], hw["w13_scale"], hw["w2"], hw["w2_scale"])
        G.assert_close(G.bf16_values(G.bf16_bits(y[:live])), ref, cfg.name,
                       bf16_store_allowance=cfg.wfmt == "fp8_block")
    ref, mag = B.combine(y.cpu(), perm.cpu(), w, h.cpu())
    B.within(out, ref, B.store(torch.bfloat16, ref) + (k + 2) * B.U * mag, "out")
    none = (idx < 0).all(1)
    assert torch.equal(out[none], h[none])


@pytest.mark.parametrize("T", [1, 96, 700])
def test_serving_step_against_the_oracle(orc, T):
    # norm -> router -> dispatch -> experts -> combine: the step's bf16 rows and codes are the norm's in 64
    # bits, each rounded once; the oracle routes those rows, runs the experts on those codes (one at a tie may
    # go either way, which the bars below do not count) and weighs their unrounded outputs.  A small
    # residual, so that the layer's bars fall on the experts' part
    import moe_block as ex
    m = G.lib()
    cfg = mi.MoEConfig("block", T=T, H=512, I=256, E=16, k=4)
    inp = G.gpu_inputs(cfg)
    hw = G.host(inp)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = inp["x"] * 2.0 ** -6
    residual = (2.0 ** -6 * torch.randn(T, cfg.H, device="cuda", generator=g)).to(torch.bfloat16)
    gamma = (1 + 0.2 * torch.randn(cfg.H, device="cuda", generator=g)).to(torch.bfloat16)
    out, h, y = ex.serve(G.problem(cfg), x, residual, gamma, inp["router_w"], inp["w13"], inp["w13_scale"],
                         inp["w2"], inp["w2_scale"])
    assert m.moe_get_last_error() == 0
    q, qs = fill(T, cfg.H, dtype=E4M3), fill(T)
    m.moe_add_rmsnorm(m.make_norm(T, cfg.H, torch.bfloat16, eps=ex.EPS), x, residual, gamma, None, None, q, qs)
    _, y64, _ = B.norm(x.cpu(), residual.cpu(), gamma.cpu(), ex.EPS)
    c = (B.chain(cfg.H) / 2 + 12) * B.U
    B.within(y, y64, B.store(torch.bfloat16, y64) + c * y64.abs(), "y")
    s64 = y64.abs().amax(1) / 448.0
    B.within(qs, s64, (c + 2 * B.U) * s64, "q_scale")
    B.within(q.cpu().double() * qs.cpu().double()[:, None], y64,
             (2.0 ** -4 + 2 * c) * y64.abs() + 2.0 ** -10 * s64[:, None] * (1 + c), "q")
    codes, scale = q.view(torch.uint8).cpu().numpy(), qs.cpu().numpy()
    idx, w = orc.topk(orc.router_logits(G.bf16_bits(y), hw["router_w"]), cfg.k)
    _, off, perm, src = orc.permute(idx, cfg.E)
    rows = orc.expert_rows(orc.FP8, off, codes[src], scale[src], np.ones(T * cfg.k, np.float32), hw["w13"],
                           hw["w13_scale"], hw["w2"], hw["w2_scale"])
    moe = (rows[perm] * w[..., None]).sum(1)
    # what is left once h's own value and the bf16 store of the sum (half a step) are taken off
    got, h64 = out.cpu().double().numpy(), (x.double() + residual.double()).cpu().numpy()
    err = np.abs(got - (h64 + moe)) - G.bf16_half_ulp(got)
    G.assert_close(moe + np.maximum(err, 0.0), moe, "serving step")
