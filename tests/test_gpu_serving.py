"""The serving operators together, as they are used: a block calibrated on its fp8 products, and experts solved by
the quantizer and run as a mixture."""
import numpy as np
import pytest
import torch

import oracle
import post_weight_quantization_21_b200 as g
from post_weight_quantization_21_b200 import pipeline as P

import gpu_support as S
from test_gpu_fp8 import _check_matmul, _ref_quantize
from test_gpu_moe import Case

pytestmark = pytest.mark.gpu


def test_fp8_products_in_the_quantized_forward():
    """linears = "fp8": the forward's products are those of the codes and of the activations rounded to e4m3.  Every
    product the forward makes is checked against fp64 on the operands it had."""
    cfg = P.BlockConfig(d_model=256, n_heads=4, d_ffn=640, seq_len=64, bits=4, group_size=128, linears="fp8")
    dev = S.dev()
    p = P.make_block(cfg, seed=5, device=dev)
    x = torch.randn(6 * cfg.seq_len, cfg.d_model, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(dev)
    bq = P.BlockQuantizer(cfg, device=dev, chunk_seqs=3)
    layers, y = bq.quantize_block(p, x)
    seen = {}
    products = P.Fp8Linears(cfg, layers, bq.status[14])

    def watched(names, act):
        out = products(names, act)
        for nm, o in zip(names, out):
            seen[nm] = (act, o)
        return out

    again = P.block_forward(cfg, p, x[:3 * cfg.seq_len], products=watched).to(x.dtype)
    assert torch.equal(again, y[:3 * cfg.seq_len])
    assert set(seen) == set(P.LINEARS)
    for nm, (act, out) in seen.items():
        q, s = _ref_quantize(act, 1)
        rep = cfg.group_size
        grid = lambda t: t.double().repeat_interleave(rep, dim=1)
        codes = layers[nm].codes.double()
        np.testing.assert_array_equal(products.B[nm].double().cpu().numpy(),
                                      (codes - grid(layers[nm].zeros)).cpu().numpy())
        A, sa = torch.from_numpy(q).to(dev), torch.from_numpy(s).to(dev)
        _check_matmul(out, A, sa, products.B[nm], products.scales[nm], 1)
    assert g.gptq_read_status(bq.status[14])[0] == g.GPTQ_OK


def test_quantized_experts_through_the_layer():
    """Experts solved with LayerSolver, stacked, and run as a mixture: the result is that of their quantized weights."""
    d, f, E, T, K = 256, 384, 3, 5, 2
    dev = S.dev()
    gen = torch.Generator().manual_seed(11)
    cal = torch.randn(512, d, generator=gen).to(torch.bfloat16).to(dev)
    cal_f = torch.relu(torch.randn(512, f, generator=gen)).to(torch.bfloat16).to(dev)

    def solve(m, k, X):
        parts = []
        for _ in range(E):
            s = g.LayerSolver(m, k, X.shape[0], 4, 128, 128, device=dev)
            s.W.copy_(torch.randn(m, k, generator=gen) / k ** 0.5)
            s.X.copy_(X)
            s.run()
            s.check_status()
            parts.append((s.packed, s.scales, s.zeros))
        return tuple(torch.stack(t) for t in zip(*parts))

    def values(w, k):  # What and scale * (q + zero) in fp64
        q = torch.from_numpy(oracle.unpack_codes(w[0].cpu().numpy().reshape(-1, k // 8), 4, k)).double().to(dev)
        q = q.reshape(*w[0].shape[:2], k)
        s, z = (t.double().repeat_interleave(128, -1) for t in w[1:])
        return s * (q - z), s * (q + z)

    c = Case.__new__(Case)
    c.t, c.e, c.top, c.d, c.f, c.bits, c.gs, c.ydt, c.act = T, E, K, d, f, 4, 128, torch.float32, g.GPTQ_ACT_SILU_GATED
    c.up, c.gate, c.down = solve(f, d, cal), solve(f, d, cal), solve(d, f, cal_f)
    (c.Wu, c.Au), (c.Wg, c.Ag), (c.Wd, c.Ad) = values(c.up, d), values(c.gate, d), values(c.down, f)
    c.x = torch.randn(T, d, generator=gen).to(torch.bfloat16).to(dev)
    c.router = torch.randn(E, d, generator=gen).to(torch.bfloat16).to(dev)
    c.ids = torch.empty(T, K, dtype=torch.int32, device=dev)
    c.w = torch.empty(T, K, device=dev)
    c.Y = torch.empty(T, d, device=dev)
    c.st = torch.zeros(2, dtype=torch.int32, device=dev)
    c.ws = torch.empty(g.gptq_moe_workspace_size(T, d, f, E, K), dtype=torch.uint8, device=dev)
    c.run(g.GPTQ_MOE_RENORMALIZE)
    c.check_routing(True)
    c.check()
    dense = torch.empty(E, f, d, device=dev)
    for e in range(E):  # the dequantizer's weights are the same ones, rounded to fp32 once or twice
        g.gptq_dequantize(c.up[0][e], c.up[1][e], c.up[2][e], 4, 128, dense[e])
    assert ((dense.double() - c.Wu).abs() <= 2.0 ** -23 * c.Wu.abs()).all()
    assert g.gptq_read_status(c.st)[0] == g.GPTQ_OK
