"""The mixture-of-experts layer over packed weights against a plain 64-bit implementation."""
import numpy as np
import pytest
import torch

import oracle
import post_weight_quantization_21_b200 as g

import gpu_support as S

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # fp32 rounding


def _experts(e, rows, cols, bits, gs, gen, dev):
    """((packed, scales, zeros) on the device, What and scale * (q + zero) [e, rows, cols] fp64)"""
    codes = torch.randint(0, 2 ** bits, (e, rows, cols), generator=gen)
    ng = cols // gs if gs else 1
    scales = ((torch.rand(e, rows, ng, generator=gen) + 0.5) / (cols ** 0.5 * 2 ** (bits - 2))).float()
    zeros = torch.randint(0, 2 ** bits, (e, rows, ng), generator=gen, dtype=torch.int32)
    packed = oracle.pack_codes(codes.reshape(e * rows, cols).numpy(), bits).reshape(e, rows, -1)
    rep = gs or cols
    s, q, z = scales.double().repeat_interleave(rep, -1), codes.double(), zeros.double().repeat_interleave(rep, -1)
    return (torch.from_numpy(packed).to(dev), scales.to(dev), zeros.to(dev)), (s * (q - z)).to(dev), (s * (q + z)).to(dev)


class Case:
    def __init__(self, t, e, top, d, f, bits, gs, xdt, ydt, act, seed=0):
        gen = torch.Generator().manual_seed(seed + t * 31 + e * 7 + d)
        dev = S.dev()
        self.t, self.e, self.top, self.d, self.f, self.bits, self.gs, self.ydt, self.act = t, e, top, d, f, bits, gs, ydt, act
        self.x = torch.randn(t, d, generator=gen).to(xdt).to(dev)
        self.router = (torch.randn(e, d, generator=gen) * (2.0 / d ** 0.5)).to(xdt).to(dev)
        self.up, self.Wu, self.Au = _experts(e, f, d, bits, gs, gen, dev)
        self.gate, self.Wg, self.Ag = _experts(e, f, d, bits, gs, gen, dev) if act == g.GPTQ_ACT_SILU_GATED else (None,) * 3
        self.down, self.Wd, self.Ad = _experts(e, d, f, bits, gs, gen, dev)
        self.ids = torch.full((t, top), -7, dtype=torch.int32, device=dev)
        self.w = torch.full((t, top), float("nan"), device=dev)
        self.Y = torch.full((t, d), float("nan"), device=dev, dtype=ydt)
        self.st = torch.zeros(2, dtype=torch.int32, device=dev)
        self.ws = torch.full((g.gptq_moe_workspace_size(t, d, f, e, top),), 0xFF, dtype=torch.uint8, device=dev)

    def run(self, flags=0, router=True, stream=None):
        g.gptq_moe_layer(self.x, self.router if router else None, self.up, self.gate, self.down, self.ids, self.w, self.Y,
                         self.st, self.ws, self.bits, self.gs, self.act, flags, stream)
        return self.Y

    def check_routing(self, renorm):
        """ids: the largest logits, in order, wherever the fp64 logits lie further apart than the fp32 sums' error
        (d roundings of sum |x r| at most); weights: their softmax, to the logits' errors and a few roundings."""
        x, r = self.x.double(), self.router.double()
        l = x @ r.t()
        err = self.d * U * (x.abs() @ r.abs().t()).amax(1)
        p = torch.softmax(l, -1)
        order = torch.argsort(l, dim=1, descending=True, stable=True)
        ls = torch.gather(l, 1, order)
        n = min(self.top + 1, self.e)
        gap = (ls[:, :n - 1] - ls[:, 1:n]).amin(1) if n > 1 else torch.full_like(err, 1.0)
        clear = gap > 2 * err
        assert clear.float().mean() > 0.8
        ids = self.ids.long()
        assert torch.equal(ids[clear], order[clear, :self.top])
        assert all(len(set(row)) == self.top for row in ids.tolist())
        w = torch.gather(p, 1, ids)
        if renorm:
            w = w / w.sum(1, keepdim=True)
        tol = w * (4 * err[:, None] + (self.e + 40) * U)
        assert ((self.w.double() - w).abs() <= tol).all()

    def check(self):
        """Y against fp64 with the device's own choice and weights.  A product is formed as s (sum q x - z sum x), so the
        terms of its sum are s q x and s z x; with n roundings on a term's way the fp32 sum is off by at most n u
        sum s (q + z) |x|.  n: at most two fp16 terms of x, each 8 tensor-core steps that add 16 exact products, counted
        as 17 additions that may truncate (2 u each): 544; sum x and its product with z: 36; the scale's product, the
        chunks of 128 columns and 8 warps: 2 + chunks + 8.  x itself: 2^-24 of each value where it takes two terms
        (fp32), exact where one holds it, and in both 2^-32 of the block's largest for values too small for fp16.
        silu's slope is below 1.1 and its own evaluation a few u; the intermediate takes two terms (2^-24 of each value),
        or one for a bf16 result (2^-12).
        For a 16-bit result the codes are fp16 subnormals q 2^(p - 24), which the tensor core aligns as if they were 2^-14:
        each of the 17 additions of the 8 steps of at most two terms may be off by 2^-24 of 2^-13 times the block's largest
        |x|, in units of the code (2^-24) and with 2^-p <= 1: 272 * 2^-13 s max|x| per block of 128."""

        def product(W, A, scales, v, ev, own):  # W v with |v's error| <= ev; own: v's rounding to its terms
            n = 544 + 36 + 10 + -(-v.numel() // 128)
            ev = ev + own * v.abs() + 2.0 ** -32 * v.abs().max()
            tol = n * U * (A @ v.abs()) + A @ ev
            if self.ydt != torch.float32:
                s = scales.double().repeat_interleave(self.gs or v.numel(), -1)
                pad = (0, -v.numel() % 128)
                s = torch.nn.functional.pad(s, pad).view(s.shape[0], -1, 128).amax(-1)
                big = torch.nn.functional.pad(v.abs() + ev, pad).view(-1, 128).amax(-1)
                tol = tol + 272 * 2.0 ** -13 * (s @ big)
            return W @ v, tol

        x, ids, w = self.x.double(), self.ids.long(), self.w.double()
        xown = 2.0 ** -24 if self.x.dtype == torch.float32 else 0.0
        hown = 2.0 ** -12 if self.ydt == torch.bfloat16 else 2.0 ** -24
        y, tol = torch.zeros_like(x), torch.zeros_like(x)
        for k in range(self.top):
            for t in range(self.t):
                e = int(ids[t, k])
                if not 0 <= e < self.e:
                    continue
                u, eu = product(self.Wu[e], self.Au[e], self.up[1][e], x[t], 0.0, xown)
                if self.act == g.GPTQ_ACT_SILU_GATED:
                    z, ez = product(self.Wg[e], self.Ag[e], self.gate[1][e], x[t], 0.0, xown)
                    sl = z * torch.sigmoid(z)
                    h = sl * u
                    eh = 1.1 * ez * (u.abs() + eu) + sl.abs() * eu + 16 * U * h.abs()
                else:
                    h, eh = torch.relu(u), eu
                v, ev = product(self.Wd[e], self.Ad[e], self.down[1][e], h, eh, hown)
                y[t] += w[t, k] * v
                tol[t] += w[t, k] * (ev + (2 + self.top) * U * v.abs())
        if self.ydt != torch.float32:
            tol = tol + torch.finfo(self.ydt).eps / 2 * (y.abs() + tol) + 2.0 ** -25
        assert torch.isfinite(self.Y).all()
        off = (self.Y.double() - y).abs()
        assert (off <= tol).all(), ((off / tol).max().item(), off.max().item())


SILU, RELU = g.GPTQ_ACT_SILU_GATED, g.GPTQ_ACT_RELU
bf, hf, ff = torch.bfloat16, torch.float16, torch.float32
CASES = [
    # t, e, top, d, f, bits, group, x, y, activation
    (1, 1, 1, 32, 32, 4, 0, bf, ff, RELU),
    (1, 4, 2, 128, 256, 4, 128, bf, bf, SILU),
    (3, 8, 2, 160, 96, 3, 32, hf, ff, SILU),       # cut-off last chunk, groups inside a chunk
    (5, 4, 4, 256, 384, 2, 64, ff, ff, SILU),
    (8, 3, 1, 1056, 544, 3, 0, ff, hf, RELU),
    (9, 2, 2, 512, 640, 4, 0, bf, ff, SILU),       # more than 8 tokens on an expert
    (33, 2, 1, 256, 288, 3, 0, hf, bf, SILU),      # lists that end inside a tile
    (64, 1, 1, 384, 128, 2, 128, bf, hf, RELU),    # every token on one expert
    (64, 256, 16, 128, 64, 4, 32, hf, ff, SILU),   # most experts, most choices
    (64, 40, 6, 1024, 512, 3, 128, ff, ff, SILU),
    (17, 5, 3, 2048, 1408, 4, 128, bf, ff, SILU),
    (2, 6, 2, 4096, 2176, 4, 128, hf, hf, SILU),
]


@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "_".join(map(str, c[:7])))
def test_layer_against_fp64(case, renorm):
    c = Case(*case)
    c.run(g.GPTQ_MOE_RENORMALIZE if renorm else 0)
    assert g.gptq_read_status(c.st)[0] == g.GPTQ_OK
    c.check_routing(renorm)
    c.check()


def test_ties_go_to_the_lowest_index():
    c = Case(4, 64, 8, 64, 32, 4, 0, bf, ff, RELU)
    c.router.zero_()
    c.run()
    assert c.ids.tolist() == [list(range(8))] * 4
    assert (c.w == 1.0 / 64).all()


def test_given_routing_with_repeats_and_bad_ids():
    """The caller's routing: an expert given twice counts twice; an id out of range adds nothing, is reported, and
    nothing else changes."""
    c = Case(4, 5, 3, 256, 160, 3, 32, bf, ff, SILU)
    gen = torch.Generator().manual_seed(1)
    c.w.copy_(torch.rand(4, 3, generator=gen))
    c.ids.copy_(torch.tensor([[0, 0, 4], [1, 2, 3], [4, 4, 4], [2, 0, 1]], dtype=torch.int32))
    c.run(router=False)
    assert g.gptq_read_status(c.st)[0] == g.GPTQ_OK
    c.check()
    good = c.Y.clone()
    c.ids[1, 1] = 5
    c.ids[3] = torch.tensor([-1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    c.run(router=False)
    code, detail = g.gptq_read_status(c.st)
    assert code == g.GPTQ_ERR_ARG and detail in (4, 9, 10, 11)
    c.check()
    assert torch.equal(c.Y[0], good[0]) and torch.equal(c.Y[2], good[2])
    assert (c.Y[3] == 0).all()


@pytest.mark.parametrize("t,e,top", [(8, 8, 8), (8, 9, 2), (9, 8, 2), (3, 32, 16), (3, 33, 16), (2, 64, 16), (5, 65, 3), (1, 255, 16)])
def test_choice_over_any_number_of_experts(t, e, top):
    """Around the counts at which the logits get a launch of their own, and around the 32 experts that a warp holds at a
    time; as many choices as experts."""
    c = Case(t, e, top, 64, 32, 4, 0, hf, ff, RELU)
    c.run(g.GPTQ_MOE_RENORMALIZE)
    assert g.gptq_read_status(c.st)[0] == g.GPTQ_OK
    c.check_routing(1)
    c.check()


@pytest.mark.parametrize("t,e,top", [(64, 20, 5), (64, 256, 16), (40, 2, 16)])
def test_given_routing_of_many_tokens(t, e, top):
    """The caller's routing with repeats, more pairs than a warp looks at in one step; one expert is never named."""
    c = Case(t, e, top, 96, 64, 3, 32, bf, ff, RELU)
    gen = torch.Generator().manual_seed(t + e)
    c.w.copy_(torch.rand(t, top, generator=gen))
    c.ids.copy_(torch.randint(0, e - 1, (t, top), generator=gen).to(torch.int32))
    c.run(router=False)
    assert g.gptq_read_status(c.st)[0] == g.GPTQ_OK
    c.check()


def test_deterministic_and_inputs_untouched():
    c = Case(40, 8, 3, 512, 256, 4, 128, hf, ff, SILU)
    before = [t.clone() for t in (c.x, c.router, *c.up, *c.gate, *c.down)]
    y = c.run().clone()
    c.ws.fill_(0x7F)
    assert torch.equal(c.run(), y)
    for t, b in zip((c.x, c.router, *c.up, *c.gate, *c.down), before):
        assert torch.equal(t, b)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_token_stays_alone(bad):
    c = Case(12, 3, 2, 256, 128, 4, 0, bf, ff, SILU)
    y = c.run().clone()
    ids = c.ids.clone()
    c.x[5, 17] = bad
    c.run()
    keep = [i for i in range(12) if i != 5]
    assert torch.equal(c.Y[keep], y[keep]) and torch.equal(c.ids[keep], ids[keep])
    assert not torch.isfinite(c.Y[5]).any()
    assert ((c.ids >= 0) & (c.ids < 3)).all()


def test_large_values_do_not_overflow_early():
    """fp32 tokens near the type's end with tiny grid scales: the terms and the sums over codes stay finite."""
    c = Case(2, 2, 1, 64, 32, 4, 0, ff, ff, RELU)
    c.x.mul_(2.0 ** 110)
    c.up[1].mul_(2.0 ** -110)
    c.Wu.mul_(2.0 ** -110)
    c.Au.mul_(2.0 ** -110)
    c.ids.fill_(1)
    c.w.fill_(0.5)
    c.run(router=False)
    c.check()


@pytest.mark.parametrize("bits,gs", [(4, 128), (3, 128), (2, 32), (3, 0)])
def test_grids_and_outputs_on_any_alignment(bits, gs):
    """Scales, zeros, routing, Y and status as views that start one value into their memory."""
    c = Case(3, 4, 2, 256, 256, bits, gs, bf, hf, SILU)

    def shifted(t):
        buf = torch.zeros(t.numel() + 1, dtype=t.dtype, device=t.device)
        buf[1:] = t.reshape(-1)
        return buf[1:].view(t.shape)

    for name in ("up", "gate", "down"):
        w = getattr(c, name)
        setattr(c, name, (w[0], shifted(w[1]), shifted(w[2])))
    c.ids, c.w, c.Y, c.st = shifted(c.ids), shifted(c.w), shifted(c.Y), shifted(c.st)
    c.run()
    assert g.gptq_read_status(c.st)[0] == g.GPTQ_OK
    c.check_routing(False)
    c.check()


def test_no_tokens_is_no_work():
    c = Case(1, 2, 1, 64, 32, 4, 0, bf, ff, RELU)
    n0 = g.gptq_kernel_launches()
    g.gptq_moe_layer(c.x[:0], c.router, c.up, None, c.down, c.ids[:0], c.w[:0], c.Y[:0], c.st, c.ws, 4, 0, RELU)
    assert g.gptq_kernel_launches() == n0


def test_on_another_stream_and_in_a_graph():
    c = Case(6, 8, 2, 256, 384, 4, 128, bf, ff, SILU)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.run(stream=side)
    side.synchronize()
    c.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    gen = torch.Generator().manual_seed(2)
    for _ in range(3):
        c.x.copy_(torch.randn(c.t, c.d, generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        c.check_routing(False)
        c.check()
    assert g.gptq_read_status(c.st)[0] == g.GPTQ_OK
