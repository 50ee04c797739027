"""The 8-bit floating-point operands and their product against plain 64-bit implementations."""
import numpy as np
import pytest
import torch

import oracle
import post_weight_quantization_21_b200 as g

import gpu_support as S

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _ref_quantize(x, block_rows):
    """(values q, scales) in fp64: scale 2^e, the smallest e >= -126 with max|finite x| <= 448 2^e (1 for a zero
    block); q = x / scale rounded to a multiple of e4m3's step at its magnitude, ties to even."""
    x = x.double().cpu().numpy()
    m, k = x.shape
    mb, kb = -(-m // block_rows), -(-k // 128)
    q, scales = np.empty_like(x), np.empty((mb, kb))
    for i in range(mb):
        for j in range(kb):
            at = np.s_[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128]
            blk = x[at]
            fin = np.isfinite(blk)
            a = np.abs(blk[fin]).max(initial=0.0)
            e = -126
            while a > 448.0 * 2.0 ** e:
                e += 1
            s = 2.0 ** e if a > 0 else 1.0
            v = np.where(fin, blk, np.nan) / s
            with np.errstate(invalid="ignore"):
                mag = np.abs(v)
                exp = np.floor(np.log2(np.where(mag > 0, mag, 1.0)))
                step = 2.0 ** (np.maximum(exp, -6) - 3)
                q[at], scales[i, j] = np.round(v / step) * step, s
    return q, scales


def _quantize(x, block_rows):
    m, k = x.shape
    Q = torch.full((m, k), 1.0, device=x.device).to(F8)
    sc = torch.full((-(-m // block_rows), -(-k // 128)), float("nan"), device=x.device)
    g.gptq_fp8_quantize(x, Q, sc, block_rows)
    return Q, sc


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,block_rows", [(1, 16, 1), (3, 128, 1), (37, 144, 1), (5, 4096 + 48, 1), (130, 2048, 1),
                                            (1, 16, 128), (127, 128, 128), (129, 400, 128), (300, 1040, 128)])
def test_quantize_matches_the_definition(m, k, block_rows, dtype):
    """Every code and scale equal: the division is by a power of two, so nothing but the one rounding is left."""
    gen = torch.Generator().manual_seed(m * 7 + k)
    x = torch.randn(m, k, generator=gen) * torch.exp2(torch.randint(-20, 12, (m, 1), generator=gen).float())
    x[:, ::37] *= 15.0
    x = x.to(dtype).to(S.dev())
    Q, sc = _quantize(x, block_rows)
    q_ref, s_ref = _ref_quantize(x, block_rows)
    np.testing.assert_array_equal(sc.double().cpu().numpy(), s_ref)
    np.testing.assert_array_equal(Q.double().cpu().numpy(), q_ref)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_edges(block_rows):
    """Zero blocks, single extreme values, exact powers of the scale's border, subnormals, NaN and infinities."""
    x = torch.zeros(9, 256)
    x[1, 5] = 448.0                      # border: scale 1
    x[2, 5] = 448.5                      # just above: scale 2
    x[3, 128:] = torch.finfo(torch.float32).max
    x[4, 0], x[4, 1] = 1e-45, -1e-40     # subnormal fp32: the scale stops at 2^-126
    x[5, 7], x[5, 8], x[5, 9] = float("nan"), 3.0, float("inf")
    x[6, 7] = float("-inf")              # nothing finite but zeros
    x[7] = torch.arange(256) * 1.0625    # ties of e4m3
    x[8] = -torch.arange(256) * 2.0 ** -130
    for rows in ([[i] for i in range(9)] if block_rows == 128 else [list(range(9))]):
        xs = x[rows].contiguous().to(S.dev())
        Q, sc = _quantize(xs, block_rows)
        q_ref, s_ref = _ref_quantize(xs, block_rows)
        np.testing.assert_array_equal(sc.double().cpu().numpy(), s_ref)
        np.testing.assert_array_equal(Q.double().cpu().numpy(), q_ref)


@pytest.mark.parametrize("m,k,bits,gs", [(1, 32, 4, 0), (33, 96, 3, 0), (7, 4096 + 32, 2, 0), (65, 512, 3, 128),
                                         (40, 1024, 4, 256), (129, 640, 2, 128)])
def test_from_packed_is_exact(m, k, bits, gs):
    rng = np.random.default_rng(m + k)
    codes = rng.integers(0, 2 ** bits, size=(m, k))
    ng = k // gs if gs else 1
    scales = rng.uniform(1e-3, 5e-2, size=(m, ng)).astype(np.float32)
    zeros = rng.integers(0, 2 ** bits, size=(m, ng)).astype(np.int32)
    dev = S.dev()
    Q = torch.zeros(m, k, device=dev).to(F8)
    qs = torch.full((m, -(-k // 128)), float("nan"), device=dev)
    g.gptq_fp8_from_packed(torch.from_numpy(oracle.pack_codes(codes, bits)).to(dev), torch.from_numpy(scales).to(dev),
                           torch.from_numpy(zeros).to(dev), bits, gs, Q, qs)
    rep = gs or k
    np.testing.assert_array_equal(Q.double().cpu().numpy(), codes - np.repeat(zeros, rep, axis=1))
    np.testing.assert_array_equal(qs.cpu().numpy(), np.repeat(scales, rep, axis=1)[:, ::128])


def _operands(m, n, k, rows, seed, dev):
    gen = torch.Generator().manual_seed(seed)
    kb = -(-k // 128)
    A = (torch.randn(m, k, generator=gen) * 60).clamp(-448, 448).to(F8).to(dev)
    B = (torch.randn(n, k, generator=gen) * 60).clamp(-448, 448).to(F8).to(dev)
    sa = ((torch.rand(m, kb, generator=gen) + 0.1) * 0.02).to(dev)
    sb = ((torch.rand(-(-n // rows), kb, generator=gen) - 0.3) * 0.01).to(dev)
    return A, sa, B, sb


def _matmul(A, sa, B, sb, rows, dtype, stream=None):
    m, n, k = A.shape[0], B.shape[0], A.shape[1]
    Y = torch.full((m, n), float("nan"), device=A.device, dtype=dtype)
    st = torch.zeros(2, dtype=torch.int32, device=A.device)
    ws = torch.empty(max(256, g.gptq_fp8_matmul_workspace_size(m, n, k)), dtype=torch.uint8, device=A.device)
    g.gptq_fp8_matmul(A, sa, B, sb, rows, Y, st, ws, stream)
    assert g.gptq_read_status(st, stream)[0] == g.GPTQ_OK
    return Y


def _check_matmul(Y, A, sa, B, sb, rows):
    """Against fp64.  With T = sum_b |sa sb| sum_t |a_t b_t| the error of the fp32 work is at most u T (u = 2^-24) times
    the roundings on one term's way: inside a block of 128 the tensor core's sum, counted as 128 additions that may
    truncate (2 u each), then two scale products and kb additions outside (and the splits' 16): 256 + 2 + kb + 16.
    A 16-bit result is rounded once more, by at most half a step (eps / 2) of its value."""
    n, k = B.shape
    kb = -(-k // 128)
    Ad, Bd = A.double(), B.double()
    sad, sbd = sa.double(), sb.double().repeat_interleave(rows, dim=0)[:n]
    spread = lambda s: s.repeat_interleave(128, dim=1)[:, :k]
    ref = (Ad * spread(sad)) @ (Bd * spread(sbd)).t()
    T = (Ad.abs() * spread(sad.abs())) @ (Bd.abs() * spread(sbd.abs())).t()
    tol = (274 + kb) * 2.0 ** -24 * T
    if Y.dtype != torch.float32:
        tol = tol + torch.finfo(Y.dtype).eps / 2 * (ref.abs() + tol) + 2.0 ** -25  # fp16 subnormals: half of 2^-24
    assert torch.isfinite(Y).all()
    bad = (Y.double() - ref).abs() > tol
    assert not bad.any(), (bad.sum().item(), ((Y.double() - ref).abs() / tol).max().item())
    return ref


# token counts around each tile width, weight rows around a tile, block counts with a cut-off last block
SHAPES = [(1, 1, 16), (1, 128, 128), (2, 129, 144), (16, 64, 4096), (17, 300, 256), (33, 4096, 1040), (65, 127, 2176),
          (129, 513, 384), (257, 1000, 1536), (1, 12288, 4096), (640, 4097, 512), (2048, 2304, 272), (8, 300, 1040), (9, 300, 1040), (333, 1000, 4224), (257, 770, 6528),
          (300, 4104, 11008), (385, 512, 2192)]


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_matmul_against_fp64(m, n, k, dtype, rows):
    A, sa, B, sb = _operands(m, n, k, rows, m + n + k, S.dev())
    _check_matmul(_matmul(A, sa, B, sb, rows, dtype), A, sa, B, sb, rows)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("m,n,k", [(9, 33, 272), (15, 200, 144), (16, 129, 2064), (16, 4096, 8192), (16, 4112, 8192), (17, 48, 256)])
def test_matmul_of_up_to_16_tokens(m, n, k, rows):
    """The second group of eight tokens, and both sides of the weights' size that ends it."""
    A, sa, B, sb = _operands(m, n, k, rows, m + n, S.dev())
    _check_matmul(_matmul(A, sa, B, sb, rows, torch.float32), A, sa, B, sb, rows)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(140, 4800, 256), (257, 4000, 512), (60, 11259, 1120), (170, 3508, 5776), (37, 1545, 6736)])
def test_matmul_in_tiles_of_96_weight_rows(m, n, k, dtype):
    """Sizes at which 96 weight rows a tile fill the GPU best, whole and with the blocks split; odd row counts."""
    A, sa, B, sb = _operands(m, n, k, 1, m + n, S.dev())
    _check_matmul(_matmul(A, sa, B, sb, 1, dtype), A, sa, B, sb, 1)


def test_matmul_is_deterministic_and_keeps_to_its_rows():
    """Two calls give equal bits; Y's memory behind the last row, and the operands, stay as they were."""
    m, n, k = 19, 1000, 4096
    A, sa, B, sb = _operands(m, n, k, 1, 5, S.dev())
    buf = torch.full((m + 3, n), 7.0, device=S.dev())
    before = [t.clone() for t in (A.view(torch.uint8), sa, B.view(torch.uint8), sb)]
    st = torch.zeros(2, dtype=torch.int32, device=S.dev())
    ws = torch.empty(max(256, g.gptq_fp8_matmul_workspace_size(m, n, k)), dtype=torch.uint8, device=S.dev())
    g.gptq_fp8_matmul(A, sa, B, sb, 1, buf[:m], st, ws)
    assert (buf[m:] == 7.0).all()
    assert torch.equal(buf[:m], _matmul(A, sa, B, sb, 1, torch.float32))
    for t, b in zip((A.view(torch.uint8), sa, B.view(torch.uint8), sb), before):
        assert torch.equal(t, b)


@pytest.mark.parametrize("m,n,k", [(9, 1, 16), (300, 3, 48), (130, 200, 16), (300, 40, 128), (4, 2, 16)])
def test_small_matrices(m, n, k):
    """Boxes larger than the matrices they are cut from, in every form."""
    A, sa, B, sb = _operands(m, n, k, 1, m + n, S.dev())
    _check_matmul(_matmul(A, sa, B, sb, 1, torch.float32), A, sa, B, sb, 1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [(5, 64, 256), (40, 64, 256), (300, 256, 256), (300, 512, 4224)])
def test_outputs_and_scales_on_any_alignment(m, n, k, dtype):
    """Y, the scales and the status as views that start one value into their memory."""
    dev = S.dev()
    A, sa, B, sb = _operands(m, n, k, 1, 3, dev)

    def shifted(t):
        buf = torch.zeros(t.numel() + 1, dtype=t.dtype, device=dev)
        buf[1:] = t.reshape(-1)
        return buf[1:].view(t.shape)

    Y = shifted(torch.full((m, n), float("nan"), dtype=dtype, device=dev))
    sa, sb, st = shifted(sa), shifted(sb), shifted(torch.zeros(2, dtype=torch.int32, device=dev))
    ws = torch.empty(max(256, g.gptq_fp8_matmul_workspace_size(m, n, k)), dtype=torch.uint8, device=dev)
    g.gptq_fp8_matmul(A, sa, B, sb, 1, Y, st, ws)
    assert g.gptq_read_status(st)[0] == g.GPTQ_OK
    _check_matmul(Y, A, sa, B, sb, 1)


def test_nan_stays_in_its_row_and_column():
    m, n, k = 40, 200, 512
    A, sa, B, sb = _operands(m, n, k, 1, 9, S.dev())
    A.view(torch.uint8)[7, 300] = 0x7F
    sb[11, 2] = float("inf")
    Y = _matmul(A, sa, B, sb, 1, torch.float32)
    assert torch.isnan(Y[7]).all()
    assert not torch.isfinite(Y[:, 11]).any()
    keep = torch.isfinite(Y)
    keep[7], keep[:, 11] = True, True
    assert keep.all()
    r = [i for i in range(m) if i != 7]
    c = [j for j in range(n) if j != 11]
    _check_matmul(Y[r][:, c], A[r].contiguous(), sa[r], B[c].contiguous(), sb[c], 1)


def test_no_rows_is_no_work():
    dev = S.dev()
    e = lambda *s, dt=torch.float32: torch.empty(*s, device=dev, dtype=dt)
    n0 = g.gptq_kernel_launches()
    g.gptq_fp8_quantize(e(0, 64), e(0, 64).to(F8), e(0, 1), 1)
    g.gptq_fp8_matmul(e(0, 64).to(F8), e(0, 1), e(8, 64).to(F8), e(8, 1), 1, e(0, 8),
                      torch.zeros(2, dtype=torch.int32, device=dev), e(64))
    assert g.gptq_kernel_launches() == n0


def test_on_another_stream_and_in_a_graph():
    """The chain quantize -> product on a side stream, then captured and replayed on new inputs."""
    dev = S.dev()
    m, n, k = 50, 768, 1024
    gen = torch.Generator().manual_seed(3)
    xs = [torch.randn(m, k, generator=gen).to(torch.bfloat16).to(dev) for _ in range(3)]
    _, _, B, sb = _operands(m, n, k, 128, 4, dev)
    x, Q, sc = xs[0].clone(), torch.zeros(m, k, device=dev).to(F8), torch.zeros(m, k // 128, device=dev)
    Y = torch.zeros(m, n, device=dev)
    st = torch.zeros(2, dtype=torch.int32, device=dev)
    ws = torch.empty(max(256, g.gptq_fp8_matmul_workspace_size(m, n, k)), dtype=torch.uint8, device=dev)

    def chain(s):
        g.gptq_fp8_quantize(x, Q, sc, 1, s)
        g.gptq_fp8_matmul(Q, sc, B, sb, 128, Y, st, ws, s)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    chain(side)
    side.synchronize()
    _check_matmul(Y, Q, sc, B, sb, 128)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(None)
    for t in xs[1:] + xs[:1]:
        x.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        q_ref, _ = _ref_quantize(t, 1)
        np.testing.assert_array_equal(Q.double().cpu().numpy(), q_ref)
        _check_matmul(Y, Q, sc, B, sb, 128)
    assert g.gptq_read_status(st)[0] == g.GPTQ_OK
