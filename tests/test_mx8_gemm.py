"""The product of MX-FP8 rows with MX-FP4 rows on the GPU against 64-bit sums."""

import pytest
import torch

import block_ref as R
from grouped_expert_ffn_router_amd import binding as B, block, runner

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
FOUR = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def _decode4(codes, scales):
    c = codes.cpu().long()
    v = FOUR[torch.stack([c & 15, c >> 4], -1)].reshape(*codes.shape[:-1], -1, 32)
    s = scales.cpu()[..., :v.shape[-2]].double()
    return (v * torch.where(s == 255, torch.nan, torch.exp2(s - 127))[..., None]).flatten(-2)


def _operands(seed, G, M, N, K, a_scales=(120, 132), b_scales=(120, 132)):
    """Random codes (no NaN among them) and scale bytes, what pads a row's scales at random too."""
    gen = torch.Generator().manual_seed(seed)
    pad = (K // 32 + 15) // 16 * 16
    a = torch.randint(0, 256, (G, M, K), generator=gen, dtype=torch.uint8)
    a[(a & 127) == 127] = 0x7e
    b = torch.randint(0, 256, (G, N, K // 2), generator=gen, dtype=torch.uint8)
    sa, sb = (torch.randint(0, 256, (G, n, pad), generator=gen, dtype=torch.uint8) for n in (M, N))
    for s, (lo, hi) in ((sa, a_scales), (sb, b_scales)):
        s[..., :K // 32] = torch.randint(lo, hi, s[..., :K // 32].shape, generator=gen, dtype=torch.uint8)
    return block.Mx8Rows(a.to(DEV), sa.to(DEV), K), runner.MxRows(b.to(DEV), sb.to(DEV), K)


def _check(out, a, b, rows):
    """Against 64-bit sums.  fp32 sums of K products: a step of their size each.  Beside them the matrix unit cuts off, of eight
    products, what is 2^-13 of the largest and less: of a block's 32 at most 32 2^-13 times the largest product that may be
    there, 448 * 6 of the blocks' scales, or 7.5 * 6 (the part of the codes below 8) with an fp32 output."""
    K = a.cols
    top = (448 if out.dtype == torch.bfloat16 else 7.5) * 6
    for g in range(out.shape[0]):
        n = rows[g]
        if n == 0:
            continue
        va, vb = R.decode8(a.codes[g, :n], a.scales[g, :n]), _decode4(b.codes[g], b.scales[g])
        ua, ub = (torch.exp2(q.scales[g].cpu()[:, :K // 32].double() - 127) for q in (a, b))
        want = va @ vb.T
        tol = (va.abs() @ vb.abs().T) * (K / 8 + 16) * U + (ua[:n] @ ub.T) * (32 * 2.0 ** -13 * top)
        tol = tol + want.abs() * torch.finfo(out.dtype).eps / 2 + 2.0 ** -126
        err = (R.bits64(out[g, :n]) - want).abs()
        assert (err <= tol).all(), (g, float((err / tol).max()))


SHAPES = [(1, 1, 1, 32), (1, 1, 16, 64), (1, 3, 17, 96), (1, 16, 40, 128), (2, 17, 33, 160), (1, 31, 130, 480), (1, 33, 64, 512),
          (1, 64, 256, 544), (3, 48, 20, 1056), (1, 5, 16, 2080), (1, 64, 48, 4128), (1, 2, 16, 8224), (1, 20, 16, 16416),
          (1, 65, 64, 32), (1, 100, 130, 64), (1, 128, 128, 96), (1, 129, 127, 128), (1, 200, 300, 160), (1, 257, 255, 256),
          (1, 300, 513, 288), (2, 130, 260, 384), (1, 500, 512, 512), (1, 260, 264, 544), (1, 70, 600, 1120), (1, 140, 140, 2080),
          (3, 300, 200, 640)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G,M,N,K", SHAPES)
def test_product(G, M, N, K, dtype):
    a, b = _operands(G * 1000 + M + N + K, G, M, N, K)
    _check(block.mx8_gemm(a, b, dtype=dtype), a, b, [M] * G)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(2300, 2200, 160), (5000, 3000, 416), (4096, 4100, 96)])
def test_product_of_many_tiles(M, N, K, dtype):
    """More tiles than the card has places for: tiles of 256 x 256 with bf16 outputs."""
    a, b = _operands(M + N, 1, M, N, K)
    _check(block.mx8_gemm(a, b, dtype=dtype), a, b, [M])


def _tile(G, M, N):
    """The tile that a bf16 output of more than 64 rows gets: 256 unless tiles of 128, two at a time on a CU and 0.65 of the time,
    are faster."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert M > 64
    rounds = lambda t, places: -(-(G * -(-M // t) * -(-N // t)) // places)  # noqa: E731
    return 128 if rounds(128, 2 * cus) * 0.65 < rounds(256, cus) else 256


@pytest.mark.parametrize("M,N,K", [(2900, 2881, 544), (2830, 3001, 736), (2817, 2945, 832), (2901, 2890, 1024), (2830, 3001, 1120),
                                   (2945, 2823, 1248), (2900, 2897, 2080), (2999, 2817, 4128)])
def test_long_rows_by_tiles_of_256(M, N, K):
    """5 to 33 steps of 128 values: every buffer again and again, scales of the next four steps loaded in between, last steps of 32,
    64, 96 and 128 values."""
    assert _tile(1, M, N) == 256
    a, b = _operands(M + K, 1, M, N, K)
    _check(block.mx8_gemm(a, b), a, b, [M])


def test_groups_by_tiles_of_256():
    """With counts, columns and rows that end inside a tile, and rows of the output at any alignment."""
    G, M, N, K, counts = 4, 1501, 1499, 1120, [1501, 0, 37, 1333]
    assert _tile(G, M, N) == 256
    a, b = _operands(8, G, M, N, K)
    wide = torch.full((G, M, N + 4), 7.0, dtype=torch.bfloat16, device=DEV)
    out = wide[..., 3:3 + N]
    block.mx8_gemm(a, b, counts=torch.tensor(counts, dtype=torch.int32, device=DEV), out=out)
    _check(out, a, b, counts)
    assert (wide[..., :3] == 7).all() and (wide[..., 3 + N:] == 7).all()
    for g in range(G):
        assert (out[g, counts[g]:] == 7).all()


@pytest.mark.parametrize("M,N,K", [(16, 4099, 2080), (64, 4099, 6144), (130, 700, 512), (500, 512, 16416), (1000, 513, 4128),
                                   (2900, 2881, 544), (2900, 2900, 6144)])
def test_bf16_outputs_are_off_by_their_rounding(M, N, K):
    """Over the whole output, on normal operands: the mean square of the rounding to bf16 alone, within 2 % (it is the mean over
    65,000 outputs and more), and the 1e-4 of an output's RMS that the matrix unit cuts off, three times over."""
    gen = torch.Generator().manual_seed(K)
    a = block.mx8_quantize(torch.randn((M, K), generator=gen).bfloat16().to(DEV))
    b = runner.mx_quantize((torch.randn((N, K), generator=gen) / 64).to(DEV))
    want = R.decode8(a.codes, a.scales) @ _decode4(b.codes, b.scales).T
    got = R.bits64(block.mx8_gemm(a, b))
    own = (want.to(torch.bfloat16).double() - want).pow(2).mean()
    assert (got - want).pow(2).mean() <= 1.02 * own + (3e-4) ** 2 * want.pow(2).mean()


@pytest.mark.parametrize("M,N,K", [(16, 40, 2080), (64, 48, 4128), (300, 200, 1120), (500, 512, 16416), (2900, 2881, 2080), (2817, 2945, 1248)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_last_block_that_outweighs_the_others(M, N, K, dtype):
    """Its scale 2^20 times theirs: what is missing or wrong there is not lost in the sum over the others."""
    a, b = _operands(K, 1, M, N, K, a_scales=(110, 112), b_scales=(126, 128))
    a.scales[:, :, K // 32 - 1] += 20
    _check(block.mx8_gemm(a, b, dtype=dtype), a, b, [M])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K,counts", [(50, 40, 96, [50, 0, 17, -4, 99]), (300, 130, 288, [300, 0, 1, 129, 400, 256]),
                                          (1200, 700, 160, [1200, 3, 0, 700])])
def test_rows_behind_the_counts_are_left_alone(M, N, K, counts, dtype):
    G = len(counts)
    a, b = _operands(M, G, M, N, K)
    out = torch.full((G, M, N), 7.0, dtype=dtype, device=DEV)
    block.mx8_gemm(a, b, counts=torch.tensor(counts, dtype=torch.int32, device=DEV), out=out)
    rows = [min(max(c, 0), M) for c in counts]
    _check(out, a, b, rows)
    for g in range(G):
        assert (out[g, rows[g]:] == 7).all()
    fresh = block.mx8_gemm(a, b, counts=torch.tensor(counts, dtype=torch.int32, device=DEV), dtype=dtype)
    for g in range(G):
        assert (fresh[g, rows[g]:] == 0).all() and torch.equal(fresh[g, :rows[g]], out[g, :rows[g]])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G,M,N,K", [(63, 300, 140, 32), (64, 70, 20, 64), (65, 260, 20, 32), (128, 90, 300, 32), (129, 140, 20, 32),
                                     (1000, 70, 20, 32), (4096, 66, 17, 32), (4096, 5, 17, 32),
                                     # up to 64 rows by tiles
                                     (8, 40, 2100, 640), (30, 64, 1500, 1056), (100, 33, 700, 512), (64, 16, 513, 544)])
def test_many_groups(G, M, N, K, dtype):
    """Tiles are dealt out 64 groups at a time: some groups empty, most, all but one, all, none."""
    a, b = _operands(G + M, G, M, N, K)
    gen = torch.Generator().manual_seed(G)
    some = torch.randint(-M // 2, M + 9, (G,), generator=gen, dtype=torch.int32)
    few = torch.where(torch.rand((G,), generator=gen) < 0.02, some, 0).int()
    first, last = torch.zeros(G, dtype=torch.int32), torch.zeros(G, dtype=torch.int32)
    first[0], last[-1] = M, 1
    whole = block.mx8_gemm(a, b, dtype=dtype)
    _check(whole, a, b, [M] * G)
    for counts in (some, few, first, last, torch.zeros(G, dtype=torch.int32)):
        out = torch.full((G, M, N), 7.0, dtype=dtype, device=DEV)
        block.mx8_gemm(a, b, counts=counts.to(DEV), out=out)
        there = torch.arange(M)[None, :, None] < counts[:, None, None]
        assert torch.equal(out, torch.where(there.to(DEV), whole, torch.full_like(out, 7.0)))


@pytest.mark.parametrize("M", [9, 130])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_extreme_and_nan_scales_and_codes(M, dtype):
    """Scales of 2^-127 .. 2^127 that balance, a NaN scale, a NaN code and one in the last chunk."""
    a, b = _operands(3, 1, M, 40, 288, a_scales=(0, 1), b_scales=(254, 255))
    out = block.mx8_gemm(a, b, dtype=dtype)
    _check(out, a, b, [M])
    a.scales[0, 4, 2] = 255
    a.codes[0, 5, 7] = 0x7f
    a.codes[0, 6, 287] = 0xff
    b.scales[0, 11, 8] = 255
    nan = block.mx8_gemm(a, b, dtype=dtype)[0].isnan()
    want = torch.zeros_like(nan)
    want[4:7], want[:, 11] = True, True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("M", [7, 300])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_outputs_and_operands(M, dtype):
    a, b = _operands(M, 1, M, 90, 320)
    want = block.mx8_gemm(a[0], b[0], dtype=dtype)
    wide = torch.full((M, 97), 3.0, dtype=dtype, device=DEV)
    block.mx8_gemm(a[0], b[0], out=wide[:, 5:95])
    assert torch.equal(wide[:, 5:95], want) and (wide[:, :5] == 3).all() and (wide[:, 95:] == 3).all()
    codes, scales = torch.zeros((M, 352), dtype=torch.uint8, device=DEV), torch.zeros((M, 32), dtype=torch.uint8, device=DEV)
    codes[:, :320], scales[:, :16] = a.codes[0], a.scales[0]
    part = block.Mx8Rows(codes[:, :320], scales[:, :16], 320)
    assert torch.equal(block.mx8_gemm(part, b[0], dtype=dtype), want)


def test_norm_to_product():
    """A token's way into 4-bit experts: the norm's 8-bit rows against quantised weights, next to the same in 64 bits."""
    gen = torch.Generator().manual_seed(1)
    x, r = (torch.randn((200, 1024), generator=gen).bfloat16().to(DEV) for _ in range(2))
    w = (torch.randn((1024,), generator=gen) * 0.2 + 1).to(DEV)
    four = runner.mx_quantize((torch.randn((352, 1024), generator=gen) / 32).to(DEV))
    rows, _ = block.rms_norm(x, w, residual=r, form="mx8")
    out = block.mx8_gemm(rows, four, dtype=torch.float32)
    _check(out[None], rows[None], four[None], [200])
    # what 8 bits cost: each value off by 2^-4 of itself at most, 2^-5.9 on average, so an output by 2 % of its RMS
    want = R.norm(R.bits64(x), R.bits64(w), R.bits64(r))[0] @ _decode4(four.codes, four.scales).T
    off = (R.bits64(out) - want).pow(2).mean().sqrt() / want.pow(2).mean().sqrt()
    assert off < 2.0 ** -5


def test_graph_and_stream():
    a, b = _operands(5, 2, 150, 96, 256)
    c = torch.tensor([150, 70], dtype=torch.int32, device=DEV)
    want = block.mx8_gemm(a, b, counts=c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block.mx8_gemm(a, b, counts=c)
    for n in (70, 150, 3):
        c[1] = n
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, block.mx8_gemm(a, b, counts=c))
    c[1] = 70
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = block.mx8_gemm(a, b, counts=c)
    side.synchronize()
    assert torch.equal(second, want)


def test_refusals():
    a, b = _operands(1, 1, 4, 8, 64)
    with pytest.raises(TypeError):
        block.mx8_gemm(b, b)
    with pytest.raises(TypeError):
        block.mx8_gemm(a, a)
    with pytest.raises(TypeError):
        runner.mx_gemm(a, b)
    with pytest.raises(TypeError):
        runner.mx_dequantize(a)
    with pytest.raises(TypeError):
        block.mx8_dequantize(b)
    with pytest.raises(ValueError):
        block.mx8_gemm(a, b[0])
    with pytest.raises(ValueError):
        block.mx8_gemm(a, b, out=torch.empty((1, 4, 9), device=DEV))
    with pytest.raises(TypeError):
        block.mx8_gemm(a, b, dtype=torch.float16)
    with pytest.raises(ValueError):
        block.mx8_gemm(a, b, counts=torch.ones(2, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        block.mx8_gemm(a, b, counts=torch.ones(1, dtype=torch.int64, device=DEV))
    with pytest.raises(B.MoeError):   # rows that are not 16-byte aligned
        block.mx8_gemm(block.Mx8Rows(torch.zeros((1, 4, 72), dtype=torch.uint8, device=DEV)[..., 8:], a.scales, 64), b)
