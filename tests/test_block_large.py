"""The block's operators where offsets pass 32 bits, bytes and values, against the same rows on their own."""

import pytest
import torch

from grouped_expert_ffn_router_amd import block, runner

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _memory():
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 100 GB")
    yield
    torch.cuda.empty_cache()


def _say(*a):
    print(*a, flush=True)


def test_norm_and_rows():
    rows, cols = 360_000, 6144   # 2.2e9 values, 4.4 GB
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    x[:1000].normal_(generator=gen)
    x[1000:].copy_(x[:1000].repeat(359, 1))   # row r is row r % 1000
    w = torch.randn((cols,), generator=gen, device=DEV).bfloat16()
    _say("forward")
    (y, q), s = block.rms_norm(x, w, residual=x, form="both")
    (y0, q0), s0 = block.rms_norm(x[:1000], w, residual=x[:1000], form="both")
    for a, b in ((y, y0), (s, s0), (q.codes, q0.codes), (q.scales, q0.scales)):
        assert torch.equal(a[-1000:], b) and torch.equal(a[:1000], b)
    _say("8-bit rows")
    back = block.mx8_dequantize(q)
    assert torch.equal(back[-1000:], block.mx8_dequantize(q0))
    assert torch.equal(block.mx8_quantize(x).codes[-1000:], block.mx8_quantize(x[:1000]).codes)
    del q, back, y
    _say("backward")
    dx, dw = block.rms_norm_backward(x, s, w, dstream=x)
    dx0, dw0 = block.rms_norm_backward(x[:1000], s0, w, dstream=x[:1000])
    assert torch.equal(dx[-1000:], dx0) and torch.equal(dx[:1000], dx0)
    # 360 times the same rows: fp32 sums of 352 rows a part, 16 parts a thread and 64 threads, of terms of one size
    assert float((dw - 360 * dw0).norm() / (360 * dw0).norm()) < 1e-4


def test_select():
    T, E = 5_700_000, 384   # 2.2e9 logits, 8.8 GB
    gen = torch.Generator(device=DEV).manual_seed(2)
    part = torch.randn((1000, E), generator=gen, device=DEV)
    logits = part.repeat(T // 1000, 1)
    rule = block.RouterRule(8, score="sigmoid", balance=torch.randn((E,), generator=gen, device=DEV) * 0.1, groups=8, top_groups=4)
    _say("choice")
    idx, w = block.select_experts(logits, rule)
    idx0, w0 = block.select_experts(part, rule)
    assert torch.equal(idx[-1000:], idx0) and torch.equal(w[-1000:], w0)
    assert torch.equal(idx.view(-1, 1000, 8)[T // 2000], idx0)
    _say("gradient")
    d = block.select_experts_backward(w, w, idx, logits, rule)
    assert torch.equal(d[-1000:], block.select_experts_backward(w0, w0, idx0, part, rule))


def test_swiglu():
    G, M, H = 3, 180_000, 2048   # 2.2e9 gate and up values
    gen = torch.Generator(device=DEV).manual_seed(3)
    part = torch.randn((500, 2 * H), generator=gen, device=DEV).bfloat16()
    gate_up = part.repeat(G * M // 500, 1).view(G, M, 2 * H)
    counts = torch.tensor([M, 0, M], dtype=torch.int32, device=DEV)
    _say("forward")
    h, saved = block.swiglu_checkpoint(gate_up, counts)
    h0, saved0 = block.swiglu_checkpoint(part)
    assert torch.equal(h[2, -500:], h0) and torch.equal(saved.codes[2, -500:], saved0.codes) and not h[1].any()
    del gate_up
    _say("backward")
    dg, h2 = block.swiglu_backward(h, saved, counts)
    dg0, h20 = block.swiglu_backward(h0, saved0)
    assert torch.equal(dg[2, -500:], dg0) and torch.equal(h2[2, -500:], h20) and not dg[1].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product(dtype):
    M, N, K = 1 << 20, 2304, 4160   # 4.4 GB of codes, 2.4e9 outputs
    gen = torch.Generator(device=DEV).manual_seed(4)
    a0 = block.mx8_quantize(torch.randn((4096, K), generator=gen, device=DEV).bfloat16())
    a = block.Mx8Rows(a0.codes.repeat(M // 4096, 1), a0.scales.repeat(M // 4096, 1), K)
    b = runner.mx_quantize(torch.randn((N, K), generator=gen, device=DEV).bfloat16())
    _say("product", dtype)
    out, out0 = block.mx8_gemm(a, b, dtype=dtype), block.mx8_gemm(a0, b, dtype=dtype)
    assert torch.equal(out[-4096:], out0) and torch.equal(out[:4096], out0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [40, 99, 255, 513, 1023, 2047, 4099, 6143, 8203, 16381])
def test_norm_of_unaligned_rows_past_the_caches(cols, dtype):
    """More bytes than the caches hold, rows that end inside a piece: row by row as in small calls, and nothing beside them."""
    some = 1001
    rows = (150_000_000 // (cols * dtype.itemsize) + some) // some * some + 7
    gen = torch.Generator(device=DEV).manual_seed(cols)
    x, r, d = (torch.randn((some, cols), generator=gen, device=DEV).to(dtype) for _ in range(3))
    w = torch.randn((cols,), generator=gen, device=DEV).to(dtype)
    at = torch.arange(rows, device=DEV) % some
    y, s = block.rms_norm(x[at], w, residual=r[at])
    y0, s0 = block.rms_norm(x, w, residual=r)
    assert torch.equal(y, y0[at]) and torch.equal(s, s0[at])
    dx, dw = block.rms_norm_backward(d[at], s, w, dstream=r[at])
    dx0, _ = block.rms_norm_backward(d, s0, w, dstream=r)
    assert torch.equal(dx, dx0[at])
    s64, d64, times = s0.double(), d.double(), torch.bincount(at).double()[:, None]
    n = s64 * ((s64 * s64).mean(-1, keepdim=True) + 1e-6) ** -0.5
    want, size = (times * d64 * n).sum(0), (times * d64 * n).abs().sum(0)
    # a thread adds up at most rows / 256 rows of a part, 16 parts of a workgroup are joined, 16 parts a thread and 64 threads; n
    # is off by 60 steps or fewer
    assert ((dw.double() - want).abs() <= size * (rows / 256 + 16 + 16 + 64 + 60) * 2.0 ** -24).all()
