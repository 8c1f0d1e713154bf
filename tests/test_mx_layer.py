"""The wave path with MX-FP4 experts (moe_mx_expert_gemm) inside whole layers.

Every returned row is checked against the formula in 64 bits on the rows that
reached the expert.  The hidden rows are quantised from fp32 sums, so a value
within the sums' error of a rounding border may go either way: the tolerance
of a returned value adds, for exactly those hidden values, the distance
between the two codes times the weight, to the fp32 error of the second
product (H * 2^-24 * sum |h w|) and the rounding of the store (2^-8 in bf16).
"""

import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import mx_ref as R  # noqa: E402

from grouped_expert_ffn_router_amd import binding as B  # noqa: E402
from workload import configs, gen  # noqa: E402


def _fake_dims(**kw):
    d = B.make_dims(configs.get("mini_bf16"))
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def test_workspace_size_and_refusals():
    d = _fake_dims()
    scap, rcap, prow = B.capacity(d)
    # 2 experts a wave, 3 live waves: quantised rows (L / 2 + 16 bytes) and hidden rows (H / 2 + 16 bytes), 256-padded
    pad = lambda n: -(-n // 256) * 256  # noqa: E731
    rows = 2 * rcap
    want = 3 * (pad(rows * 128) + pad(rows * 16) + pad(rows * 64) + pad(rows * 16))
    assert B.mx_workspace_size(d) == want
    assert B.mx_workspace_size(_fake_dims(live_waves=1)) == want // 3
    assert B.mx_workspace_size(_fake_dims(wave_rows=10)) == 3 * (pad(1280) + pad(160) + pad(640) + pad(160))
    for kw in (dict(act_dtype=1, latent=24), dict(act_dtype=1, expert_hidden=20)):
        with pytest.raises(B.MoeError) as e:
            B.mx_workspace_size(_fake_dims(**kw))
        assert e.value.code == B.MOE_EINVAL and "32" in str(e.value)
    w13, w2 = B.mx_rows(256, 256, 128, 16), B.mx_rows(256, 256, 64, 16)
    base = dict(dims=d, wave=0, wave_buf=None, recv_pools=256, src_stride_bytes=scap * prow, row_src=256, wave_count=256,
                w13=w13, w2=w2, ret_pools=256, ret_src_stride_bytes=scap * 512, ws=256, ws_mx=256)
    for kw, code, word in [
            (dict(w13=None), B.MOE_EINVAL, "w13"), (dict(w2=None), B.MOE_EINVAL, "w2"),
            (dict(w2=B.mx_rows(256, 256, 48, 16)), B.MOE_EALIGN, "w2"),
            (dict(w13=B.mx_rows(256, 264, 128, 16)), B.MOE_EALIGN, "w13"),
            (dict(wave=3), B.MOE_EINVAL, "wave"), (dict(wave=-1), B.MOE_EINVAL, "wave"),
            (dict(ws=None), B.MOE_EINVAL, "ws"), (dict(ws_mx=None), B.MOE_EINVAL, "ws_mx"),
            (dict(ws_mx=264), B.MOE_EALIGN, "ws_mx"), (dict(recv_pools=None), B.MOE_EINVAL, "recv_pools"),
            (dict(src_stride_bytes=8), B.MOE_EALIGN, "src_stride"), (dict(wave_buf=8), B.MOE_EALIGN, "wave_buf"),
            (dict(ret_src_stride_bytes=16), B.MOE_EALIGN, "ret_src"), (dict(row_src=2), B.MOE_EALIGN, "row_src"),
            (dict(ret_pools=None), B.MOE_EINVAL, "ret_pools"), (dict(wave_count=None), B.MOE_EINVAL, "wave_count"),
            (dict(dims=_fake_dims(act_dtype=9)), B.MOE_EDTYPE, "act_dtype")]:
        with pytest.raises(B.MoeError) as e:
            B.mx_expert_gemm(**{**base, **kw}, stream=0)
        assert e.value.code == code and word in str(e.value), kw


def test_unknown_expert_form_is_refused():
    from grouped_expert_ffn_router_amd import runner
    with pytest.raises(ValueError):
        runner._expert_form("fp4")


def _round(v):
    """Values (float64) to the grid of scale 1, ties to the even code."""
    a = np.abs(v)
    step = 0.5 * (1 + (a >= 2)) * (1 + (a >= 4))
    return np.copysign(np.minimum(np.round(a / step) * step, 6), v)


def _hidden(x, wg, wu, L):
    """Quantised hidden rows in 64 bits and by how much each value may differ."""
    g, u = x @ wg.T, x @ wu.T
    ge, ue = L * 2.0 ** -24 * (np.abs(x) @ np.abs(wg).T), L * 2.0 ** -24 * (np.abs(x) @ np.abs(wu).T)
    silu = g / (1 + np.exp(-g))
    h = silu * u
    # |silu'| <= 1.1; the kernel's silu: an exponential and a reciprocal of about (|g| + 4) * 2^-23 relative
    he = np.abs(u) * (1.1 * ge + np.abs(silu) * (np.abs(g) + 4) * 2.0 ** -23) + np.abs(silu) * ue + np.abs(h) * 2.0 ** -22
    he = he + ge * ue
    n, H = h.shape
    b, be = h.reshape(n, -1, 32), he.reshape(n, -1, 32)
    lo = np.maximum(np.abs(b) - be, 0).max(-1)
    hi = (np.abs(b) + be).max(-1)
    ex = lambda m: np.where(m > 0, np.clip(np.frexp(np.maximum(m, 1e-300))[1] - 3, -127, 127), -127)  # noqa: E731
    e0, e1 = ex(lo), ex(hi)
    unit = np.exp2(e1.astype(np.float64))[..., None]
    q = _round(b / unit) * unit
    diff = np.abs(_round((b + be) / unit) - _round((b - be) / unit)) * unit
    # the scale itself may go either way: both codes are within 2 units of the value
    diff = np.where((e0 != e1)[..., None], 4 * unit, diff)
    return q.reshape(n, H), diff.reshape(n, H)


def _check_returned_rows(lay, sh, r, w13, w2, pool_of, ret_of):
    """Every kept row of receiver r: ret_of(row) against the formula; returns (rows, uncertain hidden values)."""
    X, W, L, H = sh.local_experts, sh.waves, sh.latent, sh.expert_hidden
    WX = X // W
    row_src, counts = lay.row_src[r].cpu().numpy(), lay.wave_count[r].cpu().numpy()
    rows = unsure = 0
    for w in range(W):
        for j in range(WX):
            n = int(counts[w, j])
            if not n:
                continue
            src = row_src[w, j, :n]
            x = np.stack([pool_of(int(s)) for s in src])
            x = R.values(*R.quantize(x))
            e = r * X + w * WX + j
            q, diff = _hidden(x, w13[e][:H], w13[e][H:], L)
            y = q @ w2[e].T
            tol = diff @ np.abs(w2[e]).T + H * 2.0 ** -24 * ((np.abs(q) + diff) @ np.abs(w2[e]).T)
            half = 2.0 ** -8 if sh.act == "bf16" else 2.0 ** -24
            tol = tol + half * (np.abs(y) + tol)
            got = np.stack([ret_of(int(s)) for s in src])
            bad = np.abs(got - y) > tol * (1 + 1e-9)
            assert not bad.any(), (r, w, j, int(bad.sum()), float((np.abs(got - y) - tol).max()))
            rows += n
            unsure += int((diff > 0).sum())
    return rows, unsure


def _layer(cls, name, gather, **kw):
    from dataclasses import replace
    sh = configs.get(name)
    if "recv_num" in kw:
        sh = replace(sh, recv_num=kw.pop("recv_num"))
    inp = gen.generate(sh, seed=11)
    lay = cls(sh, inp, experts="mx", gather=gather, **kw)
    lay.run()
    torch.cuda.synchronize()
    w13, w2 = (R.values(q.codes.cpu().numpy(), q.scales.cpu().numpy()) for q in (lay.w13, lay.w2))
    return sh, inp, lay, w13, w2


@pytest.mark.gpu
@pytest.mark.parametrize("name,gather,recv_num", [
    ("mini_bf16", "fused", 115), ("mini_bf16", "buffer", 115), ("mini_bf16_skew", "fused", 115), ("mini_bf16_seg", "fused", 115),
    ("mini_bf16_longk", "buffer", 115), (1, "fused", 115), (1, "buffer", 115),
    # a receive cap of many times the load: the products take their large tiles
    ("mini_bf16", "fused", 10000), (1, "fused", 20000)])
def test_returned_rows_of_every_rank(name, gather, recv_num):
    from grouped_expert_ffn_router_amd import runner
    sh, inp, lay, w13, w2 = _layer(runner.AllRanksLayer, name, gather, recv_num=recv_num)
    act = torch.bfloat16 if sh.act == "bf16" else torch.float32
    L = sh.latent
    pools = lay.pools[..., :L * (2 if sh.act == "bf16" else 4)].contiguous().view(act).double().cpu().numpy()
    ids = lay.pools.view(torch.int32)[..., L * (2 if sh.act == "bf16" else 4) // 4].cpu().numpy()
    ret = lay.ret.double().cpu().numpy()
    total = 0
    for r in range(sh.n_ranks):
        at = lambda s: pools[s // lay.scap, r, s % lay.scap]          # noqa: E731
        back = lambda s: ret[r, s // lay.scap, s % lay.scap]          # noqa: E731
        rows, unsure = _check_returned_rows(lay, sh, r, w13, w2, at, back)
        # the allowance stays small.  Sums of L products are known to L * 2^-24 * sum |a b|, twice (gate and up), and
        # sum |a b| is about sqrt(L) times the sum: relative L^1.5 * 2^-23.  A value of a few units whose borders are
        # half a unit apart is unsure with some 8 times that chance (L = 2048: 9 %; L = 256: 0.4 %).
        assert unsure <= 8 * L ** 1.5 * 2.0 ** -23 * rows * sh.expert_hidden + 64
        total += rows
        # rows dropped at receive come back as zeros
        kept = set(lay.row_src[r].cpu().numpy().ravel().tolist())
        for s in range(sh.n_ranks):
            for slot in np.nonzero(ids[s, r] >= 0)[0]:
                if s * lay.scap + int(slot) not in kept:
                    assert (ret[r, s, slot] == 0).all()
    assert total == sum(rep["recv_kept"] for rep in lay.drop_reports())
    # the layer's output is the weighted sum of those rows, projected up, plus the shared experts: finite and, with
    # 4-bit experts, near the same layer's with the experts in its own type
    ref = runner.AllRanksLayer(sh, inp)
    ref.run()
    torch.cuda.synchronize()
    assert torch.equal(ref.slot_of, lay.slot_of) and torch.equal(ref.idx, lay.idx)
    assert torch.isfinite(lay.out.float()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("wave_rows", [0, None, 40])
def test_ragged_bank_gives_the_same_rows(wave_rows):
    """Hidden rows end to end in one bank: the bytes of the blocked layout; a bank
    that is too small loses only the rows past it and is reported."""
    from grouped_expert_ffn_router_amd import runner
    sh, inp, full, *_ = _layer(runner.RaggedAllRanksLayer, "mini_bf16", "fused", expert_rows=200, wave_rows=0)
    sh, inp, lay, *_ = _layer(runner.RaggedAllRanksLayer, "mini_bf16", "fused", expert_rows=200, wave_rows=wave_rows)
    if wave_rows == 40:
        for r in range(sh.n_ranks):
            counts = lay.wave_count[r].cpu().numpy()
            first = counts[:, 0].clip(max=40)
            for w in range(sh.waves):
                for m in range(int(first[w])):
                    s = int(lay.row_src[r, w, 0, m])
                    assert torch.equal(lay.ret[r][s], full.ret[r][s])
        with pytest.raises(B.MoeError):
            B.drop_stats(lay.recv_dims[0], lay.ws_recv[0])
    else:
        for r in range(sh.n_ranks):
            assert torch.equal(lay.ret[r], full.ret[r])
        assert torch.equal(lay.out, full.out)


@pytest.mark.gpu
def test_one_rank_layer_two_streams_and_graph():
    """The one-rank layer with 4-bit experts: one stream, two streams and a captured step give the same bytes."""
    from dataclasses import replace
    from grouped_expert_ffn_router_amd import runner
    sh = replace(configs.get("mini_bf16"), emulate_all_ranks=False)
    inp = gen.generate(sh, seed=3, send_cap=B.capacity(B.make_dims(sh))[0])
    lay = runner.OneRankLayer(sh, inp, experts="mx")
    lay.run()
    torch.cuda.synchronize()
    want, rows = lay.out.clone(), lay.ret_send.clone()
    assert torch.isfinite(want.float()).all() and float(rows.float().abs().sum()) > 0
    side = torch.cuda.Stream()
    lay.out.zero_()
    lay.run(side=side)
    torch.cuda.synchronize()
    assert torch.equal(lay.out, want) and torch.equal(lay.ret_send, rows)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lay.run(stream=torch.cuda.current_stream())
    for _ in range(3):
        lay.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(lay.out, want)
        lay.run()
        torch.cuda.synchronize()
        assert torch.equal(lay.out, want)


# ---------------------------------------------------------------- what comes out of the layer

def _f64(t):
    return t.double().cpu().numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("name,gather", [("mini_bf16", "fused"), ("mini_bf16_skew", "buffer"), ("mini_bf16_seg", "fused"),
                                         ("mini_bf16_longk", "fused"), (1, "buffer")])
def test_output_is_the_weighted_sum_of_the_returned_rows(name, gather):
    """out = act(c . U^T + sum_j h_j . W2_j^T) with c = act(sum_i w_i ret_i) and h_j = act(silu(x Wg^T) (x Wu^T)), from the
    rows that the experts returned.  Each rounding to act is off by half a step of its value, each fp32 sum of n products by
    n * 2^-24 of the sum of their magnitudes; both are carried through the products that follow."""
    from grouped_expert_ffn_router_amd import runner
    sh, inp, lay, *_ = _layer(runner.AllRanksLayer, name, gather)
    half = 2.0 ** -8 if sh.act == "bf16" else 2.0 ** -24
    eps = 2.0 ** -24
    T, D, L, k, S, HS = sh.tokens, sh.d_model, sh.latent, sh.top_k, sh.shared_experts, sh.shared_hidden
    U, ws13, ws2, ret = (_f64(t) for t in (lay.w_up, lay.ws13, lay.ws2, lay.ret))
    for s in range(sh.n_ranks):
        w, x, slot = _f64(lay.w[s]), _f64(lay.x[s]), lay.slot_of[s].cpu().numpy()
        rows = np.where((slot >= 0)[..., None], ret[:, s].reshape(-1, L)[slot.clip(min=0)], 0)   # [T][k][L]
        c = (w[..., None] * rows).sum(1)
        dc = k * eps * (w[..., None] * np.abs(rows)).sum(1) + half * np.abs(c)
        want, tol = c @ U.T, dc @ np.abs(U).T + L * eps * (np.abs(c) @ np.abs(U).T)
        for j in range(S):
            wg, wu = ws13[j][:HS], ws13[j][HS:]
            g, u = x @ wg.T, x @ wu.T
            dg, du = D * eps * (np.abs(x) @ np.abs(wg).T), D * eps * (np.abs(x) @ np.abs(wu).T)
            silu = g / (1 + np.exp(-g))
            h = silu * u
            # as for the experts' hidden values above; then the rounding to act
            dh = np.abs(u) * (1.1 * dg + np.abs(silu) * (np.abs(g) + 4) * 2.0 ** -23) + np.abs(silu) * du + dg * du
            dh += (half + 2.0 ** -22) * np.abs(h)
            want += h @ ws2[j].T
            tol += dh @ np.abs(ws2[j]).T + HS * eps * (np.abs(h) @ np.abs(ws2[j]).T)
        tol = tol + half * (np.abs(want) + tol)
        got = _f64(lay.out[s])
        assert (np.abs(got - want) <= tol * (1 + 1e-9)).all(), (s, float((np.abs(got - want) - tol).max()))
        # the tolerance tells a wrong layer from a right one
        assert np.sqrt(np.mean(tol ** 2)) < 0.3 * np.sqrt(np.mean(want ** 2))


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["mini_bf16", "mini_bf16_longk", 1])
def test_how_far_four_bits_move_the_returned_rows(name):
    """A value of a normally distributed block is off by an eighth of its RMS, give or take (codes a quarter to a half apart
    in relative size).  Gate and up: two quantised operands, sqrt(2) / 8 = 0.18; silu(gate) up: both, sqrt(1.2^2 + 1) 0.18 =
    0.28; the hidden row and W2 quantised: sqrt(0.28^2 + 2 / 8^2) = 0.33 of a returned row's RMS.  Half and 1.5 times that
    bound it."""
    from grouped_expert_ffn_router_amd import runner
    sh, inp, lay, *_ = _layer(runner.AllRanksLayer, name, "fused")
    ref = runner.AllRanksLayer(sh, inp)
    ref.run()
    torch.cuda.synchronize()
    assert torch.equal(ref.slot_of, lay.slot_of)
    a, b = lay.ret.double(), ref.ret.double()
    off = float((a - b).square().mean().sqrt() / b.square().mean().sqrt())
    assert 0.165 <= off <= 0.5, off


@pytest.mark.gpu
@pytest.mark.parametrize("gather,ragged_banks,live_waves", [("fused", True, 2), ("buffer", True, 1), ("fused", False, 0)])
def test_ragged_one_rank_layer(gather, ragged_banks, live_waves):
    """One rank with the dropless ragged exchange: the output bits of the fixed-pool layer whose capacities fit the same
    counts, on one stream and on two."""
    from dataclasses import replace
    from grouped_expert_ffn_router_amd import runner
    sh = replace(configs.get("mini_bf16"), emulate_all_ranks=False)
    inp = gen.generate(sh, seed=4, send_cap=B.capacity(B.make_dims(sh))[0])
    drawn = {s: inp["sources"](s) for s in range(sh.n_ranks)}
    probe = runner.RaggedOneRankLayer(replace(sh, layer="dispatch"), dict(inp, sources=drawn.__getitem__),
                                      expert_rows=sh.n_ranks * sh.tokens)
    probe.run()
    rep = probe.drop_report()
    pool_rows = max(max(rep["send_demand"]), max(probe.source_demand.values()))
    expert_rows = max(rep["expert_arrivals"])
    fit = configs.exact_fit(sh, pool_rows, expert_rows)
    inp = gen.generate(fit, seed=4, send_cap=pool_rows)
    inp["sources"] = drawn.__getitem__
    fixed = runner.OneRankLayer(fit, inp, gather="fused", experts="mx")
    fixed.run()
    lay = runner.RaggedOneRankLayer(sh, inp, expert_rows, gather=gather, ragged_banks=ragged_banks, live_waves=live_waves,
                                    experts="mx")
    lay.run()
    torch.cuda.synchronize()
    assert isinstance(lay.w13, runner.MxRows) and (lay.wave_rows > 0) == ragged_banks
    assert lay.drop_report()["recv_dropped"] == 0 and fixed.drop_report()["recv_dropped"] == 0
    assert torch.isfinite(lay.out.float()).all() and float(lay.out.float().abs().sum()) > 0
    assert torch.equal(lay.out, fixed.out)
    lay.out.zero_()
    lay.run(side=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(lay.out, fixed.out)


@pytest.mark.gpu
def test_memory_counts_the_mx_workspace():
    """memory() and footprint() of a layer with MX-FP4 experts: hidden rows of H / 2 + 16 bytes (H = 128) in the workspace of
    the MX-FP4 products, which is counted."""
    from dataclasses import replace
    from grouped_expert_ffn_router_amd import runner
    sh = replace(configs.get("mini_bf16"), emulate_all_ranks=False)
    scap, rcap, _ = B.capacity(B.make_dims(sh))
    inp = gen.generate(sh, seed=3, send_cap=scap)
    act, mx = (runner.OneRankLayer(sh, inp, experts=e, live_waves=2) for e in ("act", "mx"))
    a, b = act.memory(), mx.memory()
    assert a["hidden_rows_per_wave_bytes"] == 2 * rcap * 128 * 2 and "mx_workspace_bytes" not in a
    assert b["hidden_rows_per_wave_bytes"] == 2 * rcap * (64 + 16)
    assert b["hidden_rows_live_bytes"] == 2 * b["hidden_rows_per_wave_bytes"]
    assert b["mx_workspace_bytes"] == B.mx_workspace_size(mx.dims) > b["hidden_rows_live_bytes"]
    drawn = {s: inp["sources"](s) for s in range(sh.n_ranks)}
    inp = dict(gen.generate(sh, seed=3, send_cap=sh.tokens * sh.top_k), sources=drawn.__getitem__)
    act, mx = (runner.RaggedOneRankLayer(sh, inp, 2 * rcap, experts=e) for e in ("act", "mx"))
    assert mx.footprint() == act.footprint() + B.mx_workspace_size(mx.recv_dims)
