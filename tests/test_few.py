"""The few-token layer (moe_few_tokens, runner.FewTokenLayer) against the layer's
formula in 64 bits, and its refusals.

Tolerances.  bf16: the store is half a step off (2^-8 of the value); inside,
activations are two bf16 parts (2^-17 relative) and sums are fp32, so each of
the three products adds errors of random sign of about 2^-17 of its RMS:
2^-12 of the output's RMS is thirty times that, for the largest of all
elements.  fp32: the framework's 1e-5 of the RMS (fp32 sums), plus 2^-24.
Routing: fp32 logits are off by at most D * 2^-24 * sum |x w| (and 2^-24 for
the bias), so the i-th pick's exact logit is within twice that of the i-th
largest exact logit; where no two logits are that close, the picks are the
exact ones."""

import numpy as np
import pytest
import torch

from grouped_expert_ffn_router_amd import binding as B


def _dims(**kw):
    d = dict(tokens=4, d_model=128, latent=64, n_experts=12, top_k=2, n_ranks=1, waves=1, expert_hidden=64,
             shared_experts=1, shared_hidden=64, my_rank=0, act_dtype=0, send_num=1, send_den=1, recv_num=1, recv_den=1)
    d.update(kw)
    return B.Dims(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=65), B.MOE_EINVAL), (dict(tokens=-1), B.MOE_EINVAL), (dict(act_dtype=3), B.MOE_EDTYPE),
    (dict(d_model=0), B.MOE_EINVAL), (dict(d_model=96), B.MOE_EINVAL), (dict(latent=32), B.MOE_EINVAL),
    (dict(expert_hidden=100), B.MOE_EINVAL), (dict(shared_hidden=8), B.MOE_EINVAL), (dict(n_experts=2049), B.MOE_EINVAL),
    (dict(n_ranks=5), B.MOE_EINVAL), (dict(n_ranks=0), B.MOE_EINVAL), (dict(my_rank=1), B.MOE_EINVAL),
    (dict(top_k=13), B.MOE_EINVAL), (dict(top_k=33, n_experts=64), B.MOE_EINVAL), (dict(top_k=0), B.MOE_EINVAL),
    (dict(d_model=1 << 25), B.MOE_EINVAL), (dict(shared_experts=1 << 20), B.MOE_EINVAL),
    (dict(shared_experts=-1), B.MOE_EINVAL), (dict(expert_hidden=1 << 25), B.MOE_EINVAL),
    (dict(tokens=64, top_k=32, n_experts=2048, expert_hidden=1 << 24, act_dtype=1), B.MOE_EINVAL),
    (dict(tokens=64, top_k=32, n_experts=2048, expert_hidden=1 << 19, act_dtype=1), B.MOE_EINVAL),  # threads of a launch
    (dict(shared_experts=1 << 21, shared_hidden=4, act_dtype=1), B.MOE_EINVAL),
])
def test_bad_dims_are_refused(kw, code):
    with pytest.raises(B.MoeError) as e:
        B.few_workspace_size(_dims(**kw))
    assert e.value.code == code and B.last_error()


def test_dims_that_only_this_call_takes():
    assert B.few_workspace_size(_dims(n_experts=384, top_k=8)) > 0                # any number of local experts
    assert B.few_workspace_size(_dims(waves=7, send_den=0)) > 0                  # fields it does not look at
    assert B.few_workspace_size(_dims(act_dtype=1, d_model=33, latent=7, expert_hidden=5, shared_hidden=3)) > 0
    for kw in ({}, dict(latent=2048, expert_hidden=1536, n_experts=384, top_k=8), dict(latent=64, expert_hidden=6144)):
        sizes = [B.few_workspace_size(_dims(tokens=t, **kw)) for t in range(65)]
        assert sizes == sorted(sizes)                                            # one for 64 tokens serves fewer


@pytest.mark.parametrize("kw,code,word", [
    (dict(x=None), B.MOE_EINVAL, "x"), (dict(x=264), B.MOE_EALIGN, "x"), (dict(w_router=None), B.MOE_EINVAL, "w_router"),
    (dict(w_down=8), B.MOE_EALIGN, "w_down"), (dict(w13=None), B.MOE_EINVAL, "w13"), (dict(w2=None), B.MOE_EINVAL, "w2"),
    (dict(w_up=None), B.MOE_EINVAL, "w_up"), (dict(ws13=None), B.MOE_EINVAL, "ws13"), (dict(ws2=None), B.MOE_EINVAL, "ws2"),
    (dict(topk_idx=None), B.MOE_EINVAL, "topk_idx"), (dict(topk_w=258), B.MOE_EALIGN, "topk_w"),
    (dict(out=None), B.MOE_EINVAL, "out"), (dict(ws=None), B.MOE_EINVAL, "ws"), (dict(ws=264), B.MOE_EALIGN, "ws"),
    (dict(bias=2), B.MOE_EALIGN, "bias"), (dict(bias_row_tokens=-1), B.MOE_EINVAL, "bias_row_tokens"),
    (dict(w13_scales=256), B.MOE_EINVAL, "together"), (dict(w2_scales=256), B.MOE_EINVAL, "together"),
    (dict(w13_scales=8, w2_scales=256), B.MOE_EALIGN, "w13_scales"),
    (dict(w13_scales=256, w2_scales=256, dims=_dims(act_dtype=1)), B.MOE_EDTYPE, "bf16"),
])
def test_bad_arguments_are_refused(kw, code, word):
    base = dict(dims=_dims(), x=256, w_router=256, w_down=256, bias=None, bias_row_tokens=0, w13=256, w13_scales=None,
                w2=256, w2_scales=None, w_up=256, ws13=256, ws2=256, topk_idx=256, topk_w=256, out=256, ws=256)
    with pytest.raises(B.MoeError) as e:
        B.few_tokens(**{**base, **kw}, stream=0)
    assert e.value.code == code and word in str(e.value)


def test_no_tokens_need_no_pointers():
    B.few_tokens(_dims(tokens=0), *([None] * 4), 0, *([None] * 11), stream=0)


def test_layer_checks_its_weights():
    from grouped_expert_ffn_router_amd import runner
    z = lambda *s: torch.zeros(s)  # noqa: E731
    good = dict(w_router=z(6, 40), w_down=z(16, 40), w13=z(6, 20, 16), w2=z(6, 16, 10), w_up=z(40, 16), top_k=2)
    lay = runner.FewTokenLayer(**good)
    assert (lay.dims.n_experts, lay.dims.latent, lay.dims.expert_hidden, lay.dims.shared_experts) == (6, 16, 10, 0)
    for kw, exc in [(dict(w_down=z(16, 41)), ValueError), (dict(w13=z(5, 20, 16)), ValueError), (dict(w2=z(6, 16, 11)), ValueError),
                    (dict(w_up=z(16, 40)), ValueError), (dict(w_up=z(16, 40).t()), ValueError), (dict(w13=z(6, 20, 16).bfloat16()), TypeError),
                    (dict(ws13=z(1, 8, 40), ws2=z(1, 40, 5)), ValueError), (dict(bias=z(5)), ValueError),
                    (dict(bias=z(2, 6)), ValueError), (dict(bias=z(6).double()), ValueError), (dict(top_k=7), B.MoeError),
                    (dict(n_ranks=4), ValueError), (dict(w_router=z(6, 40).half()), TypeError),
                    (dict(w2=runner.MxRows(torch.zeros(6, 16, 16, dtype=torch.uint8), torch.zeros(6, 16, 16, dtype=torch.uint8), 32)), TypeError)]:
        with pytest.raises(exc):
            runner.FewTokenLayer(**{**good, **kw})
    for x in (z(3, 41), z(3, 40).bfloat16(), z(40), z(40, 3).t(), z(65, 40)):
        with pytest.raises((ValueError, IndexError)):
            lay(x)


# ---------------------------------------------------------------- GPU

def _weights(seed, E, D, L, H, S, HS, act, mx=False, spread=1.0):
    from grouped_expert_ffn_router_amd import runner
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16 if act == "bf16" else torch.float32
    n = lambda fan, *s: (torch.randn(s, generator=g, device="cuda") * spread / fan ** 0.5).to(dt)  # noqa: E731
    w = dict(w_router=n(D, E, D), w_down=n(D, L, D), w13=n(L, E, 2 * H, L), w2=n(H, E, L, H), w_up=n(L, D, L),
             ws13=n(D, S, 2 * HS, D), ws2=n(HS, S, D, HS))
    if mx:
        w["w13"], w["w2"] = runner.mx_quantize(w["w13"]), runner.mx_quantize(w["w2"])
    return w, g, dt


def _f64(t):
    from grouped_expert_ffn_router_amd import runner
    return (runner.mx_dequantize(t, torch.float32) if isinstance(t, runner.MxRows) else t).double().cpu()


def _formula(w, x, k, bias=None, first=0, picks=None):
    """(out, idx, topk_w) in float64 on the CPU; only the experts from `first` on that w13 holds contribute.  `picks`
    [T, k]: the library's choice, checked against the exact logits and then used."""
    x = x.double().cpu()
    bias = torch.zeros(()) if bias is None else bias.double().cpu()
    wr = _f64(w["w_router"])
    logits = x @ wr.T + bias
    s = torch.sort(logits, dim=1, descending=True, stable=True)
    idx = s.indices[:, :k]
    if picks is not None:
        picks = picks.cpu().long()
        assert all(len(set(r)) == k for r in picks.tolist())
        off = x.shape[1] * 2.0 ** -24 * (x.abs() @ wr.abs().T).amax(1, keepdim=True) + 2.0 ** -23 * (logits.abs() + bias.abs()).amax(1, keepdim=True)
        assert bool(((logits.gather(1, picks) - s.values[:, :k]).abs() <= 2 * off).all())
        clear = ((s.values[:, :-1] - s.values[:, 1:]) > 2 * off).all(1)
        assert torch.equal(picks[clear], idx[clear])
        idx = picks
    tw = torch.softmax(logits.gather(1, idx), 1)
    z = x @ _f64(w["w_down"]).T
    w13, w2 = _f64(w["w13"]), _f64(w["w2"])
    c = torch.zeros_like(z)
    for t in range(x.shape[0]):
        for i in range(k):
            e = int(idx[t, i]) - first
            if 0 <= e < w13.shape[0]:
                g, u = (w13[e] @ z[t]).chunk(2)
                c[t] += tw[t, i] * (w2[e] @ (torch.nn.functional.silu(g) * u))
    out = c @ _f64(w["w_up"]).T
    for j in range(w["ws13"].shape[0]):
        g, u = (x @ _f64(w["ws13"][j]).T).chunk(2, 1)
        out += (torch.nn.functional.silu(g) * u) @ _f64(w["ws2"][j]).T
    return out, idx, tw


def _check(got, w, x, k, act, bias=None, first=0):
    out, idx, tw = (t.cpu() for t in got)
    want, _, rw = _formula(w, x, k, bias, first, picks=idx)
    assert float((tw.double() - rw).abs().max()) <= 1e-5
    rms = float(want.square().mean().sqrt())
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -12 * rms if act == "bf16" else 2.0 ** -24 * want.abs() + 1e-5 * rms
    d = (out.double() - want).abs()
    assert bool((d <= tol).all()), (float((d - tol).max()), rms)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,D,L,H,S,HS,act,mx", [
    (1, 4, 1, 64, 64, 64, 0, 64, "bf16", False),
    (1, 48, 4, 512, 256, 128, 2, 128, "bf16", False),
    (2, 384, 8, 192, 128, 64, 1, 64, "bf16", False),
    (16, 8, 8, 320, 192, 192, 2, 64, "bf16", False),      # every expert of every token
    (17, 12, 3, 576, 64, 640, 1, 192, "bf16", False),
    (33, 6, 2, 128, 320, 576, 3, 64, "bf16", False),
    (64, 4, 2, 256, 128, 1088, 1, 128, "bf16", False),
    (64, 256, 32, 128, 64, 64, 1, 64, "bf16", False),     # 2048 pairs
    (3, 2048, 32, 128, 64, 64, 0, 64, "bf16", False),     # the most experts
    (9, 700, 5, 64, 64, 64, 2, 64, "bf16", True),
    (2, 513, 4, 24, 16, 12, 1, 8, "f32", False),
    (1, 2, 2, 64, 4096, 64, 1, 64, "bf16", False),        # one share of the down product; wide latent
    (12, 96, 6, 64, 64, 2048, 1, 64, "bf16", False),      # a wave to itself for 16 hidden units
    (1, 16, 4, 128, 64, 64, 1, 64, "bf16", True),
    (3, 8, 2, 2368, 2176, 64, 3, 2112, "bf16", False),    # whole rounds of deep steps, then groups and single steps
    (13, 8, 2, 4160, 2048, 64, 2, 192, "bf16", True),
    (12, 96, 6, 64, 320, 1024, 0, 64, "bf16", False),     # waves apart, each workgroup from another group of K on
    (20, 64, 6, 704, 448, 1088, 2, 448, "bf16", False),
    (5, 24, 2, 256, 192, 320, 2, 128, "bf16", True),
    (16, 4, 2, 128, 576, 704, 0, 64, "bf16", True),
    (40, 4, 2, 192, 128, 1152, 1, 64, "bf16", True),
    (1, 3, 1, 7, 5, 3, 1, 2, "f32", False),
    (7, 36, 3, 1000, 520, 300, 1, 260, "f32", False),
    (3, 11, 2, 37, 29, 41, 2, 13, "f32", False),          # no size a multiple of 4
    (31, 12, 3, 40, 24, 20, 2, 12, "f32", False),
    (64, 5, 5, 130, 34, 530, 0, 4, "f32", False),
])
def test_against_the_formula(T, E, k, D, L, H, S, HS, act, mx):
    from grouped_expert_ffn_router_amd import runner
    w, g, dt = _weights(T * 1000 + E, E, D, L, H, S, HS, act, mx)
    x = torch.randn((T, D), generator=g, device="cuda").to(dt)
    bias = torch.randn((E,), generator=g, device="cuda")
    lay = runner.FewTokenLayer(**w, bias=bias, top_k=k)
    lay.ws.fill_(0xFF)                                      # nothing in the workspace needs to start at zero
    got = lay(x)
    _check(got, w, x, k, act, bias)
    again = lay(x)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    # fewer tokens through the same layer
    n = max(1, T // 2)
    part = lay(x[:n].contiguous())
    _check(part, w, x[:n], k, act, bias)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [15, 20, 47, 64])
@pytest.mark.parametrize("act,mx", [("bf16", False), ("bf16", True), ("f32", False)])
def test_all_tokens_to_the_same_experts(T, act, mx):
    """A bias that sends every token to experts 5 and 2; a bias row for each 10 tokens changes the second."""
    from grouped_expert_ffn_router_amd import runner
    E, D, L, H = 12, 128, 64, 576
    w, g, dt = _weights(T, E, D, L, H, 1, 64, act, mx)
    x = torch.randn((T, D), generator=g, device="cuda").to(dt)
    nb = -(-T // 10)
    bias = torch.zeros((nb, E), device="cuda")
    bias[:, 5] = 50
    bias[torch.arange(nb), torch.arange(nb) % 3 + 7] = 25
    lay = runner.FewTokenLayer(**w, bias=bias, bias_row_tokens=10, top_k=2)
    got = lay(x)
    rows = bias[torch.arange(T, device="cuda") // 10]
    _check(got, w, x, 2, act, rows)
    assert (got[1][:, 0] == 5).all() and sorted(set(got[1][:, 1].tolist())) == sorted({7 + i % 3 for i in range(nb)})


@pytest.mark.gpu
def test_equal_logits_go_to_the_lower_expert():
    from grouped_expert_ffn_router_amd import runner
    w, g, dt = _weights(1, 16, 64, 64, 64, 0, 64, "bf16")
    w["w_router"] = torch.zeros_like(w["w_router"])
    bias = torch.tensor([0., 3, 1, 3, -0., 1, 3, 0] * 2, device="cuda")
    x = torch.randn((3, 64), generator=g, device="cuda").to(dt)
    out, idx, tw = runner.FewTokenLayer(**w, bias=bias, top_k=12)(x)
    assert idx.tolist() == [[1, 3, 6, 9, 11, 14, 2, 5, 10, 13, 0, 4]] * 3
    assert torch.isfinite(out.float()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("act,mx", [("bf16", False), ("bf16", True), ("f32", False)])
def test_ranks_shares_add_up(act, mx):
    """Four ranks with three experts each, one of them with the shared experts; a rank whose experts nobody chose."""
    from grouped_expert_ffn_router_amd import runner
    E, R, k, T, D = 12, 4, 2, 9, 192
    w, g, dt = _weights(5, E, D, 64, 128, 2, 64, act, mx)
    x = torch.randn((T, D), generator=g, device="cuda").to(dt)
    bias = torch.zeros(E, device="cuda")
    bias[9:] = -100                                          # rank 3 serves nobody
    total = torch.zeros((T, D), dtype=torch.float64)
    for r in range(R):
        mine = {**w, "w13": w["w13"][3 * r:3 * r + 3], "w2": w["w2"][3 * r:3 * r + 3]}
        if r != 1:
            mine["ws13"] = mine["ws2"] = None
        got = runner.FewTokenLayer(**mine, bias=bias, top_k=k, n_ranks=R, rank=r)(x)
        plain = mine if r == 1 else {**mine, "ws13": w["ws13"][:0], "ws2": w["ws2"][:0]}
        ref = _formula(plain, x, k, bias, first=3 * r)
        if r == 3:
            assert (got[0] == 0).all()
        else:
            _check(got, plain, x, k, act, bias, first=3 * r)
        total += ref[0]
    assert float((total - _formula(w, x, k, bias)[0]).abs().max()) < 1e-9


@pytest.mark.gpu
def test_a_token_with_nan_leaves_the_others_alone():
    from grouped_expert_ffn_router_amd import runner
    for mx in (False, True):
        w, g, dt = _weights(8, 12, 128, 64, 64, 1, 64, "bf16", mx)
        x = torch.randn((6, 128), generator=g, device="cuda").to(dt)
        lay = runner.FewTokenLayer(**w, top_k=3)
        want = lay(x)[0]
        x[2, 5] = float("nan")
        x[4, 7] = float("inf")
        got, idx, _ = lay(x)
        keep = [0, 1, 3, 5]
        # the chosen experts differ, and with them the order of some fp32 sums: a step of the output at most
        d = (got[keep].float() - want[keep].float()).abs()
        assert bool((d <= 2.0 ** -7 * want[keep].float().abs() + 2.0 ** -12).all())
        assert torch.isnan(got[2].float()).all() and not torch.isfinite(got[4].float()).all()
        assert int(idx.min()) >= 0 and int(idx.max()) < 12 and all(len(set(r)) == 3 for r in idx.tolist())


@pytest.mark.gpu
def test_agrees_with_the_layer_of_the_same_weights():
    """The batch layer's own entry points (route, pack, receive, expert FFNs, combine) on one rank with nothing dropped:
    same routing, outputs within its rounding points (the framework's bar of 2e-2 RMS)."""
    from dataclasses import replace
    from grouped_expert_ffn_router_amd import runner
    from workload import configs, gen
    sh = replace(configs.get("mini_bf16"), tokens=48, n_ranks=1, emulate_all_ranks=True, send_num=200, recv_num=2000)
    inp = gen.generate(sh, seed=2)
    ref = runner.AllRanksLayer(sh, inp)
    ref.run()
    torch.cuda.synchronize()
    assert sum(r["recv_dropped"] + r["send_dropped"] for r in ref.drop_reports()) == 0
    lay = runner.FewTokenLayer(ref.w_router, ref.w_down, ref.w13, ref.w2, ref.w_up, ref.ws13, ref.ws2, top_k=sh.top_k)
    out, idx, tw = lay(ref.x[0].contiguous())
    assert torch.equal(idx, ref.idx[0]) and float((tw - ref.w[0]).abs().max()) < 1e-5
    a, b = out.double(), ref.out[0].double()
    rms = float(b.square().mean().sqrt())
    assert float(((a - b).abs() - 2.0 ** -7 * b.abs()).max()) <= 2e-2 * rms


@pytest.mark.gpu
@pytest.mark.parametrize("act,mx", [("bf16", False), ("bf16", True), ("f32", False)])
def test_two_streams_graphs_and_reuse(act, mx):
    """Two layers on two streams at once, and captured graphs replayed between eager calls, give each call's own bits."""
    from grouped_expert_ffn_router_amd import runner
    w, g, dt = _weights(21, 24, 512, 256, 192, 2, 128, act, mx)
    xs = [torch.randn((T, 512), generator=g, device="cuda").to(dt) for T in (1, 33)]
    lays = [runner.FewTokenLayer(**w, top_k=4) for _ in xs]
    want = [tuple(t.clone() for t in lay(x)) for lay, x in zip(lays, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [None, None]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = lays[i](xs[i])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = lays[0](xs[0])
    for _ in range(3):
        for t in held:
            t.zero_()
        graph.replay()
        mid = lays[0](xs[0])
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(held, want[0])) and all(torch.equal(u, v) for u, v in zip(mid, want[0]))


@pytest.mark.gpu
def test_writes_stay_inside_the_outputs_and_the_workspace():
    """The C entry on buffers with guard bytes, workspace of exactly the asked size."""
    for act, mx, T, dims in (("bf16", False, 3, (12, 128, 64, 64, 1, 64, 2)), ("bf16", True, 20, (12, 128, 64, 576, 1, 64, 2)),
                             ("f32", False, 5, (7, 37, 29, 41, 2, 13, 3))):
        E, D, L, H, S, HS, k = dims
        w, g, dt = _weights(3, E, D, L, H, S, HS, act, mx)
        x = torch.randn((T, D), generator=g, device="cuda").to(dt)
        d = _dims(tokens=T, d_model=D, latent=L, n_experts=E, top_k=k, expert_hidden=H, shared_experts=S, shared_hidden=HS,
                  act_dtype=0 if act == "bf16" else 1)
        n = B.few_workspace_size(d)
        ws = torch.full((n + 4096,), 0x3C, dtype=torch.uint8, device="cuda")
        out = torch.full((T * D + 64,), 5.0, dtype=dt, device="cuda")
        idx = torch.full((T * k + 16,), -5, dtype=torch.int32, device="cuda")
        tw = torch.full((T * k + 16,), -5.0, device="cuda")
        c = lambda t: t.codes if mx else t          # noqa: E731
        s = lambda t: t.scales if mx else None      # noqa: E731
        B.few_tokens(d, x, w["w_router"], w["w_down"], None, 0, c(w["w13"]), s(w["w13"]), c(w["w2"]), s(w["w2"]), w["w_up"],
                     w["ws13"], w["ws2"], idx, tw, out, ws)
        torch.cuda.synchronize()
        assert (ws[n:] == 0x3C).all() and (out[T * D:] == 5).all() and (idx[T * k:] == -5).all() and (tw[T * k:] == -5).all()
        _check((out[:T * D].view(T, D), idx[:T * k].view(T, k), tw[:T * k].view(T, k)), w, x, k, act)


@pytest.mark.gpu
@pytest.mark.parametrize("L,H", [(64, 128), (128, 64), (192, 64), (320, 192), (128, 128)])
def test_infinities_in_the_last_blocks_of_a_row(L, H):
    """MX-FP4 rows whose width is 64 beyond a multiple of 128: lanes past the row's end must not meet its values, since
    their 0 * inf would be NaN.  All experts' weights are 1, so an infinite latent value makes every sum +inf."""
    from grouped_expert_ffn_router_amd import runner
    one = lambda *s: torch.ones(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    D = 64
    for at in (0, L - 64, L - 1):
        w_down = one(L, D) / 64
        w_down[at] = 3e38                              # 64 * 3e38 passes fp32
        lay = runner.FewTokenLayer(torch.zeros_like(one(2, D)), w_down, runner.mx_quantize(one(2, 2 * H, L)),
                                   runner.mx_quantize(one(2, L, H)), one(D, L), top_k=1)
        x = one(3, D)
        x[1] = 0                                       # a token of zeros beside the infinite ones
        out = lay(x)[0]
        assert (out[0] == float("inf")).all() and (out[2] == float("inf")).all() and (out[1] == 0).all()


# ---------------------------------------------------------------- calls at once

def _cpu_layer(monkeypatch, call, stream, **kw):
    """A layer on CPU tensors whose library call is `call` and whose current stream is stream()."""
    import contextlib
    from grouped_expert_ffn_router_amd import runner
    z = lambda *s: torch.zeros(s)  # noqa: E731
    monkeypatch.setattr(runner, "_on", lambda t: (stream(), contextlib.nullcontext()))
    monkeypatch.setattr(B, "few_tokens", call)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    good = dict(w_router=z(6, 40), w_down=z(16, 40), w13=z(6, 20, 16), w2=z(6, 16, 10), w_up=z(40, 16), top_k=2)
    return runner.FewTokenLayer(**{**good, **kw})


def test_calls_on_two_streams_share_no_workspace(monkeypatch):
    seen = []
    now = [7]
    lay = _cpu_layer(monkeypatch, lambda *a: seen.append(a[16:18]), lambda: now[0])
    for now[0] in (7, 8):
        lay(torch.zeros(3, 40))
    (a, sa), (b, sb) = seen
    n = B.few_workspace_size(lay.dims)
    assert (sa, sb) == (7, 8) and a.numel() >= n and b.numel() >= n
    assert a.data_ptr() + a.numel() <= b.data_ptr() or b.data_ptr() + b.numel() <= a.data_ptr()


def test_calls_of_two_threads_keep_their_own_batch_size(monkeypatch):
    """The library call releases the interpreter: while one thread is in it, another thread's call begins."""
    import threading
    inside, other_done = threading.Event(), threading.Event()
    read = []

    def call(dims, x, *rest):
        if dims.tokens == 3:
            inside.set()
            assert other_done.wait(20)
            read.append(dims.tokens)
        else:
            other_done.set()

    lay = _cpu_layer(monkeypatch, call, lambda: 7)
    t = threading.Thread(target=lambda: lay(torch.zeros(3, 40)))
    t.start()
    assert inside.wait(20)
    lay(torch.zeros(5, 40))
    t.join(20)
    assert read == [3]


@pytest.mark.parametrize("mx", [False, True])
def test_weights_are_read_where_they_are(monkeypatch, mx):
    """Memory put in a weight's place is what the next call reads, and is checked first: addresses kept from the
    construction would point into freed memory."""
    from grouped_expert_ffn_router_amd import runner
    seen = []
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    rows = lambda *s: runner.MxRows(torch.zeros(s[:-1] + (s[-1] // 2,), dtype=torch.uint8),  # noqa: E731
                                    torch.zeros(s[:-1] + (16,), dtype=torch.uint8), s[-1]) if mx else z(*s)
    kw = dict(w_router=z(6, 64), w_down=z(128, 64), w13=rows(6, 128, 128), w2=rows(6, 128, 64), w_up=z(64, 128),
              ws13=z(2, 128, 64), ws2=z(2, 64, 64), bias=torch.zeros(6))
    lay = _cpu_layer(monkeypatch, lambda *a: seen.append(a), lambda: 7, **kw)
    at = dict(w_router=2, w_down=3, bias=4, w13=6, w13_scales=7, w2=8, w2_scales=9, w_up=10, ws13=11, ws2=12)
    names = [n for n in at if mx or not n.endswith("_scales")]

    def tensor(n):
        t = kw[n.replace("_scales", "")]
        return (t.scales if n.endswith("_scales") else t.codes) if isinstance(t, runner.MxRows) else t

    for n in names:
        tensor(n).data = torch.zeros_like(tensor(n))
        lay(z(3, 64))
        for m in names:
            assert seen[-1][at[m]] == tensor(m).data_ptr(), (n, m)
    lay.w_up = kw["w_up"] = z(64, 128)
    lay(z(3, 64))
    assert seen[-1][at["w_up"]] == lay.w_up.data_ptr()
    n = len(seen)
    for name in names:
        old = tensor(name).data
        tensor(name).data = torch.zeros(tuple(old.shape[:-1]) + (old.shape[-1] + 1,), dtype=old.dtype)
        with pytest.raises(ValueError):
            lay(z(3, 64))
        tensor(name).data = old
    lay.w_router = torch.zeros(6, 64)
    with pytest.raises((ValueError, TypeError)):
        lay(torch.zeros(3, 64))
    assert len(seen) == n


def test_rows_follow_their_tensors():
    """MxRows hands on the tensors' addresses and strides as they are, not as they were at the first call."""
    from grouped_expert_ffn_router_amd import runner
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    q = runner.MxRows(u8(3, 32), u8(3, 16), 64)
    assert (q.arg.codes, q.arg.scales) == (q.codes.data_ptr(), q.scales.data_ptr())
    q.codes.data = u8(5, 48)[:3, :32]
    q.scales.data = u8(3, 32)
    assert (q.arg.codes, q.arg.scales) == (q.codes.data_ptr(), q.scales.data_ptr())
    assert (q.arg.code_stride_bytes, q.arg.scale_stride_bytes) == (48, 32)
    for codes, scales in ((u8(3, 33), u8(3, 16)), (u8(4, 32), u8(3, 16)), (u8(3, 32), u8(3, 8))):
        q.codes, q.scales = codes, scales
        with pytest.raises(ValueError):
            q.arg


@pytest.mark.gpu
@pytest.mark.parametrize("act,mx", [("bf16", False), ("bf16", True), ("f32", False)])
def test_one_layer_on_two_streams_in_two_graphs_and_from_threads(act, mx):
    """One layer object: calls on two streams at once, two graphs captured from it replayed at once beside an eager call,
    and two threads on one stream give each call's own bits."""
    import threading
    from grouped_expert_ffn_router_amd import runner
    w, g, dt = _weights(22, 24, 512, 256, 192, 2, 128, act, mx)
    xs = [torch.randn((T, 512), generator=g, device="cuda").to(dt) for T in (1, 33)]
    lay = runner.FewTokenLayer(**w, top_k=4)
    want = [tuple(t.clone() for t in lay(x)) for x in xs]
    torch.cuda.synchronize()
    same = lambda a, b: all(torch.equal(u, v) for u, v in zip(a, b))  # noqa: E731
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(lay(xs[i]))
    torch.cuda.synchronize()
    assert all(same(want[i], one) for i in range(2) for one in got[i])
    graphs, held = [], []
    for i, s in enumerate(streams):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=s):
            held.append(lay(xs[i]))
    for _ in range(4):
        for h in held:
            for t in h:
                t.zero_()
        torch.cuda.synchronize()
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                graphs[i].replay()
        mid = lay(xs[1])
        torch.cuda.synchronize()
        assert all(same(want[i], held[i]) for i in range(2)) and same(want[1], mid)
    # a layer made on a side stream and captured on that stream
    with torch.cuda.stream(streams[0]):
        side = runner.FewTokenLayer(**w, top_k=4)
        first = side(xs[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        inside = side(xs[0])
    for _ in range(3):
        graph.replay()
        with torch.cuda.stream(streams[0]):
            mid = side(xs[1])
        torch.cuda.synchronize()
        assert same(inside, want[0]) and same(first, want[0]) and same(mid, want[1])
    outs = [[], []]

    def work(i):
        for _ in range(100):
            outs[i].append(lay(xs[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert [len(o) for o in outs] == [100, 100]
    assert all(same(want[i], one) for i in range(2) for one in outs[i])


# ---------------------------------------------------------------- weights that do not go together

def test_shared_experts_need_both_weights():
    """One of ws13 and ws2 alone, or of another number of experts, is refused and not taken as no shared experts."""
    from grouped_expert_ffn_router_amd import runner
    z = lambda *s: torch.zeros(s)  # noqa: E731
    good = dict(w_router=z(6, 40), w_down=z(16, 40), w13=z(6, 20, 16), w2=z(6, 16, 10), w_up=z(40, 16), top_k=2)
    assert runner.FewTokenLayer(**good, ws13=z(2, 8, 40), ws2=z(2, 40, 4)).dims.shared_experts == 2
    assert runner.FewTokenLayer(**good, ws13=z(0, 8, 40), ws2=z(0, 40, 4)).dims.shared_experts == 0
    for ws13, ws2 in ((None, z(2, 40, 4)), (z(2, 8, 40), None), (z(0, 8, 40), z(2, 40, 4)), (z(2, 8, 40), z(0, 40, 4)),
                      (z(2, 8, 40), z(1, 40, 4))):
        with pytest.raises(ValueError):
            runner.FewTokenLayer(**good, ws13=ws13, ws2=ws2)


def test_mx_experts_need_a_bf16_layer():
    """Refused when the layer is made, not at its first call."""
    from grouped_expert_ffn_router_amd import runner
    rows = lambda *s: runner.MxRows(torch.zeros(s[:-1] + (s[-1] // 2,), dtype=torch.uint8),  # noqa: E731
                                    torch.zeros(s[:-1] + (16,), dtype=torch.uint8), s[-1])
    for dt in (torch.bfloat16, torch.float32):
        z = lambda *s: torch.zeros(s, dtype=dt)  # noqa: E731, B023
        kw = dict(w_router=z(6, 64), w_down=z(64, 64), w13=rows(6, 128, 64), w2=rows(6, 64, 64), w_up=z(64, 64))
        if dt == torch.bfloat16:
            assert runner.FewTokenLayer(**kw).dims.expert_hidden == 64
        else:
            with pytest.raises(TypeError):
                runner.FewTokenLayer(**kw)


@pytest.mark.gpu
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
def test_values_between_the_largest_of_bf16_and_of_fp32(sign, mx):
    """A latent value of 1.9970 * 2^127 rounds to an infinity in bf16, but not as two bf16 parts.  D = 64 weights of it:
    the largest bf16 value and 1.25 * 2^119.  The experts' weights of 2^-124 bring it back: gate = up = sign * 15.98."""
    from grouped_expert_ffn_router_amd import runner
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    D = L = H = 64
    w_down = z(L, D)
    w_down[0, 0] = sign * torch.finfo(torch.bfloat16).max
    w_down[0, 1] = sign * 1.25 * 2.0 ** 119
    w13 = z(1, 2 * H, L)
    w13[:, :, 0] = 2.0 ** -124
    w2 = z(1, L, H) + 2.0 ** -10
    if mx:
        w13, w2 = runner.mx_quantize(w13), runner.mx_quantize(w2)
    w = dict(w_router=z(1, D), w_down=w_down, w13=w13, w2=w2, w_up=z(D, L) + 1, ws13=z(0, 2, D), ws2=z(0, D, 1))
    x = z(3, D) + 1
    got = runner.FewTokenLayer(**w, top_k=1)(x)
    assert torch.isfinite(got[0].float()).all()
    _check(got, w, x, 1, "bf16")


# ---------------------------------------------------------------- scale bytes of the experts' blocks

@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 7, 40])
@pytest.mark.parametrize("L,H,E", [(192, 320, 6), (128, 1024, 64)])     # the second: a wave to itself for 16 units (T > 7)
def test_zero_and_nan_scales_of_the_experts(T, L, H, E):
    """Scale byte 255 in one block of w13 and of w2 gives NaN to the tokens that choose those experts and to no other;
    blocks of scale byte 0 (2^-127, some with codes 0) count as what they stand for."""
    from grouped_expert_ffn_router_amd import runner
    w, g, dt = _weights(31 + T, E, 256, L, H, 1, 64, "bf16", mx=True)
    for q in (w["w13"], w["w2"]):
        q.scales[3, 5, 1] = 0                                                # random codes times 2^-127
        q.scales[4, :, 0] = 0
        q.codes[4, :, :16] = 0
    x = torch.randn((T, 256), generator=g, device="cuda").to(dt)
    bias = torch.zeros((T, E), device="cuda")
    for t in range(T):                                                       # token t: experts t % 6 and (t + 2) % 6
        bias[t, [t % 6, (t + 2) % 6]] = 50
    kw = dict(bias=bias, bias_row_tokens=1, top_k=2)
    _check(runner.FewTokenLayer(**w, **kw)(x), w, x, 2, "bf16", bias)
    w["w13"].scales[1, 2 * H - 1, L // 32 - 1] = 255                         # the last block of the last up row
    w["w2"].scales[2, 17, 0] = 255
    out, idx, tw = runner.FewTokenLayer(**w, **kw)(x)
    hit = ((idx == 1) | (idx == 2)).any(1)
    assert torch.isnan(out[hit].float()).all() and torch.isfinite(out[~hit].float()).all()
    if bool((~hit).any()):
        _check((out[~hit], idx[~hit], tw[~hit]), w, x[~hit], 2, "bf16", bias[~hit])


@pytest.mark.gpu
@pytest.mark.parametrize("byte", [0, 1, 2, 127, 251, 252, 253, 254])
def test_every_kind_of_scale_times_a_latent_value_that_balances_it(byte):
    """One expert whose gate and up blocks all have one scale byte, and latent values of about its inverse; codes up to the
    largest whose value bf16 holds (6, but 3 with byte 253 and 1.5 with 254: of a magnitude above that a product is not
    finite)."""
    from grouped_expert_ffn_router_amd import runner
    g = torch.Generator().manual_seed(byte)
    D = L = H = 64
    top = {253: 6, 254: 4}.get(byte, 8)                                      # magnitudes' codes below this
    mag = lambda *s: torch.randint(0, top, s, generator=g) + 8 * torch.randint(0, 2, s, generator=g)  # noqa: E731
    codes = (mag(1, 2 * H, L // 2) | mag(1, 2 * H, L // 2) << 4).to(torch.uint8)
    scales = torch.full((1, 2 * H, 16), byte, dtype=torch.uint8)
    w2 = runner.mx_quantize((torch.randn((1, L, H), generator=g) / 8).cuda())
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    unit = 2.0 ** -max(-120, min(120, byte - 127))
    w = dict(w_router=z(1, D), w_down=(torch.eye(L) * unit).bfloat16().cuda(),
             w13=runner.MxRows(codes.cuda(), scales.cuda(), L), w2=w2, w_up=torch.eye(D).bfloat16().cuda(),
             ws13=z(0, 2, D), ws2=z(0, D, 1))
    x = torch.randint(1, 4, (5, D), generator=g).bfloat16().cuda()
    _check(runner.FewTokenLayer(**w, top_k=1)(x), w, x, 1, "bf16")


# ---------------------------------------------------------------- the forms that large layers take

def _forms(T, E, k, L, H, act, mx):
    """What the launches go by (ops/few.hip): waves that share K in the experts' gate and up products, row tiles of the
    down product, and the most tokens of an expert whose rows are staged in LDS (MX-FP4, a wave to itself)."""
    up = lambda a, b: -(-a // b)  # noqa: E731
    most = min(E, T * k)
    waves = 1 if most * up(H, 16) >= 16 * 256 else 8
    parts = up(most * up(H, 128 if act == "f32" else 256), 8)
    row_tiles = 2 if up(L, 32) * parts >= 2 * 256 else 1
    return waves, row_tiles, min(16, 32 * 1024 // ((2 * L + 8) * 2)) if mx and waves == 1 else 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,L,H,act,mx,forms", [
    (12, 96, 6, 320, 1024, "bf16", True, (1, 1, 16)),
    (16, 128, 8, 1088, 512, "bf16", True, (1, 2, 7)),     # in one launch, experts of few tokens from LDS and others not
    (20, 64, 8, 192, 1088, "bf16", True, (1, 1, 16)),
    (40, 64, 8, 512, 1024, "bf16", True, (1, 2, 15)),
    (64, 64, 8, 512, 1024, "bf16", True, (1, 2, 15)),
    (64, 16, 4, 2304, 576, "bf16", True, (8, 1, 0)),
    (33, 32, 4, 1024, 1024, "bf16", True, (8, 2, 0)),
    (64, 64, 8, 512, 1024, "bf16", False, (1, 2, 0)),     # 64 KB of LDS a workgroup in the down product
    (64, 32, 4, 1024, 1024, "bf16", False, (8, 2, 0)),
    (9, 128, 8, 576, 1024, "bf16", False, (1, 2, 0)),
    (12, 64, 6, 53, 1030, "f32", False, (1, 1, 0)),
    (12, 64, 6, 245, 1030, "f32", False, (1, 2, 0)),
    (40, 64, 3, 61, 1027, "f32", False, (1, 1, 0)),
    (20, 64, 6, 245, 1030, "f32", False, (1, 2, 0)),
    (64, 64, 2, 421, 530, "f32", False, (8, 2, 0)),
])
def test_forms_of_large_layers(T, E, k, L, H, act, mx, forms):
    """Every token has expert 1; the other picks are spread, so that experts of one token and of all T are in one launch."""
    from grouped_expert_ffn_router_amd import runner
    assert _forms(T, E, k, L, H, act, mx) == forms
    w, g, dt = _weights(T + L, E, 128, L, H, 1, 64, act, mx)
    x = torch.randn((T, 128), generator=g, device="cuda").to(dt)
    bias = torch.zeros(E, device="cuda")
    bias[1] = 50
    lay = runner.FewTokenLayer(**w, bias=bias, top_k=k)
    lay.ws.fill_(0xFF)
    got = lay(x)
    assert (got[1][:, 0] == 1).all()
    tokens = torch.bincount(got[1].flatten().long(), minlength=E)
    assert int(tokens.max()) == T and (T >= 40 or bool((tokens == 1).any()))
    _check(got, w, x, k, act, bias)
    again = lay(x)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 3, 16, 17, 40, 64])
@pytest.mark.parametrize("D,act", [(4096, "bf16"), (4160, "bf16"), (4096, "f32"), (4099, "f32")])
def test_row_tiles_of_the_last_product(D, act, T):
    """Output widths whose tiles of 16 rows are 256 and more: a tile a workgroup, or two with more than two tokens.  The
    width 4099 ends inside the first tile of a pair."""
    from grouped_expert_ffn_router_amd import runner
    w, g, dt = _weights(T, 6, D, 64, 64, 2, 64, act)
    x = torch.randn((T, D), generator=g, device="cuda").to(dt)
    lay = runner.FewTokenLayer(**w, top_k=2)
    guard = torch.full((T * D + 64,), 5.0, dtype=dt, device="cuda")
    got = lay(x, out=guard[:T * D].view(T, D))
    _check(got, w, x, 2, act)
    assert (guard[T * D:] == 5).all()


# ---------------------------------------------------------------- copies

@pytest.mark.parametrize("mx", [False, True])
def test_a_copied_layer_serves_its_own_weights(monkeypatch, mx):
    """copy.deepcopy and pickle give a layer of its own: its weights' addresses, its workspace, its lock."""
    import copy
    import pickle
    from grouped_expert_ffn_router_amd import runner
    seen = []
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    rows = lambda *s: runner.MxRows(torch.zeros(s[:-1] + (s[-1] // 2,), dtype=torch.uint8),  # noqa: E731
                                    torch.zeros(s[:-1] + (16,), dtype=torch.uint8), s[-1]) if mx else z(*s)
    lay = _cpu_layer(monkeypatch, lambda *a: seen.append(a), lambda: 7, w_router=z(6, 64), w_down=z(128, 64),
                     w13=rows(6, 128, 128), w2=rows(6, 128, 64), w_up=z(64, 128))
    lay(z(3, 64))
    if mx:
        assert lay.w13.arg.codes == lay.w13.codes.data_ptr()
    for twin in (copy.deepcopy(lay), pickle.loads(pickle.dumps(lay))):
        twin(z(3, 64))
        tensor = lambda t: t.codes if mx else t  # noqa: E731
        for i, name in ((2, "w_router"), (3, "w_down"), (6, "w13"), (8, "w2"), (10, "w_up")):
            mine, other = (tensor(getattr(x, name)) if name in ("w13", "w2") else getattr(x, name) for x in (twin, lay))
            assert seen[-1][i] == mine.data_ptr() != other.data_ptr()
        assert twin.ws.data_ptr() != lay.ws.data_ptr() and twin.ws.numel() == lay.ws.numel()
        assert twin.dims.latent == 128 and twin.dims is not lay.dims and twin._ws_lock is not lay._ws_lock
        if mx:
            assert twin.w13.arg.codes == twin.w13.codes.data_ptr()


# ---------------------------------------------------------------- other tensors at the same address

def test_attributes_set_to_other_views_are_checked(monkeypatch):
    """A view that begins where the old tensor did has the old address; its shape and strides count all the same."""
    from grouped_expert_ffn_router_amd import runner
    seen = []
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    lay = _cpu_layer(monkeypatch, lambda *a: seen.append(a), lambda: 7, w_router=z(6, 64), w_down=z(128, 64),
                     w13=z(6, 128, 128), w2=z(6, 128, 64), w_up=z(64, 128))
    lay(z(3, 64))
    for name in ("w_router", "w_down", "w13", "w2", "w_up"):
        old = getattr(lay, name)
        for new in (old[:3], old[..., :32], old.transpose(-1, -2)):
            setattr(lay, name, new)
            with pytest.raises(ValueError):
                lay(z(3, 64))
        setattr(lay, name, old)
        lay(z(3, 64))
    assert len(seen) == 6
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    q = runner.MxRows(u8(4, 6, 32), u8(4, 6, 16), 64)
    assert q.arg.code_stride_bytes == 32
    q.codes, q.scales = q.codes[:, :5], q.scales[:, :5]
    with pytest.raises(ValueError):      # rows 0..4, 6..10, ..: not evenly spaced
        q.arg
    q.codes, q.scales = u8(4, 6, 32)[:, ::2], u8(4, 6, 16)[:, ::2]
    assert (q.arg.code_stride_bytes, q.arg.scale_stride_bytes) == (64, 32)


@pytest.mark.gpu
@pytest.mark.parametrize("act,mx", [("bf16", False), ("bf16", True), ("f32", False)])
def test_output_in_the_place_of_the_input(act, mx):
    """out may be x: the last product, which writes it, reads no token."""
    from grouped_expert_ffn_router_amd import runner
    w, g, dt = _weights(41, 12, 256, 128, 192, 2, 64, act, mx)
    lay = runner.FewTokenLayer(**w, top_k=3)
    for T in (1, 20):
        x = torch.randn((T, 256), generator=g, device="cuda").to(dt)
        want = [t.clone() for t in lay(x)]
        got = lay(x, out=x)
        assert got[0] is x and all(torch.equal(a, b) for a, b in zip(got, want))
