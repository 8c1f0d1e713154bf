"""The block's operators under autograd, together, and by a router rule in the layers."""

from dataclasses import replace
from functools import partial
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import block_ref as R
import test_gpu_parity as parity
from grouped_expert_ffn_router_amd import block, runner, training
from oracle import moe_oracle as O
from workload import configs, gen

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _leaf(gen, shape, scale=1.0):
    return (torch.randn(shape, generator=gen) * scale).to(DEV).requires_grad_()


def _close(got, want, rel, what):
    """In the 2-norm."""
    got, want = R.bits64(got), want.detach()
    assert got.shape == want.shape and float((got - want).norm()) <= rel * float(want.norm()), (what, float((got - want).norm() / want.norm()))


def _block64(x, res, w, wr, w13, w2, rule, counts_of=None):
    """A block in 64 bits from its definition: norm, router, every token through its experts, SwiGLU, weighted sum, residual."""
    y, s = R.norm(x, w, res)
    logits = y @ wr.T
    idx, _ = R.select(logits.detach(), rule.top_k, score=rule.score, balance=R.bits64(rule.balance), groups=rule.groups,
                      top_groups=rule.top_groups)
    wt = R.select_weights(logits, idx, torch.zeros_like(idx, dtype=torch.bool), rule.score, True, 1.0)
    out = s.clone()
    for t in range(x.shape[0]):
        for i, e in enumerate(idx[t].tolist()):
            out[t] = out[t] + wt[t, i] * (R.swiglu(y[t] @ w13[e].T) @ w2[e].T)
    return out, idx


def test_a_block_of_them_together_and_its_gradients():
    """Norm with residual -> router rule -> the experts' rows grouped by expert -> SwiGLU with its 8-bit checkpoint -> weighted sum,
    in fp32: the output to fp32 accuracy, every leaf's gradient to what the 8-bit checkpoint leaves of it."""
    g = torch.Generator().manual_seed(0)
    T, D, H, E, k = 40, 64, 96, 8, 2
    x, res = _leaf(g, (T, D)), _leaf(g, (T, D))
    w, wr = _leaf(g, (D,)), _leaf(g, (E, D), D ** -0.5)
    w13, w2 = _leaf(g, (E, 2 * H, D), D ** -0.5), _leaf(g, (E, D, H), H ** -0.5)
    rule = block.RouterRule(k, score="sigmoid", balance=(torch.randn((E,), generator=g) * 0.1).to(DEV), groups=4, top_groups=2)
    y, s = training.rms_norm(x, w, residual=res)
    idx, wt = training.select_experts(y @ wr.T, rule)
    # rows grouped by expert, padded to the longest group
    token = torch.arange(T, device=DEV).repeat_interleave(k)
    order = torch.argsort(idx.flatten(), stable=True)
    counts = torch.bincount(idx.flatten().long(), minlength=E)
    M = int(counts.max())
    place = torch.arange(T * k, device=DEV) - (torch.cumsum(counts, 0) - counts)[idx.flatten()[order].long()]
    rows = torch.zeros((E, M, D), device=DEV).index_put((idx.flatten()[order].long(), place), y[token[order]])
    h = training.swiglu(torch.bmm(rows, w13.transpose(1, 2).contiguous()), counts.int())
    back = torch.bmm(h, w2.transpose(1, 2).contiguous())[idx.flatten()[order].long(), place]
    out = s.index_add(0, token[order], back * wt.flatten()[order][:, None])
    dout = torch.randn((T, D), generator=g).to(DEV)
    (out * dout).sum().backward()

    leaves = [x, res, w, wr, w13, w2]
    ref = [R.bits64(t).requires_grad_() for t in leaves]
    want, want_idx = _block64(*ref, rule)
    assert torch.equal(idx.cpu(), want_idx)
    _close(out, want, 1e-5, "out")
    (want * R.bits64(dout)).sum().backward()
    for t, r, name in zip(leaves, ref, ("x", "res", "w", "wr", "w13", "w2")):
        # a gradient has the kept gate and the kept up value as factors, each off by 2^-4 of itself at most
        _close(t.grad, r.grad, 2.0 ** -3, name)
    _close(w2.grad, ref[5].grad, 1e-5, "w2")   # h itself is not rounded


def test_norm_without_and_with_unused_outputs():
    g = torch.Generator().manual_seed(1)
    x, w, res = _leaf(g, (6, 40)), _leaf(g, (40,)), _leaf(g, (6, 40))
    y = training.rms_norm(x, w)
    y.sum().backward()   # an expanded gradient
    dx, dw = R.norm_backward(torch.ones((6, 40), dtype=torch.float64), R.bits64(x), R.bits64(w))
    _close(x.grad, dx, 1e-5, "dx")
    _close(w.grad, dw, 1e-5, "dw")
    x.grad = w.grad = None
    _, s = training.rms_norm(x, w, residual=res)
    s.sum().backward()
    assert (x.grad == 1).all() and (res.grad == 1).all() and w.grad is None
    x.grad = res.grad = None
    y, _ = training.rms_norm(x, w, residual=res)
    y.sum().backward()
    assert torch.equal(x.grad, res.grad)
    with torch.no_grad():
        assert not training.rms_norm(x, w).requires_grad


def test_bf16_weight_gradients_have_the_weights_type():
    g = torch.Generator().manual_seed(2)
    x, w = (torch.randn(s, generator=g).bfloat16().to(DEV).requires_grad_() for s in ((300, 64), (64,)))
    training.rms_norm(x, w).float().square().sum().backward()
    assert x.grad.dtype == w.grad.dtype == torch.bfloat16


def test_selection_and_swiglu_gradients():
    g = torch.Generator().manual_seed(3)
    logits = _leaf(g, (30, 24))
    rule = block.RouterRule(3, score="softmax", renormalise=False)
    idx, w = training.select_experts(logits, rule)
    assert not idx.requires_grad
    dw = torch.randn((30, 3), generator=g).to(DEV)
    (w * dw).sum().backward()
    ref = R.bits64(logits).requires_grad_()
    (R.select_weights(ref, idx.cpu(), torch.zeros((30, 3), dtype=torch.bool), "softmax", False, 1.0) * R.bits64(dw)).sum().backward()
    _close(logits.grad, ref.grad, 1e-5, "dlogits")
    gate_up = _leaf(g, (2, 9, 128))
    h = training.swiglu(gate_up, torch.tensor([9, 4], dtype=torch.int32, device=DEV))
    assert (h[1, 4:] == 0).all()
    h.sum().backward()
    assert (gate_up.grad[1, 4:] == 0).all()
    want = R.swiglu_backward(torch.ones((9, 64), dtype=torch.float64), R.grid8(R.bits64(gate_up[0]))[0])[0]
    _close(gate_up.grad[0], want, 1e-5, "dgate_up")


# ---------------------------------------------------------------- a rule in the layers

RULE = dict(score="sigmoid", groups=4, top_groups=2, scale=1.5)


def _ruled(monkeypatch, sh):
    """The rule's balance, and the oracle choosing by the rule."""
    rng = np.random.default_rng(5)
    balance = torch.from_numpy(rng.standard_normal(sh.n_experts) * 0.1).float()

    def choose(logits, k):
        idx, w = R.select(torch.from_numpy(np.asarray(logits, np.float64)), k, balance=balance.double(), **RULE)
        return idx.numpy(), w.numpy()

    monkeypatch.setattr(O, "select_topk", choose)
    return block.RouterRule(sh.top_k, balance=balance.to(DEV), **RULE)


@pytest.mark.parametrize("name", ["mini_bf16", "mini_f32"])
def test_layer_with_a_rule(name, monkeypatch):
    """Every rank emulated, on the grid where the oracle's logits are the GPU's bit for bit."""
    sh = configs.get(name)
    rule = _ruled(monkeypatch, sh)
    inp = gen.generate(sh, seed=1, grid=True)
    ref = O.layer_all_ranks(sh, inp)
    lay = runner.AllRanksLayer(sh, inp, rule=rule)
    lay.run()
    torch.cuda.synchronize()
    for s in range(sh.n_ranks):
        d = ref["dispatch"][s]
        assert np.array_equal(lay.idx[s].cpu().numpy(), d["idx"]) and np.array_equal(lay.slot_of[s].cpu().numpy(), d["slot_of"])
        exact = ref["out"][s]["out_exact"]
        err = np.abs(lay.out[s].float().cpu().numpy().astype(np.float64) - exact).max() / np.sqrt(np.mean(exact ** 2))
        assert err <= 2e-2
    plain = runner.AllRanksLayer(sh, inp)
    plain.run()
    assert not torch.equal(plain.idx, lay.idx)


def test_layers_refuse_a_rule_of_another_k():
    sh = configs.get("mini_f32")
    with pytest.raises(ValueError):
        runner.AllRanksLayer(sh, gen.generate(sh, seed=1), rule=block.RouterRule(sh.top_k + 1))


def test_ragged_layer_with_a_rule(monkeypatch):
    sh = configs.get("mini_bf16")
    rule = _ruled(monkeypatch, sh)
    inp = gen.generate(sh, seed=1, grid=True)
    lay = runner.RaggedAllRanksLayer(sh, inp, expert_rows=sh.n_ranks * sh.tokens, rule=rule)
    lay.run()
    torch.cuda.synchronize()
    ref = O.layer_all_ranks(sh, inp)
    for s in range(sh.n_ranks):
        assert np.array_equal(lay.idx[s].cpu().numpy(), ref["dispatch"][s]["idx"])


def _drawn(sh, inp):
    """Every rank's tokens, drawn once."""
    tokens = [inp["sources"](s) for s in range(sh.n_ranks)]
    return dict(inp, sources=tokens.__getitem__)


@pytest.mark.parametrize("name", ["mini_bf16", "mini_bf16_skew"])
def test_one_rank_layer_with_a_rule(name, monkeypatch):
    """The other ranks choose by it too (at set-up): their pools, every count and row, and the output against the oracle."""
    sh = replace(configs.get(name), emulate_all_ranks=False)
    rule = _ruled(monkeypatch, sh)
    parity._one_rank_case(SimpleNamespace(OneRankLayer=partial(runner.OneRankLayer, rule=rule)), sh, 0)


def _ragged_pair(sh, rule):
    """(a ragged one-rank layer that has not run, the layer with fixed pools whose capacities fit the same counts)."""
    seed = 4
    inp = _drawn(sh, gen.generate(sh, seed=seed, send_cap=O.capacities(sh)[0]))
    probe = runner.RaggedOneRankLayer(replace(sh, layer="dispatch"), inp, expert_rows=sh.n_ranks * sh.tokens, rule=rule)
    probe.run()
    rep = probe.drop_report()
    pool_rows = max(max(rep["send_demand"]), max(probe.source_demand.values()))
    expert_rows = max(rep["expert_arrivals"])
    fit = configs.exact_fit(sh, pool_rows, expert_rows)
    inp = dict(gen.generate(fit, seed=seed, send_cap=pool_rows), sources=inp["sources"])
    return runner.RaggedOneRankLayer(sh, inp, expert_rows, rule=rule), runner.OneRankLayer(fit, inp, rule=rule)


def test_ragged_one_rank_layer_with_a_rule(monkeypatch):
    """The output bits of the fixed-pool layer under the same rule, and another choice than without it."""
    sh = replace(configs.get("mini_bf16"), emulate_all_ranks=False)
    lay, fixed = _ragged_pair(sh, _ruled(monkeypatch, sh))
    for x in (lay, fixed):
        x.run()
    torch.cuda.synchronize()
    assert lay.drop_report()["recv_dropped"] == 0 and fixed.drop_report()["recv_dropped"] == 0
    assert torch.isfinite(lay.out.float()).all() and float(lay.out.float().abs().sum()) > 0
    assert torch.equal(lay.idx, fixed.idx) and torch.equal(lay.w, fixed.w) and torch.equal(lay.out, fixed.out)
    assert torch.equal(lay.idx, block.select_experts(lay.logits, lay.rule)[0])
    plain, _ = _ragged_pair(sh, None)
    plain.run()
    torch.cuda.synchronize()
    assert not torch.equal(plain.idx, lay.idx)


def test_ragged_one_rank_layer_keeps_its_rule(monkeypatch):
    """A balance changed after set-up would put rows where the segments and banks of set-up have no room for them: the layer goes
    on with the one that it was made with.  The layer with fixed pools follows."""
    sh = replace(configs.get("mini_bf16"), emulate_all_ranks=False)
    rule = _ruled(monkeypatch, sh)
    lay, fixed = _ragged_pair(sh, rule)
    outs = []
    for change in (0.0, 0.2):
        rule.balance.add_(torch.linspace(-change, change, sh.n_experts, device=DEV))
        for x in (lay, fixed):
            x.run()
        torch.cuda.synchronize()
        outs.append([t.clone() for t in (lay.idx, lay.w, lay.out, fixed.idx)])
        assert lay.drop_report()["recv_bad_ids"] == 0
    for a, b in zip(outs[0][:3], outs[1]):
        assert torch.equal(a, b)
    assert not torch.equal(outs[0][3], outs[1][3])
