"""The measured cases of the operators around the experts' products, with their plain forms.

* norm: root-mean-square norm of rows, with the residual stream's addition before it, as activations, as MX-FP8 rows or as
  both, and its backward pass (rms_norm, rms_norm_backward);
* select: the choice of experts from router logits: softmax or sigmoid scores, a balance bias that counts for the choice
  alone, groups of experts, the k best, weights renormalised over them, and the logits' gradient (select_experts,
  select_experts_backward);
* swiglu: silu(gate) * up of the experts' rows, the gate and up values kept for the backward pass as MX-FP8 rows, and that
  backward pass (swiglu_checkpoint, swiglu_backward);
* gemm: out[g] = A[g] . B[g]^T of MX-FP8 rows A with MX-FP4 rows B, grouped by expert (mx8_gemm).

MX-FP8: a block of 32 consecutive values along a row shares the scale 2^e with the smallest e in [-127, 127] for which
max|x| 2^-e is at most 448 (stored as e + 127); a value is x 2^-e rounded to the nearest E4M3 value (ties to the even one).
MX-FP4: blocks of 32 values of 0, .5, 1, 1.5, 2, 3, 4, 6 and a sign, two codes a byte with the first in the low half.  Rows of
scales are padded to a multiple of 16 bytes in both.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one token of a decode on its way into 4-bit experts: a latency-bound call
        {"name": "norm_one_token", "op": "norm", "rows": 1, "cols": 6144, "form": "mx8", "residual": True, "back": "no", "pad": 0,
         "act": "bf16"},
        # a 4K-context batch: the router reads the bf16 rows, the products the 8-bit ones
        {"name": "norm_prompt", "op": "norm", "rows": 8192, "cols": 6144, "form": "both", "residual": True, "back": "no", "pad": 0,
         "act": "bf16"},
        # a training step of a small fp32 layer, rows that are part of a wider buffer
        {"name": "norm_step_odd_f32", "op": "norm", "rows": 2077, "cols": 1000, "form": "act", "residual": True, "back": "step",
         "pad": 36, "act": "f32"},
        # the backward pass over a long context
        {"name": "norm_back_long", "op": "norm", "rows": 65536, "cols": 6144, "form": "act", "residual": True, "back": "only",
         "pad": 0, "act": "bf16"},
        # one token's choice: 8 of 384 experts out of the 4 best of 8 groups
        {"name": "select_one_token", "op": "select", "t": 1, "e": 384, "k": 8, "score": "sigmoid", "groups": 8, "top_groups": 4,
         "balance": True, "renorm": True, "masked": 0, "back": False},
        # the long-context batch's choice under the plain rule
        {"name": "select_long", "op": "select", "t": 65536, "e": 384, "k": 8, "score": "softmax", "groups": 1, "top_groups": 1,
         "balance": False, "renorm": True, "masked": 0, "back": False},
        # a training step's choice and its gradient, balanced, in groups, some experts out of service
        {"name": "select_step_groups", "op": "select", "t": 8192, "e": 384, "k": 8, "score": "sigmoid", "groups": 8,
         "top_groups": 4, "balance": True, "renorm": True, "masked": 5, "back": True},
        # an odd number of rows a small fp32 expert got
        {"name": "swiglu_few_f32", "op": "swiglu", "groups": 6, "m": 37, "h": 352, "ragged": True, "act": "f32"},
        # one wave of a rank's experts at their receive cap (the 4K-context layer's loads)
        {"name": "swiglu_wave", "op": "swiglu", "groups": 2, "m": 12562, "h": 2048, "ragged": True, "act": "bf16"},
        # a small batch of tokens against a projection
        {"name": "gemm_16_rows", "op": "gemm", "groups": 1, "m": 16, "n": 4096, "k": 6144, "ragged": False, "act": "bf16"},
        # the local experts of one rank, each with its own number of rows, odd widths
        {"name": "gemm_six_experts", "op": "gemm", "groups": 6, "m": 1178, "n": 2815, "k": 2080, "ragged": True, "act": "bf16"},
        # a prompt's batch against a model-wide projection
        {"name": "gemm_prompt", "op": "gemm", "groups": 1, "m": 8192, "n": 6144, "k": 6144, "ragged": False, "act": "bf16"},
    ]


def draw(rng):
    def upto(lo, hi):  # spread over the logarithm
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["norm", "select", "swiglu", "gemm"])
    act = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        back = rng.choice(["no", "step", "only"])
        form = "act" if back != "no" else rng.choice(["act", "mx8", "both"])
        cols = 32 * upto(1, 192) if form != "act" else rng.choice([upto(8, 6144), 8 * upto(1, 768)])
        return {"op": op, "rows": upto(1, 65536 if act == "bf16" else 16384), "cols": cols, "form": form,
                "residual": rng.random() < 0.7, "back": back, "pad": 8 * rng.randrange(4) if cols % 8 == 0 else rng.randrange(4),
                "act": act}
    if op == "select":
        groups = rng.choice([1, 1, 2, 4, 8, 12])
        e = groups * upto(max(1, 8 // groups), 2048 // groups)
        top_groups = rng.randint(1, groups)
        room = top_groups * (e // groups)   # experts to choose from
        k = rng.randint(1, min(room, rng.choice([2, 8, 16])))
        masked = rng.randint(0, min(4, e // groups - 1, room - k)) if rng.random() < 0.3 else 0
        return {"op": op, "t": min(upto(1, 65536), 65536 * 384 // e), "e": e, "k": k, "score": rng.choice(["softmax", "sigmoid"]),
                "groups": groups, "top_groups": top_groups, "balance": rng.random() < 0.5,
                "renorm": k > 1 and rng.random() < 0.7,   # the only expert's weight would be 1, its gradient 0
                "masked": masked, "back": rng.random() < 0.5}
    if op == "swiglu":
        groups = rng.choice([1, 2, 3, 6])
        return {"op": op, "groups": groups, "m": upto(1, 25000 // groups), "h": 32 * upto(1, 64), "ragged": groups > 1, "act": act}
    groups = rng.choice([1, 1, 2, 3, 6, 8])
    return {"op": op, "groups": groups, "m": upto(1, 8192 // groups), "n": upto(1, 6144), "k": 32 * upto(1, 192),
            "ragged": groups > 1, "act": act}


FILL = 0.8  # the mean of prepare()'s row counts, as a share of the rows a group has room for


def work(case):
    size = 2 if case.get("act") == "bf16" else 4
    if case["op"] == "norm":
        n, moved, flops = case["rows"] * case["cols"], 0, 0
        if case["back"] != "only":
            eight = 0 if case["form"] == "act" else 33 / 32
            wide = 0 if case["form"] == "mx8" else size
            moved += size * (3 if case["residual"] else 1) + wide
            moved += eight * 2 + size if eight else 0   # written, and read back as the values it stands for
            flops += 6
        if case["back"] != "no":
            moved += size * (4 if case["residual"] else 3)
            flops += 10
        return {"bytes": n * moved + 8 * case["cols"], "flops": flops * n}
    if case["op"] == "select":
        t, e, k = case["t"], case["e"], case["k"]
        return {"bytes": t * (4 * e + 8 * k) + (t * (4 * e + 4 * k) if case["back"] else 0), "flops": 10 * t * e}
    if case["op"] == "swiglu":
        n = case["groups"] * case["m"] * case["h"] * (FILL if case["ragged"] else 1)
        # gate and up read, h written, 8-bit rows written and read again, h's gradient read, h and two gradients written
        return {"bytes": n * (size * 7 + 4 * 33 / 32), "flops": 30 * n}
    g, m, n, k = case["groups"], case["m"], case["n"], case["k"]
    if case["ragged"]:
        m = m * FILL
    return {"bytes": g * (m * k * 33 / 32 + n * k * 17 / 32 + m * n * size), "flops": 2.0 * g * m * n * k}


# ---------------------------------------------------------------- inputs

def _counts(gen, groups, m):
    fill = 2 * FILL - 1 + 2 * (1 - FILL) * torch.rand((groups,), generator=gen, device=DEV)
    return (fill * m).round().to(torch.int32)


def _rows(gen, shape, pad, act, spread):
    """Rows of normal values (some channels much larger than others where `spread`), part of wider ones where `pad`."""
    cols = shape[-1]
    x = torch.randn(shape[:-1] + (cols + pad,), generator=gen, device=DEV)
    if spread:
        x *= torch.exp(torch.randn((cols + pad,), generator=gen, device=DEV) * spread)
    return x.to(act)[..., :cols]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    act = TYPES[case.get("act", "f32")]
    if case["op"] == "norm":
        shape, pad = (case["rows"], case["cols"]), case["pad"]
        st = {"op": "norm", "form": case["form"], "back": case["back"], "act": act, "plan": None,
              "x": _rows(gen, shape, pad, act, 0.7),
              "residual": _rows(gen, shape, pad, act, 0.7).mul_(3) if case["residual"] and case["back"] != "only" else None,
              "weight": (1 + 0.2 * torch.randn((case["cols"],), generator=gen, device=DEV)).to(act)}
        if case["back"] != "no":
            st["dy"] = _rows(gen, shape, pad, act, 0).mul_(0.1)
            st["dstream"] = _rows(gen, shape, pad, act, 0).mul_(0.1) if case["residual"] else None
        return st
    if case["op"] == "select":
        t, e = case["t"], case["e"]
        logits = torch.randn((t, e), generator=gen, device=DEV) * 1.5 + torch.randn((e,), generator=gen, device=DEV) * 0.5
        if case["masked"]:
            logits[:, torch.randperm(e, generator=gen, device=DEV)[:case["masked"]]] = -math.inf
        return {"op": "select", "logits": logits, "plan": None, "back": case["back"],
                "balance": torch.randn((e,), generator=gen, device=DEV) * 0.05 if case["balance"] else None,
                "dw": torch.randn((t, case["k"]), generator=gen, device=DEV),
                **{n: case[n] for n in ("k", "score", "groups", "top_groups", "renorm")}}
    if case["op"] == "swiglu":
        g, m, h = case["groups"], case["m"], case["h"]
        gate_up = torch.empty((g, m, 2 * h), dtype=act, device=DEV)
        for i in range(g):   # group by group, as the largest are some GB in fp32
            gate_up[i] = _rows(gen, (m, 2 * h), 0, act, 0.5)
        dh = torch.randn((g, m, h), generator=gen, device=DEV).mul_(0.1).to(act)
        return {"op": "swiglu", "gate_up": gate_up, "dh": dh, "act": act, "counts": _counts(gen, g, m) if case["ragged"] else None,
                "plan": {"h": torch.zeros_like(dh), "dgate_up": torch.zeros_like(gate_up), "hidden": torch.zeros_like(dh)}}
    g, m, n, k = case["groups"], case["m"], case["n"], case["k"]
    a = torch.empty((g, m, k), dtype=torch.uint8, device=DEV)
    a_scales = torch.zeros((g, m, (k // 32 + 15) // 16 * 16), dtype=torch.uint8, device=DEV)
    b = torch.empty((g, n, k // 2), dtype=torch.uint8, device=DEV)
    b_scales = torch.zeros((g, n, (k // 32 + 15) // 16 * 16), dtype=torch.uint8, device=DEV)
    for i in range(g):
        x = torch.randn((m, k), generator=gen, device=DEV) * torch.exp(torch.randn((k,), generator=gen, device=DEV) * 0.5)
        values, a_scales[i, :, :k // 32] = _eight(x)
        a[i] = _eight_codes(values, a_scales[i, :, :k // 32])
        b[i] = torch.randint(0, 256, (n, k // 2), generator=gen, device=DEV, dtype=torch.uint8)
        # scales around those of weights of about 1 / sqrt(k)
        b_scales[i, :, :k // 32] = (124 - int(math.log2(k) / 2)
                                    + torch.randint(0, 3, (n, k // 32), generator=gen, device=DEV)).to(torch.uint8)
    return {"op": "gemm", "a": a, "a_scales": a_scales, "b": b, "b_scales": b_scales, "act": act,
            "counts": _counts(gen, g, m) if case["ragged"] else None, "out": torch.zeros((g, m, n), dtype=act, device=DEV)}


# ---------------------------------------------------------------- plain forms

def _eight(x):
    """fp32 rows -> (their MX-FP8 values in fp32, scale bytes)."""
    blocks = x.reshape(*x.shape[:-1], -1, 32)
    bits = blocks.abs().amax(-1).view(torch.int32)
    e = (((bits + 0x1fffff) >> 23) - 135).clamp(min=-127)   # one more where the largest's fraction is above 1.75
    y = blocks * ((127 - e) << 23).view(torch.float32)[..., None]
    exponent = (y.abs().view(torch.int32) >> 23) - 127
    step = (exponent.clamp(min=-6) + (127 - 3)).bitwise_left_shift(23).view(torch.float32)   # spacing of E4M3 at y
    unit = (e + 128 << 23).view(torch.float32) * 0.5                                          # 2^e, 2^-127 among them
    return (torch.round(y / step) * step * unit[..., None]).reshape(x.shape), (e + 127).to(torch.uint8)


def _eight_codes(values, scales):
    """Values on the MX-FP8 grid of their blocks -> E4M3 codes."""
    y = values.reshape(*values.shape[:-1], -1, 32) * ((254 - scales.int()) << 23).view(torch.float32)[..., None]
    bits = y.abs().view(torch.int32)
    normal = (bits >> 20) - (120 << 3)   # exponent field and three fraction bits
    code = torch.where(bits >= 121 << 23, normal, torch.round(y.abs() * 512).int()) + 128 * (y < 0).int()
    return code.to(torch.uint8).reshape(values.shape)


def _unit(scales, k):
    """Scale bytes -> 2^(byte - 127) in fp32."""
    return ((scales[..., :k // 32].int() + 1 << 23).view(torch.float32) * 0.5)[..., None]


def _eight_values(codes, scales):
    c = codes.int()
    field, fraction = (c >> 3) & 15, (c & 7).float()
    v = torch.where(field == 0, fraction / 512, (1 + fraction / 8) * (field + 120 << 23).view(torch.float32))
    v = torch.where(c >= 128, -v, v).reshape(*codes.shape[:-1], -1, 32)
    return (v * _unit(scales, codes.shape[-1])).reshape(codes.shape)


def _four_values(codes, scales):
    half = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    byte = torch.arange(256, device=codes.device)
    v = torch.stack([half[byte & 15], half[byte >> 4]], -1)[codes.int()].reshape(*codes.shape[:-1], -1, 32)
    return (v * _unit(scales, codes.shape[-1] * 2)).reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def _plain_norm(st):
    out, act, w = {}, st["act"], st["weight"].float()
    s = st["x"]
    if st["back"] != "only":
        wide = s.float()
        if st["residual"] is not None:
            wide = wide + st["residual"].float()
            s = out["stream"] = wide.to(act)
        y = wide * torch.rsqrt((wide * wide).mean(-1, keepdim=True) + EPS) * w
        if st["form"] != "mx8":
            out["y"] = y.to(act)
        if st["form"] != "act":
            out["rows"] = _eight(y)[0].to(act)
    if st["back"] != "no":
        s, dy = s.float(), st["dy"].float()
        r = torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS)
        n = s * r
        out["dweight"] = (dy * n).sum(0, dtype=torch.float64).float()
        g = dy * w
        dx = (g - n * (g * n).mean(-1, keepdim=True)) * r
        if st["dstream"] is not None:
            dx = dx + st["dstream"].float()
        out["dx"] = dx.to(act)
    return out


def _plain_select(st):
    # in 64 bits: experts whose scores differ in the last places of 32 change places otherwise
    logits = st["logits"].double()
    score = torch.sigmoid(logits) if st["score"] == "sigmoid" else torch.softmax(logits, 1)
    t, e, g = *logits.shape, st["groups"]
    rank = score if st["balance"] is None else score + st["balance"].double()
    rank = rank.masked_fill(logits == -math.inf, -math.inf)   # an expert out of service
    if st["top_groups"] < g:
        best = rank.view(t, g, e // g).topk(min(2, e // g), -1).values
        best = torch.where(best[..., 0] > -math.inf, torch.where(best > -math.inf, best, 0.0).sum(-1), -math.inf)
        kept = torch.zeros((t, g), dtype=torch.bool, device=DEV)
        kept.scatter_(1, torch.sort(best, dim=1, descending=True, stable=True).indices[:, :st["top_groups"]], True)
        rank = rank.view(t, g, -1).masked_fill(~kept[..., None], -math.inf).view(t, e)
    idx = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :st["k"]]
    w = score.gather(1, idx)
    if st["renorm"]:
        w = w / w.sum(1, keepdim=True)
    out = {"idx": idx.int(), "w": w.float()}
    if st["back"]:
        dw = st["dw"].double()
        mean = (w * dw).sum(1, keepdim=True)
        if st["score"] == "sigmoid":
            chosen = w * (1 - score.gather(1, idx)) * (dw - mean if st["renorm"] else dw)
            out["dlogits"] = torch.zeros_like(logits).scatter_(1, idx, chosen).float()
        elif st["renorm"]:
            out["dlogits"] = torch.zeros_like(logits).scatter_(1, idx, w * (dw - mean)).float()
        else:
            out["dlogits"] = (-score * mean).scatter_add_(1, idx, w * dw).float()
    return out


def _plain_swiglu(st):
    gate_up, dh, act = st["gate_up"].float(), st["dh"].float(), st["act"]
    n = dh.shape[-1]
    here = None if st["counts"] is None else (torch.arange(dh.shape[1], device=DEV) < st["counts"][:, None])[..., None]
    keep = lambda v: (v if here is None else v * here).to(act)  # noqa: E731
    sig = torch.sigmoid(gate_up[..., :n])
    out = {"h": keep(gate_up[..., :n] * sig * gate_up[..., n:])}
    kept = _eight(gate_up)[0]
    gate, up = kept[..., :n], kept[..., n:]
    sig = torch.sigmoid(gate)
    out["hidden"] = keep(gate * sig * up)
    out["dgate_up"] = keep(torch.cat([dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig], -1))
    return out


def _plain(st):
    if st["op"] == "norm":
        return _plain_norm(st)
    if st["op"] == "select":
        return _plain_select(st)
    if st["op"] == "swiglu":
        return _plain_swiglu(st)
    out = torch.matmul(_eight_values(st["a"], st["a_scales"]), _four_values(st["b"], st["b_scales"]).transpose(1, 2))
    if st["counts"] is not None:
        out = out * (torch.arange(out.shape[1], device=DEV) < st["counts"][:, None])[..., None]
    return {"out": out.to(st["act"])}


def _own(st):
    from grouped_expert_ffn_router_amd import block, runner
    if st["op"] == "norm":
        out, s = {}, st["x"]
        if st["back"] != "only":
            y, s = block.rms_norm(s, st["weight"], residual=st["residual"], eps=EPS, form=st["form"])
            y, rows = y if st["form"] == "both" else (None, y) if st["form"] == "mx8" else (y, None)
            if st["residual"] is not None:
                out["stream"] = s
            if y is not None:
                out["y"] = y
            if rows is not None:
                out["rows"] = block.mx8_dequantize(rows, st["act"])
        if st["back"] != "no":
            dx, dw = block.rms_norm_backward(st["dy"], s, st["weight"], dstream=st["dstream"], eps=EPS)
            out["dweight"], out["dx"] = dw, dx
        return out
    if st["op"] == "select":
        if st["plan"] is None:   # the rule a program is configured with
            st["plan"] = block.RouterRule(st["k"], score=st["score"], balance=st["balance"], groups=st["groups"],
                                          top_groups=st["top_groups"], renormalise=st["renorm"])
        idx, w = block.select_experts(st["logits"], st["plan"])
        out = {"idx": idx, "w": w}
        if st["back"]:
            out["dlogits"] = block.select_experts_backward(st["dw"], w, idx, st["logits"], st["plan"])
        return out
    if st["op"] == "swiglu":
        bufs = st["plan"]
        h, saved = block.swiglu_checkpoint(st["gate_up"], counts=st["counts"], out=bufs["h"])
        dgate_up, hidden = block.swiglu_backward(st["dh"], saved, counts=st["counts"], out=bufs["dgate_up"],
                                                 hidden_out=bufs["hidden"])
        return {"h": h, "hidden": hidden, "dgate_up": dgate_up}
    cols = st["a"].shape[-1]
    return {"out": block.mx8_gemm(block.Mx8Rows(st["a"], st["a_scales"], cols), runner.MxRows(st["b"], st["b_scales"], cols),
                                  counts=st["counts"], out=st["out"])}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- in 64 bits

def _grid(x):
    """Rows in 64 bits -> the MX-FP8 values of each block, from the definition."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / 448))
    e = torch.where(top * torch.exp2(-e) > 448, e + 1, e)       # where the logarithm was rounded
    e = torch.where(top * torch.exp2(1 - e) <= 448, e - 1, e)
    e = e.clamp(-127, 127)
    y = b * torch.exp2(-e)
    quantum = torch.exp2((torch.frexp(y.abs()).exponent - 1).clamp(min=-6).double() - 3)
    return (torch.round(y / quantum) * quantum * torch.exp2(e)).reshape(x.shape)


def _decode(codes, scales, bits):
    if bits == 4:
        c = torch.stack([codes % 16, codes // 16], -1).flatten(-2).to(torch.int64)
        sign, exp, frac, places, bias = c // 8, (c % 8) // 2, c % 2, 1, 1
    else:
        c = codes.to(torch.int64)
        sign, exp, frac, places, bias = c // 128, (c % 128) // 8, c % 8, 3, 7
    f = frac.double() / 2 ** places
    v = torch.where(exp == 0, f * 2.0 ** (1 - bias), (1 + f) * torch.exp2(exp.double() - bias))
    v = torch.where(sign > 0, -v, v).unflatten(-1, (-1, 32))
    return (v * torch.exp2(scales[..., :v.shape[-2]].double() - 127)[..., None]).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    if st["op"] == "norm":
        return _exact_norm(st)
    if st["op"] == "select":
        return _exact_select(st)
    if st["op"] == "swiglu":
        shape, n = st["dh"].shape, st["dh"].shape[-1]
        out = {"h": torch.zeros(shape, dtype=torch.float64, device=DEV), "hidden": torch.zeros(shape, dtype=torch.float64, device=DEV),
               "dgate_up": torch.zeros(st["gate_up"].shape, dtype=torch.float64, device=DEV)}
        for i in range(shape[0]):
            rows = shape[1] if st["counts"] is None else int(st["counts"][i])
            full = st["gate_up"][i, :rows].double()
            gate, up = full.chunk(2, -1)
            out["h"][i, :rows] = gate / (1 + torch.exp(-gate)) * up
            gate, up = _grid(full).chunk(2, -1)
            d, sig = st["dh"][i, :rows].double(), 1 / (1 + torch.exp(-gate))
            out["hidden"][i, :rows] = gate * sig * up
            out["dgate_up"][i, :rows, :n] = d * up * (sig + gate * torch.exp(-gate) * sig * sig)
            out["dgate_up"][i, :rows, n:] = d * gate * sig
        return out
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    for g in range(out.shape[0]):
        rows = out.shape[1] if st["counts"] is None else int(st["counts"][g])
        out[g, :rows] = _decode(st["a"][g, :rows], st["a_scales"][g, :rows], 8) @ _decode(st["b"][g], st["b_scales"][g], 4).T
    return {"out": out}


def _exact_norm(st):
    out, w = {}, st["weight"].double()
    s = st["x"].double()
    cols = s.shape[1]
    if st["back"] != "only":
        if st["residual"] is not None:
            s = out["stream"] = s + st["residual"].double()
        y = s / torch.sqrt(torch.linalg.vector_norm(s, dim=1, keepdim=True) ** 2 / cols + EPS) * w
        if st["form"] != "mx8":
            out["y"] = y
        if st["form"] != "act":
            out["rows"] = _grid(y)
    if st["back"] != "no":
        s, dy = s.to(st["act"]).double(), st["dy"].double()   # the stream as it is kept
        square = torch.linalg.vector_norm(s, dim=1, keepdim=True) ** 2 / cols + EPS
        out["dweight"] = torch.einsum("rc,rc,r->c", dy, s, square[:, 0] ** -0.5)
        dx = dy * w / torch.sqrt(square) - s * (dy * w * s).sum(1, keepdim=True) / (cols * square ** 1.5)
        out["dx"] = dx if st["dstream"] is None else dx + st["dstream"].double()
    return out


def _exact_select(st):
    logits, k, g = st["logits"].double(), st["k"], st["groups"]
    t, e = logits.shape
    top = logits.amax(1, keepdim=True)
    score = 1 / (1 + torch.exp(-logits)) if st["score"] == "sigmoid" else torch.exp(logits - top) / torch.exp(logits - top).sum(1, keepdim=True)
    rank = score.clone() if st["balance"] is None else score + st["balance"].double()
    out_of_service = torch.isneginf(logits)
    if st["top_groups"] < g:
        parts = torch.where(out_of_service, math.nan, rank).view(t, g, e // g)
        ordered = torch.sort(torch.nan_to_num(parts, nan=-math.inf), -1, descending=True).values[..., :2]
        total = torch.where(torch.isinf(ordered), 0.0, ordered).sum(-1)
        total[torch.isinf(ordered[..., 0])] = -math.inf
        place = torch.argsort(torch.argsort(-total, dim=1, stable=True), dim=1)   # a group's place among the groups
        out_of_service = out_of_service | (place >= st["top_groups"]).repeat_interleave(e // g, 1)
    idx = torch.argsort(torch.where(out_of_service, math.inf, -rank), dim=1, stable=True)[:, :k]
    chosen = torch.zeros_like(logits).scatter_(1, idx, 1.0)
    # weight of expert j as a function of all logits, its Jacobian applied to the weights' gradient
    picked = score * chosen
    total = picked.sum(1, keepdim=True)
    dense = picked / total if st["renorm"] else picked
    out = {"idx": idx.int(), "w": dense.gather(1, idx)}
    if st["back"]:
        dwide = torch.zeros_like(logits).scatter_(1, idx, st["dw"].double())
        dscore = chosen * (dwide / total - (dwide * picked).sum(1, keepdim=True) / total ** 2) if st["renorm"] else dwide
        if st["score"] == "sigmoid":
            out["dlogits"] = dscore * score * (1 - score)
        else:
            out["dlogits"] = score * (dscore - (dscore * score).sum(1, keepdim=True))
    return out
