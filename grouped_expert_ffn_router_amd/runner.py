"""Device buffers and the call sequence of the MoE layer on one GPU.

torch provides device memory, copies and streams; every step of the layer is
a libmoe call (see binding.py).  Two layouts of the expert-parallel domain
are provided:

* ``OneRankLayer``: one rank's share at its real shape.  The rank's own
  tokens go through route -> pack; its receive buffer holds its own pool for
  itself plus the pools the other ranks sent; its combine reads the rows it
  computed for itself plus the rows the other ranks returned (inputs).  When
  the workload gives the other ranks' tokens, their pools are made at set-up
  by running those ranks' route -> pack through the same library calls
  (untimed: it stands for what the other GPUs do); otherwise they are
  inputs.  The only copies in a step are the self-blocks of the exchanges.
* ``AllRanksLayer``: every rank of a small domain on one device.  All send
  pools sit in one [R_src][R_dst][send_cap][stride] block and all return rows
  in one [R_recv][R_src][send_cap][L] block, so each exchange is a strided
  view: zero copies.
"""

import contextlib
import threading

import numpy as np
import torch

from . import binding as B


def upload(arr, device):
    """Host array (uint16 bf16 bit patterns, float32, int32 or raw bytes) -> device tensor."""
    a = np.ascontiguousarray(arr)
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).to(device).view(torch.bfloat16)
    if a.dtype == np.float32:
        return torch.from_numpy(a).to(device)
    if a.dtype in (np.int32, np.uint8):
        return torch.from_numpy(a).to(device)
    raise TypeError(f"unsupported host dtype {a.dtype}")


def rank_blocks(R, shape, dtype, device):
    """An [R][*shape] tensor whose per-rank blocks each start 256-byte aligned
    (the library takes 16-byte aligned activation pointers; a plain [R][T][n]
    tensor puts rank r at r*T*n elements, unaligned for odd widths)."""
    n = int(np.prod(shape))
    es = torch.empty((), dtype=dtype).element_size()
    stride = -(-n * es // 256) * 256 // es
    return torch.empty((R, stride), dtype=dtype, device=device)[:, :n].unflatten(1, tuple(shape))


def upload_rank_blocks(arr, device):
    """upload() of a host [R][...] array into 256-byte aligned per-rank blocks."""
    t = upload(arr, device)
    out = rank_blocks(t.shape[0], t.shape[1:], t.dtype, device)
    out.copy_(t)
    return out


def _act(shape):
    return torch.bfloat16 if shape.act == "bf16" else torch.float32


def pool_block_host(ids, rows, prow, act):
    """Host bytes of pools in the row layout of moe_pack_pools: [n][cap][prow]."""
    n, cap = ids.shape
    L = rows.shape[-1]
    esize = 2 if act == "bf16" else 4
    out = np.zeros((n, cap, prow), dtype=np.uint8)
    payload = np.ascontiguousarray(rows).view(np.uint8).reshape(n, cap, L * esize)
    out[:, :, :L * esize] = payload
    out[:, :, L * esize:L * esize + 4] = np.ascontiguousarray(ids, dtype=np.int32).view(np.uint8).reshape(n, cap, 4)
    return out


def _expert_form(experts):
    if experts not in ("act", "mx"):
        raise ValueError(f"experts={experts!r}: 'act' (the layer's type) or 'mx' (MX-FP4)")
    return experts


def _expert_gemm(dims, wave, wave_buf, pools, src_stride, row_src, wave_count, w13, w2, ret, ret_stride, ws, ws_mx,
                 stream):
    """The expert FFNs of one wave, by the form of the weights (tensors or MxRows)."""
    if ws_mx is None:
        B.expert_gemm(dims, wave, wave_buf, pools, src_stride, row_src, wave_count, w13, w2, ret, ret_stride, ws, stream)
    else:
        B.mx_expert_gemm(dims, wave, wave_buf, pools, src_stride, row_src, wave_count, w13.arg, w2.arg, ret, ret_stride,
                         ws, ws_mx, stream)


class OneRankLayer:
    """One EP rank's layer.  ``inp`` is a workload.gen.generate() dict.
    experts="mx" quantises the routed experts to MX-FP4 rows and runs their
    products on them (moe_mx_expert_gemm), which rounds the tokens' rows and
    the hidden rows to 4 bits too."""

    def __init__(self, shape, inp, device="cuda", gather="fused", keep_source_logits=False, live_waves=0,
                 experts="act"):
        self.shape, self.device = shape, device
        self.experts = _expert_form(experts)
        self.gather = gather
        # waves whose scratch (hidden rows, partial tiles) the workspace holds at once
        self.live_waves = live_waves if live_waves else shape.waves
        # keep_source_logits: the router logits each other rank computed at
        # set-up, as host float32 arrays (source_logits[s]), for inspection
        self.source_logits = {} if keep_source_logits else None
        r = int(inp["receiver"])
        self.rank = r
        self.dims = B.make_dims(shape, my_rank=r, live_waves=self.live_waves)
        self.scap, self.rcap, self.prow = B.capacity(self.dims)
        T, D, L, E, k, R = shape.tokens, shape.d_model, shape.latent, shape.n_experts, shape.top_k, shape.n_ranks
        X, W, H = shape.local_experts, shape.waves, shape.expert_hidden
        WX = X // W
        act = _act(shape)
        dev = device
        self.full = shape.layer == "full"
        # inputs
        self.x = upload(inp["x"], dev)
        self.w_router = upload(inp["w_router"], dev)
        self.w_down = upload(inp["w_down"], dev)
        self.bias = None if inp["bias"] is None else upload(np.ascontiguousarray(inp["bias"], np.float32), dev)
        self.bias_row_tokens = int(inp["bias_row_tokens"])
        # route / pack outputs
        self.logits = torch.empty((T, E), dtype=torch.float32, device=dev)
        self.z = torch.empty((T, L), dtype=act, device=dev)
        self.idx = torch.empty((T, k), dtype=torch.int32, device=dev)
        self.w = torch.empty((T, k), dtype=torch.float32, device=dev)
        self.send_pools = torch.empty((R, self.scap, self.prow), dtype=torch.uint8, device=dev)
        self.slot_of = torch.empty((T, k), dtype=torch.int32, device=dev)
        self.send_count = torch.empty((R,), dtype=torch.int32, device=dev)
        # receive side: slot s holds the pool source s sent; slot r is our own pool
        if "sources" in inp:
            self.recv_pools = torch.zeros((R, self.scap, self.prow), dtype=torch.uint8, device=dev)
        else:
            self.recv_pools = upload(pool_block_host(inp["foreign_ids"], inp["foreign_rows"], self.prow, shape.act),
                                     dev)
        self.row_src = torch.empty((W, WX, self.rcap), dtype=torch.int32, device=dev)
        self.wave_count = torch.empty((W, WX), dtype=torch.int32, device=dev)
        self.wave_buf = torch.empty((WX, self.rcap, L), dtype=act, device=dev) if gather == "buffer" else None
        self.ws = torch.empty((B.workspace_size(self.dims),), dtype=torch.uint8, device=dev)
        if self.full:
            self.w13 = upload(inp["w13"], dev)
            self.w2 = upload(inp["w2"], dev)
            self._quantize_experts(self.dims)
            self.w_up = upload(inp["w_up"], dev)
            self.ws13 = upload(inp["ws13"], dev)
            self.ws2 = upload(inp["ws2"], dev)
            self.ret_send = torch.zeros((R, self.scap, L), dtype=act, device=dev)
            self.ret_recv = upload(inp["foreign_ret"], dev)
            self.out = torch.empty((T, D), dtype=act, device=dev)
            self._ev_go, self._ev_shared, self._ev_ranked = torch.cuda.Event(), torch.cuda.Event(), torch.cuda.Event()
        self.source_demand = {}
        if "sources" in inp:
            self._route_other_ranks(inp["sources"])

    def _route_other_ranks(self, sources):
        """Each other rank s routes its own tokens and packs its pools; keep the
        pool it sends to this rank (uses this layer's dispatch buffers, which
        the rank's own dispatch overwrites later)."""
        from concurrent.futures import ThreadPoolExecutor
        others = [s for s in range(self.shape.n_ranks) if s != self.rank]
        with ThreadPoolExecutor(max_workers=8) as ex:  # host draws overlap the GPU work
            drawn = ex.map(sources, others)
            for s, host_x in zip(others, drawn):
                self._route_one(s, host_x)
        torch.cuda.synchronize()

    def _route_one(self, s, host_x):
        xs = upload(host_x, self.device)
        d = self.dims
        B.route(d, xs, self.w_router, self.w_down, self.bias, self.bias_row_tokens, self.logits, self.z,
                self.idx, self.w, self.ws)
        B.pack_pools(d, self.z, self.idx, self.send_pools, self.scap * self.prow, self.slot_of, self.send_count,
                     self.ws)
        self.recv_pools[s].copy_(self.send_pools[self.rank])
        if self.source_logits is not None:
            self.source_logits[s] = self.logits.cpu().numpy()
        # rows source s wants to send here, before its send cap (the count a
        # dropless exchange would send ahead of the rows)
        self.source_demand[s] = B.drop_stats(d, self.ws, raise_on_bad_ids=False).send_demand[self.rank]

    @property
    def esize(self):
        return 2 if self.shape.act == "bf16" else 4

    def dispatch(self, stream=None):
        d = self.dims
        B.route(d, self.x, self.w_router, self.w_down, self.bias, self.bias_row_tokens, self.logits, self.z,
                self.idx, self.w, self.ws, stream)
        B.pack_pools(d, self.z, self.idx, self.send_pools, self.scap * self.prow, self.slot_of,
                     self.send_count, self.ws, stream)
        # self-block of the dispatch exchange
        self.recv_pools[self.rank].copy_(self.send_pools[self.rank])

    def receive_rank(self, stream=None):
        B.recv_rank(self.dims, self.recv_pools, self.scap * self.prow, self.ws, stream)

    def receive_wave(self, w, stream=None):
        B.recv_waves(self.dims, self.recv_pools, self.scap * self.prow, w, self.wave_buf, self.row_src[w],
                     self.wave_count[w], self.ws, stream)

    def _quantize_experts(self, dims):
        """experts="mx": the routed experts as MX-FP4 rows, and the scratch of their products."""
        self.ws_mx = None
        if self.experts == "mx":
            self.w13, self.w2 = mx_quantize(self.w13), mx_quantize(self.w2)
            self.ws_mx = torch.empty((B.mx_workspace_size(dims),), dtype=torch.uint8, device=self.device)

    def expert_wave(self, w, stream=None):
        _expert_gemm(self.dims, w, self.wave_buf, self.recv_pools, self.scap * self.prow, self.row_src[w],
                     self.wave_count[w], self.w13, self.w2, self.ret_send, self.scap * self.shape.latent * self.esize,
                     self.ws, self.ws_mx, stream)

    def shared(self, stream=None):
        B.shared_experts(self.dims, self.x, self.ws13, self.ws, stream)

    def combine(self, stream=None):
        # self-block of the return exchange
        self.ret_recv[self.rank].copy_(self.ret_send[self.rank])
        B.combine(self.dims, self.ret_recv, self.scap * self.shape.latent * self.esize, self.slot_of, self.w,
                  self.w_up, self.ws2, self.out, self.ws, stream)

    def run(self, stream=None, side=None):
        """One batch on `stream` (torch's current stream if None).  With `side`,
        a second stream, the shared experts and the waves of odd scratch
        blocks (wave w is in block w mod live_waves) run there, beside the
        routed path and the other waves: the shared experts start once
        everything queued before on `stream` (the previous batch's combine,
        which reads their output) is done, the side waves once the receive
        ranking is, and the combine waits for both.  A block's waves always
        share a stream, so they run in order; with one live wave every wave
        runs on `stream`."""
        main = stream if stream is not None else torch.cuda.current_stream()
        waves = self.shape.waves
        with torch.cuda.stream(main):
            if self.full:
                if side is not None:
                    self._ev_go.record(main)
                    side.wait_event(self._ev_go)
                    self.shared(side)
                else:
                    self.shared(main)
            self.dispatch(main)
            self.receive_rank(main)
            # a shared wave buffer ("buffer" gather) keeps the waves in order
            two = side is not None and self.full and self.wave_buf is None and self.live_waves > 1
            if two:
                self._ev_ranked.record(main)
                side.wait_event(self._ev_ranked)
            for w in range(waves):
                st = side if two and (w % self.live_waves) % 2 else main
                self.receive_wave(w, st)
                if self.full:
                    self.expert_wave(w, st)
            if self.full:
                if side is not None:
                    self._ev_shared.record(side)
                    main.wait_event(self._ev_shared)
                self.combine(main)

    def drop_report(self, stream=None):
        return B.drop_stats(self.dims, self.ws, stream, raise_on_bad_ids=False).as_dict()

    def memory(self):
        """Device bytes of one step's buffers.  The SwiGLU hidden rows of a wave
        ([X/W][recv_cap][H] activations) are the part of the receive bank that
        the waves keep small; the workspace holds live_waves such blocks (with
        MX-FP4 experts the MX workspace does, as MX-FP4 rows)."""
        sh = self.shape
        rows = getattr(self, "wave_rows", 0) or (sh.local_experts // sh.waves) * self.rcap
        hidden_wave = rows * sh.expert_hidden * self.esize if self.full else 0
        ws_mx = self.ws_mx if self.full else None
        if ws_mx is not None:
            hidden_wave = rows * sum(_mx_strides(sh.expert_hidden))
        exch = self.send_pools.numel() + self.recv_pools.numel()
        ret = (self.ret_send.numel() + self.ret_recv.numel()) * self.esize if self.full else 0
        return {"live_waves": self.live_waves, "hidden_rows_per_wave_bytes": hidden_wave,
                "hidden_rows_live_bytes": hidden_wave * self.live_waves, "workspace_bytes": self.ws.numel(),
                "wave_buffer_bytes": 0 if self.wave_buf is None else self.wave_buf.numel() * self.esize,
                "exchange_pool_bytes": exch, "return_row_bytes": ret,
                **({} if ws_mx is None else {"mx_workspace_bytes": ws_mx.numel()})}


class RaggedOneRankLayer(OneRankLayer):
    """One EP rank's layer with the dropless ragged exchange (the counterpart of
    RaggedAllRanksLayer at one rank's real shape).  The rank packs its rows
    back to back by destination (moe_pack_ragged, no send cap).  At set-up the
    other ranks route and pack their own tokens the same way (untimed: it
    stands for the other GPUs) and their counts toward this rank fix where
    every source's segment sits in the receive buffer; the inputs are the same
    every step, so the counts are too, and a step copies only the self
    segments of the two exchanges.  ``foreign_ret`` rows (the rows the other
    ranks return, [R][pool_rows][L]) are laid into this rank's ragged order
    once.  ``expert_rows`` is the receive cap of every expert.  With
    ``ragged_banks`` each wave's hidden rows are laid end to end in one bank
    sized to the largest number of rows any wave keeps (moe_dims.wave_rows),
    from per-expert arrival counts taken at set-up (the counts a dropless
    exchange would send ahead of the rows, split by expert); otherwise every
    expert has a bank of expert_rows rows."""

    def __init__(self, shape, inp, expert_rows, device="cuda", gather="fused", ragged_banks=True, live_waves=2,
                 experts="act"):
        from workload.configs import exact_fit
        self.experts = _expert_form(experts)
        if "sources" not in inp:
            raise ValueError("the ragged layer needs a workload whose other ranks route their own tokens")
        self.shape, self.device, self.gather = shape, device, gather
        self.live_waves = min(live_waves, shape.waves) if live_waves else shape.waves
        self.source_logits = None
        r = int(inp["receiver"])
        self.rank = r
        T, D, L, E, k, R = shape.tokens, shape.d_model, shape.latent, shape.n_experts, shape.top_k, shape.n_ranks
        X, W = shape.local_experts, shape.waves
        WX = X // W
        act = _act(shape)
        dev = device
        self.full = shape.layer == "full"
        self._fit = lambda pool_rows: exact_fit(shape, pool_rows, int(expert_rows))
        # set-up dims: neither cap is used by route and pack, and cap 1 keeps
        # the receive parts of the set-up workspace small
        setup_dims = B.make_dims(exact_fit(shape, 1, 1), my_rank=r)
        self.rcap = int(expert_rows)
        self.prow = B.capacity(setup_dims)[2]
        self.x = upload(inp["x"], dev)
        self.w_router = upload(inp["w_router"], dev)
        self.w_down = upload(inp["w_down"], dev)
        self.bias = None if inp["bias"] is None else upload(np.ascontiguousarray(inp["bias"], np.float32), dev)
        self.bias_row_tokens = int(inp["bias_row_tokens"])
        self.logits = torch.empty((T, E), dtype=torch.float32, device=dev)
        self.z = torch.empty((T, L), dtype=act, device=dev)
        self.idx = torch.empty((T, k), dtype=torch.int32, device=dev)
        self.w = torch.empty((T, k), dtype=torch.float32, device=dev)
        self.send_rows = torch.empty((T * k, self.prow), dtype=torch.uint8, device=dev)
        self.send_off = torch.empty((R + 1,), dtype=torch.int32, device=dev)
        self.slot_of = torch.empty((T, k), dtype=torch.int32, device=dev)
        self.send_count = torch.empty((R,), dtype=torch.int32, device=dev)
        ws_setup = torch.zeros((B.workspace_size(setup_dims),), dtype=torch.uint8, device=dev)
        # the other ranks' segments toward this rank, and this rank's own count
        segs = {}
        for s in range(R):
            host_x = inp["x"] if s == r else inp["sources"](s)
            xs = upload(host_x, dev)
            B.route(setup_dims, xs, self.w_router, self.w_down, self.bias, self.bias_row_tokens, self.logits,
                    self.z, self.idx, self.w, ws_setup)
            B.pack_ragged(setup_dims, self.z, self.idx, self.send_rows, self.send_off, self.slot_of,
                          self.send_count, ws_setup)
            off = self.send_off.cpu().numpy()
            segs[s] = self.send_rows[int(off[r]):int(off[r + 1])].clone()
            if s == r:
                self.own_off = off.astype(np.int64)
        cnt = np.array([segs[s].shape[0] for s in range(R)], dtype=np.int64)
        self.seg_off = np.concatenate([[0], np.cumsum(cnt)])
        self.n_recv = int(self.seg_off[-1])
        self.view_rows = max(-(-self.n_recv // R), 1)
        self.scap = self.view_rows
        self.recv_pools = torch.empty((R * self.view_rows, self.prow), dtype=torch.uint8, device=dev)
        self.recv_pools.view(torch.int32)[self.n_recv:, (L * self.esize) // 4] = -1
        for s in range(R):   # the own segment too: a step copies the same rows again
            if cnt[s]:
                self.recv_pools[self.seg_off[s]:self.seg_off[s + 1]].copy_(segs[s])
        del segs, ws_setup
        self.wave_rows = 0
        if ragged_banks:
            arr = receive_arrivals(shape, exact_fit(shape, self.view_rows, 1), r, self.recv_pools,
                                   self.view_rows * self.prow, dev)
            self.wave_rows = max(int(sum(arr[w * WX:(w + 1) * WX])) for w in range(W))
        self.recv_dims = B.make_dims(self._fit(self.view_rows), my_rank=r, wave_rows=self.wave_rows,
                                     live_waves=self.live_waves)
        assert B.capacity(self.recv_dims)[:2] == (self.view_rows, self.rcap)
        # one workspace and one set of dims for the whole step (moe_pack_ragged
        # ignores the send cap, moe_combine reads the ragged return rows with
        # any cap)
        self.dims = self.recv_dims
        self.ws = self.ws_recv = torch.zeros((B.workspace_size(self.recv_dims),), dtype=torch.uint8, device=dev)
        self.row_src = torch.empty((W, WX, self.rcap), dtype=torch.int32, device=dev)
        self.wave_count = torch.empty((W, WX), dtype=torch.int32, device=dev)
        self.wave_buf = torch.empty((WX, self.rcap, L), dtype=act, device=dev) if gather == "buffer" else None
        self.source_demand = {s: int(cnt[s]) for s in range(R) if s != r}
        if self.full:
            self.w13 = upload(inp["w13"], dev)
            self.w2 = upload(inp["w2"], dev)
            self._quantize_experts(self.recv_dims)
            self.w_up = upload(inp["w_up"], dev)
            self.ws13 = upload(inp["ws13"], dev)
            self.ws2 = upload(inp["ws2"], dev)
            self.ret_send = torch.zeros((R * self.view_rows, L), dtype=act, device=dev)
            self.ret_back = torch.zeros((T * k, L), dtype=act, device=dev)
            fr = upload(inp["foreign_ret"], dev)                 # [R][pool_rows][L]
            own_cnt = np.diff(self.own_off)
            for d in range(R):
                c = int(own_cnt[d])
                if d != r and c:
                    assert c <= fr.shape[1], "foreign_ret has fewer rows than this rank sends"
                    self.ret_back[self.own_off[d]:self.own_off[d] + c].copy_(fr[d, :c])
            del fr
            self.out = torch.empty((T, D), dtype=act, device=dev)
            self._ev_go, self._ev_shared, self._ev_ranked = torch.cuda.Event(), torch.cuda.Event(), torch.cuda.Event()
        torch.cuda.synchronize()

    def dispatch(self, stream=None):
        d, r = self.dims, self.rank
        B.route(d, self.x, self.w_router, self.w_down, self.bias, self.bias_row_tokens, self.logits, self.z,
                self.idx, self.w, self.ws, stream)
        B.pack_ragged(d, self.z, self.idx, self.send_rows, self.send_off, self.slot_of, self.send_count, self.ws,
                      stream)
        # self segment of the dispatch exchange (its place fixed by the count exchange)
        c = int(self.own_off[r + 1] - self.own_off[r])
        if c:
            self.recv_pools[self.seg_off[r]:self.seg_off[r] + c].copy_(
                self.send_rows[self.own_off[r]:self.own_off[r] + c])

    def receive_rank(self, stream=None):
        B.recv_rank(self.recv_dims, self.recv_pools, self.view_rows * self.prow, self.ws_recv, stream)

    def receive_wave(self, w, stream=None):
        B.recv_waves(self.recv_dims, self.recv_pools, self.view_rows * self.prow, w, self.wave_buf, self.row_src[w],
                     self.wave_count[w], self.ws_recv, stream)

    def expert_wave(self, w, stream=None):
        _expert_gemm(self.recv_dims, w, self.wave_buf, self.recv_pools, self.view_rows * self.prow,
                     self.row_src[w], self.wave_count[w], self.w13, self.w2, self.ret_send,
                     self.view_rows * self.shape.latent * self.esize, self.ws_recv, self.ws_mx, stream)

    def combine(self, stream=None):
        r = self.rank
        c = int(self.own_off[r + 1] - self.own_off[r])
        if c:   # self segment of the return exchange
            self.ret_back[self.own_off[r]:self.own_off[r] + c].copy_(self.ret_send[self.seg_off[r]:self.seg_off[r] + c])
        scap = B.capacity(self.dims)[0]
        B.combine(self.dims, self.ret_back, scap * self.shape.latent * self.esize, self.slot_of, self.w, self.w_up,
                  self.ws2, self.out, self.ws, stream)

    def footprint(self):
        """Bytes of the exchange buffers and the workspaces."""
        n = self.send_rows.numel() + self.recv_pools.numel() + self.ws.numel()
        if self.full:
            n += (self.ret_send.numel() + self.ret_back.numel()) * self.esize
            n += 0 if self.ws_mx is None else self.ws_mx.numel()
        return n


def receive_arrivals(shape, fit_shape, rank, recv_pools, src_stride_bytes, device):
    """Rows arriving at each local expert of ``rank`` from the pools in
    ``recv_pools`` (a set-up pass of moe_recv_rank with a small workspace:
    the ranking does not depend on the expert widths or the receive cap)."""
    from dataclasses import replace
    probe = replace(fit_shape, expert_hidden=64, shared_experts=0, shared_hidden=64)
    d = B.make_dims(probe, my_rank=rank, live_waves=1, wave_rows=1)
    ws = torch.zeros((B.workspace_size(d),), dtype=torch.uint8, device=device)
    B.recv_rank(d, recv_pools, src_stride_bytes, ws)
    rep = B.drop_stats(d, ws, raise_on_bad_ids=False)
    return list(rep.expert_arrivals[:shape.local_experts])


class AllRanksLayer:
    """Every rank of a small EP domain on one device (zero-copy exchanges).
    experts="mx": the routed experts as MX-FP4 rows."""

    def __init__(self, shape, inp, device="cuda", gather="fused", experts="act"):
        self.shape, self.device, self.gather = shape, device, gather
        self.experts = _expert_form(experts)
        T, D, L, E, k, R = shape.tokens, shape.d_model, shape.latent, shape.n_experts, shape.top_k, shape.n_ranks
        X, W = shape.local_experts, shape.waves
        WX = X // W
        act = _act(shape)
        dev = device
        self.dims = [B.make_dims(shape, my_rank=r) for r in range(R)]
        self.scap, self.rcap, self.prow = B.capacity(self.dims[0])
        self.x = upload_rank_blocks(inp["x"], dev)                      # [R][T][D]
        self.w_router = upload(inp["w_router"], dev)
        self.w_down = upload(inp["w_down"], dev)
        bias = inp["bias"]
        if bias is not None and bias.ndim == 2:
            bias = np.broadcast_to(bias, (R,) + bias.shape)
        self.bias = None if bias is None else upload_rank_blocks(np.ascontiguousarray(bias, np.float32), dev)
        self.bias_row_tokens = int(inp["bias_row_tokens"])
        self.w13 = upload(inp["w13"], dev)                              # [E][2H][L]
        self.w2 = upload(inp["w2"], dev)                                # [E][L][H]
        self.w_up = upload(inp["w_up"], dev)
        self.ws13 = upload(inp["ws13"], dev)
        self.ws2 = upload(inp["ws2"], dev)
        self.logits = rank_blocks(R, (T, E), torch.float32, dev)
        self.z = torch.empty((R, T, L), dtype=act, device=dev)
        self.idx = torch.empty((R, T, k), dtype=torch.int32, device=dev)
        self.w = torch.empty((R, T, k), dtype=torch.float32, device=dev)
        self.pools = torch.empty((R, R, self.scap, self.prow), dtype=torch.uint8, device=dev)   # [src][dst]
        self.slot_of = torch.empty((R, T, k), dtype=torch.int32, device=dev)
        self.send_count = torch.empty((R, R), dtype=torch.int32, device=dev)
        self.row_src = torch.empty((R, W, WX, self.rcap), dtype=torch.int32, device=dev)
        self.wave_count = torch.empty((R, W, WX), dtype=torch.int32, device=dev)
        # "buffer" gather: one wave buffer per (rank, wave), all kept for inspection
        self.wave_buf = (torch.empty((R, W, WX, self.rcap, L), dtype=act, device=dev) if gather == "buffer"
                         else None)
        self.ret = torch.zeros((R, R, self.scap, L), dtype=act, device=dev)                     # [recv][src]
        self.out = rank_blocks(R, (T, D), act, dev)
        self.ws = [torch.empty((B.workspace_size(self.dims[0]),), dtype=torch.uint8, device=dev)
                   for _ in range(R)]
        self.ws_mx = None   # the ranks run one after the other: one scratch serves them all
        if self.experts == "mx":
            self.w13, self.w2 = mx_quantize(self.w13), mx_quantize(self.w2)
            self.ws_mx = torch.empty((B.mx_workspace_size(self.dims[0]),), dtype=torch.uint8, device=dev)

    def run(self, stream=None):
        sh = self.shape
        R, L = sh.n_ranks, sh.latent
        esize = 2 if sh.act == "bf16" else 4
        pool_bytes = self.scap * self.prow
        for s in range(R):
            d = self.dims[s]
            bias = None if self.bias is None else self.bias[s]
            B.route(d, self.x[s], self.w_router, self.w_down, bias, self.bias_row_tokens, self.logits[s],
                    self.z[s], self.idx[s], self.w[s], self.ws[s], stream)
            B.pack_pools(d, self.z[s], self.idx[s], self.pools[s], pool_bytes, self.slot_of[s],
                         self.send_count[s], self.ws[s], stream)
        X = sh.local_experts
        for r in range(R):
            d = self.dims[r]
            recv_view = self.pools[0, r]                 # pool from source s at + s * R * pool_bytes
            B.recv_rank(d, recv_view, R * pool_bytes, self.ws[r], stream)
            for w in range(sh.waves):
                wb = None if self.wave_buf is None else self.wave_buf[r, w]
                B.recv_waves(d, recv_view, R * pool_bytes, w, wb, self.row_src[r, w],
                             self.wave_count[r, w], self.ws[r], stream)
                _expert_gemm(d, w, wb, recv_view, R * pool_bytes, self.row_src[r, w],
                             self.wave_count[r, w], self.w13[r * X:(r + 1) * X], self.w2[r * X:(r + 1) * X],
                             self.ret[r], self.scap * L * esize, self.ws[r], self.ws_mx, stream)
        for s in range(R):
            d = self.dims[s]
            ret_view = self.ret[0, s]                    # rows from receiver d at + d * R * scap * L
            B.shared_experts(d, self.x[s], self.ws13, self.ws[s], stream)
            B.combine(d, ret_view, R * self.scap * L * esize, self.slot_of[s], self.w[s], self.w_up, self.ws2,
                      self.out[s], self.ws[s], stream)

    def drop_reports(self, stream=None):
        return [B.drop_stats(self.dims[r], self.ws[r], stream, raise_on_bad_ids=False).as_dict()
                for r in range(self.shape.n_ranks)]


def _ceil_div(a, b):
    return -(-a // b)


class RaggedAllRanksLayer:
    """Every rank of a small EP domain on one device with the dropless ragged
    exchange: each rank packs its rows back to back by destination
    (moe_pack_ragged) and nothing is capped on the send side.  The row counts
    are exchanged first (a host read of send_count here); each receiver's
    buffer then holds the segments sent to it laid end to end, source by
    source, viewed by the receive calls as R pools of ceil(n/R) rows with id
    -1 past the n received rows; the return rows go back into each sender's
    ragged order.  The two exchanges are device copies standing for the
    ragged all-to-all.  ``expert_rows`` sizes every expert's bank (the
    receive cap).  ``wave_rows``: 0 keeps a bank of expert_rows hidden rows
    per expert; None lays each wave's hidden rows end to end in one bank sized
    to the rows that receiver's fullest wave keeps (per-expert arrival counts
    at set-up, see RaggedOneRankLayer); a number forces that bank size."""

    def __init__(self, shape, inp, expert_rows, device="cuda", gather="fused", wave_rows=None, experts="act"):
        from workload.configs import exact_fit
        self.experts = _expert_form(experts)
        self.wave_rows_arg = wave_rows
        self.shape, self.device, self.gather = shape, device, gather
        T, D, L, E, k, R = shape.tokens, shape.d_model, shape.latent, shape.n_experts, shape.top_k, shape.n_ranks
        X, W = shape.local_experts, shape.waves
        WX = X // W
        act = _act(shape)
        dev = device
        self.expert_rows = int(expert_rows)
        self._fit = lambda pool_rows: exact_fit(shape, pool_rows, self.expert_rows)
        # send side (route, pack, shared experts, combine): neither cap is used,
        # and cap 1 keeps the receive parts of its workspace small
        self.send_dims = [B.make_dims(exact_fit(shape, 1, 1), my_rank=r) for r in range(R)]
        self.rcap = self.expert_rows
        self.prow = B.capacity(self.send_dims[0])[2]
        self.x = upload_rank_blocks(inp["x"], dev)
        self.w_router = upload(inp["w_router"], dev)
        self.w_down = upload(inp["w_down"], dev)
        bias = inp["bias"]
        if bias is not None and bias.ndim == 2:
            bias = np.broadcast_to(bias, (R,) + bias.shape)
        self.bias = None if bias is None else upload_rank_blocks(np.ascontiguousarray(bias, np.float32), dev)
        self.bias_row_tokens = int(inp["bias_row_tokens"])
        self.w13 = upload(inp["w13"], dev)
        self.w2 = upload(inp["w2"], dev)
        self.w_up = upload(inp["w_up"], dev)
        self.ws13 = upload(inp["ws13"], dev)
        self.ws2 = upload(inp["ws2"], dev)
        self.logits = rank_blocks(R, (T, E), torch.float32, dev)
        self.z = torch.empty((R, T, L), dtype=act, device=dev)
        self.idx = torch.empty((R, T, k), dtype=torch.int32, device=dev)
        self.w = torch.empty((R, T, k), dtype=torch.float32, device=dev)
        self.send_rows = torch.empty((R, T * k, self.prow), dtype=torch.uint8, device=dev)
        self.send_off = torch.empty((R, R + 1), dtype=torch.int32, device=dev)
        self.slot_of = torch.empty((R, T, k), dtype=torch.int32, device=dev)
        self.send_count = torch.empty((R, R), dtype=torch.int32, device=dev)
        self.ret_back = torch.zeros((R, T * k, L), dtype=act, device=dev)   # returned rows, sender's order
        self.row_src = torch.empty((R, W, WX, self.rcap), dtype=torch.int32, device=dev)
        self.wave_count = torch.empty((R, W, WX), dtype=torch.int32, device=dev)
        self.wave_buf = torch.empty((WX, self.rcap, L), dtype=act, device=dev) if gather == "buffer" else None
        self.out = rank_blocks(R, (T, D), act, dev)
        self.ws_send = [torch.zeros((B.workspace_size(d),), dtype=torch.uint8, device=dev) for d in self.send_dims]
        self.recv_dims, self.recv, self.ret, self.ws_recv, self.seg_off = [], [], [], [], []
        if self.experts == "mx":
            self.w13, self.w2 = mx_quantize(self.w13), mx_quantize(self.w2)

    def run(self, stream=None):
        sh = self.shape
        R, L, X = sh.n_ranks, sh.latent, sh.local_experts
        esize = 2 if sh.act == "bf16" else 4
        for s in range(R):
            d = self.send_dims[s]
            bias = None if self.bias is None else self.bias[s]
            B.route(d, self.x[s], self.w_router, self.w_down, bias, self.bias_row_tokens, self.logits[s],
                    self.z[s], self.idx[s], self.w[s], self.ws_send[s], stream)
            B.pack_ragged(d, self.z[s], self.idx[s], self.send_rows[s], self.send_off[s], self.slot_of[s],
                          self.send_count[s], self.ws_send[s], stream)
        # the count exchange
        torch.cuda.synchronize()
        cnt = self.send_count.cpu().numpy().astype(np.int64)      # [src][dst]
        off = self.send_off.cpu().numpy().astype(np.int64)        # [src][R+1]
        self.recv_dims, self.recv, self.ret, self.ws_recv, self.seg_off = [], [], [], [], []
        id_col = (L * esize) // 4
        for r in range(R):
            n = int(cnt[:, r].sum())
            view_rows = max(_ceil_div(n, R), 1)
            seg = np.concatenate([[0], np.cumsum(cnt[:, r])])
            buf = torch.empty((R * view_rows, self.prow), dtype=torch.uint8, device=self.device)
            buf.view(torch.int32)[n:, id_col] = -1
            for s in range(R):                                  # the dispatch exchange
                c = int(cnt[s, r])
                if c:
                    buf[seg[s]:seg[s] + c].copy_(self.send_rows[s, off[s, r]:off[s, r] + c])
            wave_rows = self.wave_rows_arg
            if wave_rows is None:
                arr = receive_arrivals(sh, self._fit(view_rows), r, buf, view_rows * self.prow, self.device)
                WX = X // sh.waves
                wave_rows = max(int(sum(arr[w * WX:(w + 1) * WX])) for w in range(sh.waves))
            d = B.make_dims(self._fit(view_rows), my_rank=r, wave_rows=wave_rows)
            assert B.capacity(d)[:2] == (view_rows, self.rcap)
            ws = torch.zeros((B.workspace_size(d),), dtype=torch.uint8, device=self.device)
            ws_mx = (torch.empty((B.mx_workspace_size(d),), dtype=torch.uint8, device=self.device)
                     if self.experts == "mx" else None)
            ret = torch.zeros((R * view_rows, L), dtype=self.out.dtype, device=self.device)
            pool_bytes = view_rows * self.prow
            B.recv_rank(d, buf, pool_bytes, ws, stream)
            for w in range(sh.waves):
                B.recv_waves(d, buf, pool_bytes, w, self.wave_buf, self.row_src[r, w], self.wave_count[r, w], ws,
                             stream)
                _expert_gemm(d, w, self.wave_buf, buf, pool_bytes, self.row_src[r, w], self.wave_count[r, w],
                             self.w13[r * X:(r + 1) * X], self.w2[r * X:(r + 1) * X], ret, view_rows * L * esize,
                             ws, ws_mx, stream)
            for s in range(R):                                  # the return exchange
                c = int(cnt[s, r])
                if c:
                    self.ret_back[s, off[s, r]:off[s, r] + c].copy_(ret[seg[s]:seg[s] + c])
            self.recv_dims.append(d)
            self.recv.append(buf)
            self.ret.append(ret)
            self.ws_recv.append(ws)
            self.seg_off.append(seg)
        for s in range(R):
            d = self.send_dims[s]
            B.shared_experts(d, self.x[s], self.ws13, self.ws_send[s], stream)
            scap = B.capacity(d)[0]
            B.combine(d, self.ret_back[s], scap * L * esize, self.slot_of[s], self.w[s], self.w_up, self.ws2,
                      self.out[s], self.ws_send[s], stream)

    def drop_reports(self, stream=None):
        """Send fields from each rank's dispatch, receive fields from its receive."""
        out = []
        for r in range(self.shape.n_ranks):
            snd = B.drop_stats(self.send_dims[r], self.ws_send[r], stream, raise_on_bad_ids=False).as_dict()
            rcv = B.drop_stats(self.recv_dims[r], self.ws_recv[r], stream, raise_on_bad_ids=False).as_dict()
            for key in ("recv_arrivals", "recv_kept", "recv_dropped", "recv_bad_ids", "expert_arrivals",
                        "expert_kept"):
                snd[key] = rcv[key]
            out.append(snd)
        return out


# ---------------------------------------------------------------- MX-FP4 rows

_DTYPE = {torch.bfloat16: B.MOE_ACT_BF16, torch.float32: B.MOE_ACT_F32}


_HERE = contextlib.nullcontext()
# the raw handle of a device's current stream, without a Stream object around it (1 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on(t):
    """(stream handle, device guard) for work on tensor t: its device's current stream."""
    if not t.is_cuda:
        raise ValueError("the library works on GPU tensors")
    index = t.get_device()
    stream = _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream
    # a guard costs as much as a launch: only where the device is not the current one
    return stream, _HERE if index == torch.cuda.current_device() else torch.cuda.device(index)


def _mx_strides(cols):
    """B.mx_strides without the call (it also refuses what that refuses)."""
    if cols <= 0 or cols % 32 or cols > 1 << 24:
        return B.mx_strides(cols)
    return cols // 2, (cols // 32 + 15) // 16 * 16


def _row_stride(t, what):
    """Elements from row to row of t [..., rows, cols], whose rows must be evenly spaced and contiguous."""
    if t.dim() >= 2 and t.is_contiguous():
        return max(t.shape[-1], 1)
    if t.dim() < 2 or t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{what}: rows of contiguous values are needed")
    if t.dim() == 2:
        return t.stride(0)
    stride = None
    rows = 1
    for size, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size > 1:
            if stride is None:
                if st % rows:
                    raise ValueError(f"{what}: its rows are not evenly spaced")
                stride = st // rows
            elif st != stride * rows:
                raise ValueError(f"{what}: its rows are not evenly spaced")
        rows *= size
    return t.shape[-1] if stride is None else stride


class MxRows:
    """Rows of `cols` MX-FP4 values on the GPU (include/moe.h describes the format):
    codes [..., rows, cols / 2] and scales [..., rows, cols / 32 rounded up to 16], uint8."""

    def __init__(self, codes, scales, cols):
        self._codes, self._scales, self.cols = codes, scales, cols
        self._layout()

    @classmethod
    def _made(cls, codes, scales, cols, code_stride, scale_stride, at):
        """From contiguous tensors made here, which are at the addresses `at`."""
        q = cls.__new__(cls)
        q._codes, q._scales, q.cols = codes, scales, cols
        q.code_stride, q.scale_stride, q._at, q._arg = code_stride, scale_stride, at, None
        return q

    @property
    def codes(self):
        return self._codes

    @codes.setter
    def codes(self, t):
        self._codes, self._at = t, None   # checked at the next use

    @property
    def scales(self):
        return self._scales

    @scales.setter
    def scales(self, t):
        self._scales, self._at = t, None

    def _layout(self):
        """Checks the tensors and takes their strides."""
        codes, scales = self._codes, self._scales
        cb, sb = _mx_strides(self.cols)
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("codes and scales are uint8")
        if codes.shape[:-1] != scales.shape[:-1] or codes.shape[-1] != cb or scales.shape[-1] < sb:
            raise ValueError(f"codes {tuple(codes.shape)} and scales {tuple(scales.shape)} are not rows of {self.cols} "
                             "values")
        if codes.device != scales.device:
            raise ValueError("codes and scales are on different devices")
        self.code_stride, self.scale_stride = _row_stride(codes, "codes"), _row_stride(scales, "scales")
        self._at, self._arg = (codes.data_ptr(), scales.data_ptr()), None

    def __getstate__(self):
        return {**self.__dict__, "_arg": None}   # ctypes pointers do not go into copies

    def _where(self):
        """The tensors' addresses now; memory put in their place since the last call is checked first."""
        at = (self._codes.data_ptr(), self._scales.data_ptr())
        if at != self._at:
            self._layout()
        return at

    @property
    def arg(self):
        """moe_mx_rows of the tensors as they are now."""
        at, arg = self._where(), self._arg
        if arg is None:
            arg = self._arg = B.MxRowsArg(at[0], at[1], self.code_stride, self.scale_stride)
        return arg

    @property
    def shape(self):
        return tuple(self.codes.shape[:-1]) + (self.cols,)

    @property
    def rows(self):
        n = 1
        for s in self.codes.shape[:-1]:
            n *= s
        return n

    def __getitem__(self, i):
        """A part along the leading dimension(s), as of the tensors."""
        return MxRows(self.codes[i], self.scales[i], self.cols)


def mx_quantize(x):
    """x [..., rows, cols] (bf16 or fp32, evenly spaced rows) as MxRows."""
    code = _DTYPE.get(x.dtype)
    if code is None:
        raise TypeError(f"mx_quantize takes bf16 or fp32, not {x.dtype}")
    st, dev = _on(x)
    ld = _row_stride(x, "x")
    lead, cols = x.shape[:-1], x.shape[-1]
    cb, sb = _mx_strides(cols)
    with dev:
        codes = torch.empty(lead + (cb,), dtype=torch.uint8, device=x.device)
        scales = torch.empty(lead + (sb,), dtype=torch.uint8, device=x.device)
        at = (codes.data_ptr(), scales.data_ptr())
        B.mx_quantize(code, x.numel() // cols, cols, x, ld * x.element_size(), at[0], cb, at[1], sb, st)
    return MxRows._made(codes, scales, cols, cb, sb, at)


def mx_dequantize(q, dtype=torch.bfloat16):
    """The values of MxRows q as a bf16 or fp32 tensor."""
    code = _DTYPE.get(dtype)
    if code is None:
        raise TypeError(f"mx_dequantize gives bf16 or fp32, not {dtype}")
    st, dev = _on(q.codes)
    with dev:
        out = torch.empty(q.codes.shape[:-1] + (q.cols,), dtype=dtype, device=q.codes.device)
        at = q._where()
        B.mx_dequantize(code, out.numel() // q.cols, q.cols, at[0], q.code_stride, at[1], q.scale_stride, out,
                        q.cols * out.element_size(), st)
    return out


def mx_gemm(a, b, counts=None, out=None, dtype=torch.bfloat16):
    """out[g] = a[g] . b[g]^T of MxRows a [G, M, K] and b [G, N, K] (or [M, K] and
    [N, K]) as bf16 or fp32.  counts: int32 [G] rows of each group (the rows of
    `out` behind them are left as they were)."""
    ca, cb = a.codes, b.codes
    sa, sb = ca.shape, cb.shape
    if len(sa) != len(sb) or len(sa) not in (2, 3) or a.cols != b.cols or sa[:-2] != sb[:-2]:
        raise ValueError(f"mx_gemm of rows {a.shape} and {b.shape}")
    G = sa[0] if len(sa) == 3 else 1
    M, N = sa[-2], sb[-2]
    st, dev = _on(ca)
    shape = sa[:-1] + (N,)
    with dev:
        if out is None:
            out = (torch.empty if counts is None else torch.zeros)(shape, dtype=dtype, device=ca.device)
        code = _DTYPE.get(out.dtype)
        if out.shape != shape or code is None:
            raise ValueError(f"out {tuple(out.shape)} {out.dtype}, expected {tuple(shape)} bf16 or fp32")
        if counts is not None and (counts.dtype != torch.int32 or counts.shape != (G,) or not counts.is_contiguous()):
            raise ValueError("counts is a contiguous int32 tensor with one value a group")
        if cb.device != ca.device or out.device != ca.device or counts is not None and counts.device != ca.device:
            raise ValueError("mx_gemm: tensors on different devices")
        B.mx_gemm(code, G, M, N, a.cols, a.arg, counts, b.arg, out, _row_stride(out, "out") * out.element_size(), st)
    return out


class FewTokenLayer:
    """A whole layer for up to 64 tokens at a time on one GPU (moe_few_tokens), as a
    decode step runs it: __call__(x [T, D]) -> (out [T, D], topk_idx [T, k] int32,
    topk_w [T, k] fp32).  Forward only.  Weights, x and out start 16-byte aligned.

    Activations keep two bf16 parts (2^-17) with bf16 and MX-FP4 weights; the wave
    path's MX-FP4 products (experts="mx" above) round them to 4 bits, so the two differ
    by that on the same weights.

    w_router [E, D], w_down [L, D], w_up [D, L], ws13 [S, 2 HS, D], ws2 [S, D, HS]
    are bf16 or fp32, as x; the routed experts w13 [X, 2H, L] and w2 [X, L, H] too,
    or MxRows of those shapes (bf16 layers).  ws13 = ws2 = None (or S = 0): no
    shared experts.  bias: fp32 [E], or [nb, E] of which row t // bias_row_tokens
    serves token t.  With n_ranks > 1 this rank holds X = E / n_ranks experts and
    `out` is its share of the sum over the ranks.

    The weights are read where they are at each call: values changed in place and
    memory put in a tensor's place (w.data = ..., or an attribute of the layer set)
    count from the next call on, but for graphs captured before; sizes and types stay.

    Calls may come from any stream and any thread, and may be captured.  The layer
    keeps its weights and one workspace, for eager calls on the stream that was
    current when it was made; a call on another stream, or one that is being
    captured, takes a workspace of its own from torch's allocator (a graph's lies
    in its memory pool), so that calls that run at once share nothing.
    """

    def __init__(self, w_router, w_down, w13, w2, w_up, ws13=None, ws2=None, bias=None, bias_row_tokens=0, top_k=1,
                 n_ranks=1, rank=0):
        self.w_router, self.w_down, self.w13, self.w2, self.w_up = w_router, w_down, w13, w2, w_up
        if (ws13 is None) != (ws2 is None) or ws13 is not None and ws13.shape[0] != ws2.shape[0]:
            raise ValueError("ws13 and ws2 go together, with as many shared experts each")
        self.ws13, self.ws2 = (ws13, ws2) if ws13 is not None and ws13.shape[0] else (None, None)
        self.bias, self.bias_row_tokens, self.n_ranks = bias, int(bias_row_tokens), n_ranks
        self._made_of = E, D, L, H, S, HS, dt, dev, _ = self._sizes()
        self.dims = B.Dims(tokens=B.MOE_FEW_TOKENS_MAX, d_model=D, latent=L, n_experts=E, top_k=top_k, n_ranks=n_ranks,
                           waves=1, expert_hidden=H, shared_experts=S, shared_hidden=HS, my_rank=rank,
                           act_dtype=_DTYPE[dt], send_num=1, send_den=1, recv_num=1, recv_den=1)
        self._prepare()

    def _prepare(self):
        """What a layer object has to itself, beside its weights and sizes."""
        dev = self.w_router.device
        self._by_tokens = {}   # the dims of each batch size met; self.dims are those of the largest
        self.ws = torch.empty((B.few_workspace_size(self.dims),), dtype=torch.uint8, device=dev)
        self._ws_stream = _on(self.ws)[0] if dev.type == "cuda" else None
        self._ws_lock = threading.Lock()   # a call launches several kernels: those of two threads must not mix
        self._at = self._addresses()

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name in ("w_router", "w_down", "w13", "w2", "w_up", "ws13", "ws2", "bias", "bias_row_tokens", "n_ranks"):
            self.__dict__["_at"] = None   # checked at the next call, which the address alone might not ask for

    def __getstate__(self):
        own = ("_by_tokens", "ws", "_ws_stream", "_ws_lock", "_at")
        return {k: v for k, v in self.__dict__.items() if k not in own}

    def __setstate__(self, state):
        self.__dict__.update(state)
        self._made_of = self._sizes()
        self._prepare()

    def _sizes(self):
        """Checks the weights and gives what a call takes for granted of them."""
        w_router, w_down, w13, w2, ws13, bias = self.w_router, self.w_down, self.w13, self.w2, self.ws13, self.bias
        dt, dev, n_ranks = w_router.dtype, w_router.device, self.n_ranks
        if dt not in _DTYPE:
            raise TypeError(f"weights are bf16 or fp32, not {dt}")
        if w_router.dim() != 2 or w_down.dim() != 2:
            raise ValueError("w_router is [E, D] and w_down [L, D]")
        E, D = w_router.shape
        L = w_down.shape[0]
        S = 0 if ws13 is None else ws13.shape[0]
        HS = ws13.shape[1] // 2 if S else 64
        if len(w13.shape) != 3 or n_ranks < 1 or E % n_ranks:
            raise ValueError("w13 is [E / n_ranks, 2 H, L]")
        X, H = E // n_ranks, w13.shape[1] // 2
        mx = isinstance(w13, MxRows)
        if mx != isinstance(w2, MxRows):
            raise TypeError("w13 and w2 are both MxRows, or neither")
        if mx and dt != torch.bfloat16:
            raise TypeError("MxRows as experts need bf16 weights beside them")
        want = {"w_router": (w_router, (E, D)), "w_down": (w_down, (L, D)), "w_up": (self.w_up, (D, L)),
                "w13": (w13, (X, 2 * H, L)), "w2": (w2, (X, L, H))}
        if S:
            want |= {"ws13": (ws13, (S, 2 * HS, D)), "ws2": (self.ws2, (S, D, HS))}
        bias_tokens = B.MOE_FEW_TOKENS_MAX   # that the bias serves
        if bias is not None:
            if bias.dtype != torch.float32 or bias.dim() not in (1, 2) or (bias.dim() == 2) != (self.bias_row_tokens > 0):
                raise ValueError("bias is fp32 [E], or [nb, E] with bias_row_tokens > 0")
            want["bias"] = (bias, tuple(bias.shape[:-1]) + (E,))
            if bias.dim() == 2:
                bias_tokens = bias.shape[0] * self.bias_row_tokens
        for name, (t, shape) in want.items():
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
            if isinstance(t, MxRows):
                t._layout()
            parts = [t.codes, t.scales] if isinstance(t, MxRows) else [t]
            for p in parts:
                if p.device != dev or not p.is_contiguous():
                    raise ValueError(f"{name} must be contiguous and on {dev}")
            if name != "bias" and not isinstance(t, MxRows) and t.dtype != dt:
                raise TypeError(f"{name} is {t.dtype}, not {dt}")
            if isinstance(t, MxRows) and t.scales.shape[-1] != B.mx_strides(t.cols)[1]:
                raise ValueError(f"{name}: scale rows at their smallest stride are needed")
        return E, D, L, H, S, HS, dt, dev, (mx, bias_tokens)

    def _addresses(self):
        """The weights as moe_few_tokens takes them."""
        w13, w2, bias, ws13 = self.w13, self.w2, self.bias, self.ws13
        experts = ((w13.codes.data_ptr(), w13.scales.data_ptr(), w2.codes.data_ptr(), w2.scales.data_ptr())
                   if isinstance(w13, MxRows) else (w13.data_ptr(), None, w2.data_ptr(), None))
        shared = (None, None) if ws13 is None else (ws13.data_ptr(), self.ws2.data_ptr())
        return (self.w_router.data_ptr(), self.w_down.data_ptr(), None if bias is None else bias.data_ptr(),
                self.bias_row_tokens, *experts, self.w_up.data_ptr(), *shared)

    def __call__(self, x, out=None):
        T, k = x.shape[0], self.dims.top_k
        if x.dim() != 2 or x.shape[1] != self.dims.d_model or x.dtype != self.w_router.dtype or not x.is_contiguous():
            raise ValueError(f"x {tuple(x.shape)} {x.dtype}: contiguous rows of {self.dims.d_model} "
                             f"{self.w_router.dtype} values are needed")
        if x.device != self.w_router.device:
            raise ValueError("x is on another device than the layer")
        if T > self._made_of[-1][1]:
            raise ValueError(f"{T} tokens are more than the layer (or its bias) takes")
        if out is not None and (out.shape != x.shape or out.dtype != x.dtype or not out.is_contiguous()
                                or out.device != x.device):
            raise ValueError("out must be like x")
        at = self._addresses()
        if at != self._at:   # memory put in a weight's place since the last call
            if self._sizes() != self._made_of:
                raise ValueError("the weights' sizes or types are not those the layer was made with")
            self._at = at
        st, dev = _on(x)
        with dev:
            if out is None:
                out = torch.empty_like(x)
            idx = torch.empty((T, k), dtype=torch.int32, device=x.device)
            w = torch.empty((T, k), dtype=torch.float32, device=x.device)
            dims = self._by_tokens.get(T)
            if dims is None:
                dims = B.Dims.from_buffer_copy(self.dims)
                dims.tokens = T
                self._by_tokens[T] = dims
            args = (dims, x.data_ptr(), *at, idx, w, out)
            # the default stream (0) cannot be captured
            if st == self._ws_stream and not (st and torch.cuda.is_current_stream_capturing()):
                with self._ws_lock:
                    B.few_tokens(*args, self.ws, st)
            else:
                B.few_tokens(*args, torch.empty_like(self.ws), st)
        return out, idx, w
