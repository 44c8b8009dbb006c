"""Device-buffer owner for the compression + decode path.

`Compressor` allocates (with torch) every output and workspace the four C-ABI
calls need, builds the RoPE tables with `kvc_rope_table`, and runs
kvc_score -> kvc_select -> kvc_merge_pack and kvc_decode_attn steps.  It only
allocates and marshals; all arithmetic runs in libkvc's kernels.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence

import numpy as np
import torch

from . import kvc

TORCH_DT = {kvc.KVC_BF16: torch.bfloat16, kvc.KVC_F32: torch.float32}


def packed_capacity(p: kvc.kvc_params, ctx_len: Sequence[int]) -> int:
    """Rows the packed cache needs at most: every sequence's budget (at least its
    window) plus the decode reserve of every (b, l, h)."""
    LH = p.L * p.H
    rows = 0
    for n in ctx_len:
        per = p.budget_entries_per_lh if p.budget_entries_per_lh > 0 else math.floor(p.budget_ratio * n)
        rows += max(per, p.W) * LH + LH * p.decode_reserve
    return int(rows)


# ---------------------------------------------------------------- packed-cache files
PACKED_FORMAT = 1
_PACKED_ARRAYS = ("Kp", "Vp", "logm", "pos", "len_lh", "cap_lh", "off_lh")


def write_packed(path: str, p: kvc.kvc_params, tensors: dict) -> None:
    """Writes a packed cache to an .npz file: the parameter block's scalar
    fields, and Kp, Vp, logm, pos (the first sum(cap_lh) rows, i.e. every
    (b, l, h)'s entries and its decode reserve) with len_lh, cap_lh and
    off_lh.  bf16 rows are stored as their uint16 bit patterns, so a reload is
    bit for bit.  Tensors may live on any device."""
    rows = int(tensors["cap_lh"].to(torch.int64).sum())
    out = {"format": np.int64(PACKED_FORMAT)}
    for name, ctype in p._fields_:
        if name == "tree_cuts":                      # a pointer: not part of the cache
            continue
        out["param_" + name] = np.asarray(getattr(p, name))
    for name in _PACKED_ARRAYS:
        t = tensors[name].detach()
        if name in ("Kp", "Vp", "logm", "pos"):
            t = t[:rows]
        t = t.cpu().contiguous()
        if t.dtype == torch.bfloat16:
            out[name + "_bf16bits"] = t.view(torch.int16).numpy()
        else:
            out[name] = t.numpy()
    np.savez(path, **out)


def read_packed(path: str):
    """(params dict, tensors dict on the CPU) of a file written by write_packed."""
    with np.load(path) as z:
        if int(z["format"]) != PACKED_FORMAT:
            raise ValueError(f"{path}: packed-cache format {int(z['format'])}, expected {PACKED_FORMAT}")
        params = {k[len("param_"):]: z[k].item() for k in z.files if k.startswith("param_")}
        tensors = {}
        for name in _PACKED_ARRAYS:
            if name + "_bf16bits" in z.files:
                tensors[name] = torch.from_numpy(z[name + "_bf16bits"].copy()).view(torch.bfloat16)
            else:
                tensors[name] = torch.from_numpy(z[name].copy())
    return params, tensors


class Compressor:
    def __init__(self, p: kvc.kvc_params, ctx_len: Sequence[int], device="cuda",
                 tensor_cores: bool = True, tree_cuts: bool = False, salient: bool = False):
        """tree_cuts=True: every scoring call first runs kvc_tree_cuts, and
        scoring, selection and packing use those curvature-chosen trees
        (p.tree_cuts points at this object's cut table); otherwise the
        midpoint trees.  salient=True: the depth-2 nodes may isolate their most
        relevant token in a three-way child set (kvc_params.salient_extract);
        kvc_score records the choice in the cut table, which is reset to the
        binary cuts (kvc_tree_cuts, or zeros for midpoint trees) before every
        scoring call."""
        self.p = p
        self.device = device
        self.ctx_host = [int(n) for n in ctx_len]
        # the tensor-core scoring passes need the exact extent of K
        p.total_ctx = sum(self.ctx_host) if tensor_cores else 0
        assert len(self.ctx_host) == p.B and max(self.ctx_host) <= p.n_max
        B, L, H, R, S = p.B, p.L, p.H, p.G * p.P, p.S_max
        rows = sum(L * H * n for n in self.ctx_host)
        dt = TORCH_DT[p.dtype]
        f32, i32 = torch.float32, torch.int32
        z = dict(device=device)
        self.ctx_len = torch.tensor(self.ctx_host, dtype=i32, **z)
        n_half = 2 * p.n_max
        self.rope_cos = torch.empty((n_half, p.d // 2), dtype=f32, **z)
        self.rope_sin = torch.empty((n_half, p.d // 2), dtype=f32, **z)
        kvc.kvc_rope_table(p.d, p.rope_base, n_half, self.rope_cos, self.rope_sin)
        self.lse = torch.empty((B, L, H, R), dtype=f32, **z)
        self.feats = torch.empty((rows, 5), dtype=f32, **z)
        self.relevance = torch.empty((rows,), dtype=f32, **z)
        self.op_util = torch.empty((B, L, H, S, 16), dtype=f32, **z)
        self.op_cost = torch.empty((B, L, H, S, 16), dtype=i32, **z)
        self.taken = torch.empty((B, L, H, S, 16), dtype=torch.uint8, **z)
        self.len_lh = torch.empty((B, L, H), dtype=i32, **z)
        self.cap_lh = torch.empty((B, L, H), dtype=i32, **z)
        self.off_lh = torch.empty((B, L, H), dtype=torch.int64, **z)
        self.total = torch.empty((1,), dtype=torch.int64, **z)
        cap = packed_capacity(p, self.ctx_host)
        # the tensor-core decode needs the extent of the packed cache
        p.packed_rows = cap if tensor_cores else 0
        # zeros: packed-cache files hold the rows of the decode reserve too, which no call
        # writes before they are appended to; nothing of what the memory held before gets in
        self.Kp = torch.zeros((cap, p.d), dtype=dt, **z)
        self.Vp = torch.zeros((cap, p.d), dtype=dt, **z)
        self.logm = torch.zeros((cap,), dtype=f32, **z)
        self.pos = torch.zeros((cap,), dtype=f32, **z)
        self.ws_score = kvc.workspace(kvc.KVC_WS_SCORE, p, device)
        self.ws_select = kvc.workspace(kvc.KVC_WS_SELECT, p, device)
        self.ws_pack = kvc.workspace(kvc.KVC_WS_PACK, p, device)
        self.ws_decode = kvc.workspace(kvc.KVC_WS_DECODE, p, device, zero=True)
        self.tree_kappa = torch.empty((rows,), dtype=f32, **z) if tree_cuts else None
        self.curvature_trees = bool(tree_cuts)
        self.cuts = (torch.zeros((B, L, H, S, 8), dtype=torch.uint8, **z)
                     if (tree_cuts or salient) else None)
        p.tree_cuts = self.cuts.data_ptr() if self.cuts is not None else None
        p.salient_extract = 1 if salient else 0
        self._graphs = {}
        self._ws_chunk = None
        self._ws_outgrown = []                       # calls in flight or captured may still use them

    # ---------------------------------------------------------------- calls
    # With graph=True a call is captured into a CUDA graph once per set of
    # buffers and replayed on the current stream (the library launches many
    # small kernels per call); the last replay's kernel count is kept in
    # `graph_launches`.
    def _graphed(self, key, fn):
        g = self._graphs.get(key)
        if g is None:
            dev = self.Kp.device
            kvc.kvc_device_error()                   # error-word lookup outside capture
            side = torch.cuda.Stream(device=dev)
            side.wait_stream(torch.cuda.current_stream(dev))
            graph = torch.cuda.CUDAGraph()
            n0 = kvc.kvc_launch_count()
            with torch.cuda.graph(graph, stream=side):
                fn(side)
            torch.cuda.current_stream(dev).wait_stream(side)
            g = (graph, kvc.kvc_launch_count() - n0)
            self._graphs[key] = g
        g[0].replay()
        self.graph_launches = g[1]

    @staticmethod
    def _key(name, *tensors):
        return (name,) + tuple(t.data_ptr() if t is not None else 0 for t in tensors)

    def score(self, K, V, Qp, slot_bounds, n_slots, head_sens=None, stream=None, graph=False):
        def run(st):
            if self.curvature_trees:
                kvc.kvc_tree_cuts(self.p, self.ctx_len, K, self.rope_cos, self.rope_sin,
                                  slot_bounds, n_slots, self.tree_kappa, self.cuts, st)
            elif self.cuts is not None:              # midpoint trees: an all-zero table
                with torch.cuda.stream(torch.cuda.current_stream() if st is None else st):
                    self.cuts.zero_()
            kvc.kvc_score(self.p, self.ctx_len, K, V, Qp, self.rope_cos, self.rope_sin,
                          slot_bounds, n_slots, head_sens, self.lse, self.feats, self.relevance,
                          self.op_util, self.op_cost, self.ws_score, st)
        if graph:
            self._graphed(self._key("score", K, V, Qp, slot_bounds, n_slots, head_sens), run)
        else:
            run(stream)

    def select(self, slot_bounds, n_slots, head_sens=None, op_util=None, relevance=None,
               stream=None, graph=False):
        rel = self.relevance if relevance is None else relevance
        util = self.op_util if op_util is None else op_util

        def run(st):
            kvc.kvc_select(self.p, self.ctx_len, slot_bounds, n_slots, rel, head_sens, util,
                           self.op_cost, self.taken, self.len_lh, self.cap_lh, self.off_lh,
                           self.total, self.ws_select, st)
        if graph:
            self._graphed(self._key("select", slot_bounds, n_slots, head_sens, rel, util), run)
        else:
            run(stream)

    def merge_pack(self, K, V, slot_bounds, n_slots, taken=None, stream=None, graph=False):
        tk = self.taken if taken is None else taken

        def run(st):
            kvc.kvc_merge_pack(self.p, self.ctx_len, K, V, self.relevance, self.rope_cos,
                               self.rope_sin, slot_bounds, n_slots, tk, self.len_lh, self.off_lh,
                               self.Kp, self.Vp, self.logm, self.pos, self.ws_pack, st)
        if graph:
            self._graphed(self._key("pack", K, V, slot_bounds, n_slots, tk), run)
        else:
            run(stream)

    def compress(self, K, V, Qp, slot_bounds, n_slots, head_sens=None, stream=None, graph=False):
        self.score(K, V, Qp, slot_bounds, n_slots, head_sens, stream, graph)
        self.select(slot_bounds, n_slots, head_sens, stream=stream, graph=graph)
        self.merge_pack(K, V, slot_bounds, n_slots, stream=stream, graph=graph)

    def compress_from_host(self, h_K, h_V, h_Qp, K, V, Qp, slot_bounds, n_slots,
                           head_sens=None, chunks: int = 4, copy_stream=None, graph=False):
        """Batch 1, inputs in pinned host memory: copies K, V and the probes into the
        device buffers K, V, Qp one layer chunk at a time on `copy_stream` while the
        chunks already on the device are scored on the current stream (scoring has
        no coupling across layers; the budget couples them only in select), then
        selects and packs (as graph replays with graph=True).  The first chunk is
        about half the size of the others, so less of the copy is exposed.  Same
        results as copying everything, then compress().  Copies the caller queues
        on `copy_stream` afterwards run behind the chunks."""
        p = self.p
        if p.B != 1:
            raise ValueError("compress_from_host copies layer chunks of one sequence")
        L, H, n = p.L, p.H, self.ctx_host[0]
        dev = K.device
        cur = torch.cuda.current_stream(dev)
        cs = copy_stream if copy_stream is not None else torch.cuda.Stream(device=dev)
        cs.wait_stream(cur)                          # the buffers are free to overwrite
        # a small first chunk, so scoring starts early; the rest in equal parts
        chunks = max(1, min(chunks, L))
        first = max(1, -(-L // (2 * chunks))) if chunks > 1 else L
        cuts = [0] + [first + round(c * (L - first) / (chunks - 1)) for c in range(chunks)] \
            if chunks > 1 else [0, L]
        events = []
        for c in range(chunks):
            l0, l1 = cuts[c], cuts[c + 1]
            r0, r1 = l0 * H * n, l1 * H * n
            with torch.cuda.stream(cs):
                K[r0:r1].copy_(h_K[r0:r1], non_blocking=True)
                V[r0:r1].copy_(h_V[r0:r1], non_blocking=True)
                Qp[:, l0:l1].copy_(h_Qp[:, l0:l1], non_blocking=True)
                ev = torch.cuda.Event()
                ev.record(cs)
            events.append(ev)
        for c in range(chunks):
            l0, l1 = cuts[c], cuts[c + 1]
            if l1 == l0:
                continue
            r0, r1 = l0 * H * n, l1 * H * n
            cur.wait_event(events[c])
            pc = kvc.kvc_params.from_buffer_copy(p)
            pc.L = l1 - l0
            if self.cuts is not None and not self.curvature_trees:
                pc.tree_cuts = self.cuts[:, l0:l1].data_ptr()
                with torch.cuda.stream(cur):
                    self.cuts[:, l0:l1].zero_()
            if self.curvature_trees:
                pc.tree_cuts = self.cuts[:, l0:l1].data_ptr()
                kvc.kvc_tree_cuts(pc, self.ctx_len, K[r0:r1], self.rope_cos, self.rope_sin,
                                  slot_bounds, n_slots, self.tree_kappa[r0:r1],
                                  self.cuts[:, l0:l1], cur)
            kvc.kvc_score(pc, self.ctx_len, K[r0:r1], V[r0:r1], Qp[:, l0:l1], self.rope_cos,
                          self.rope_sin, slot_bounds, n_slots,
                          None if head_sens is None else head_sens[l0:l1], self.lse[:, l0:l1],
                          self.feats[r0:r1], self.relevance[r0:r1], self.op_util[:, l0:l1],
                          self.op_cost[:, l0:l1], self.ws_score, cur)
        self.select(slot_bounds, n_slots, head_sens, graph=graph)
        self.merge_pack(K, V, slot_bounds, n_slots, graph=graph)

    # ---------------------------------------------------------------- packed-cache files
    def save_packed(self, path: str) -> None:
        """Writes this object's packed cache (after kvc_merge_pack and any
        decode steps) to an .npz file (write_packed)."""
        torch.cuda.synchronize(self.Kp.device)
        write_packed(path, self.p, {n: getattr(self, n) for n in _PACKED_ARRAYS})

    def load_packed(self, path: str) -> None:
        """Replaces this object's packed cache with a saved one, so decoding
        resumes where the saving process stopped.  The file's shape fields
        (B, L, H, G, d, dtype) must match this object's and its rows must fit
        the packed buffers."""
        params, t = read_packed(path)
        for k in ("B", "L", "H", "G", "d", "dtype"):
            if params[k] != getattr(self.p, k):
                raise ValueError(f"{path}: {k} = {params[k]}, this cache has {getattr(self.p, k)}")
        rows = t["Kp"].shape[0]
        if rows > self.Kp.shape[0]:
            raise ValueError(f"{path}: {rows} rows, the packed buffers hold {self.Kp.shape[0]}")
        for n in ("Kp", "Vp", "logm", "pos"):
            getattr(self, n)[:rows].copy_(t[n])
        for n in ("len_lh", "cap_lh", "off_lh"):
            getattr(self, n).copy_(t[n].view(getattr(self, n).shape))
        self.ws_decode.zero_()                       # fresh arrival counters
        torch.cuda.synchronize(self.Kp.device)

    def decode(self, q, k_new, v_new, out, pos_new=None, stream=None):
        kvc.kvc_decode_attn(self.p, q, k_new, v_new, pos_new, self.Kp, self.Vp, self.logm,
                            self.pos, self.len_lh, self.cap_lh, self.off_lh, out, self.ws_decode,
                            stream)

    def extend(self, q, k_new, v_new, out, pos_new, n_new=None, lse=None, layers=None, softcap=0.0,
               window=0.0, slopes=None, stream=None):
        """A chunk of new tokens over the packed cache (kvc_chunk_attn): the
        follow-up turn of a conversation, or drafted tokens.  q, out
        [B, Lr, H*G, T, d], k_new, v_new [B, Lr, H, T, d] over the layers
        (begin, end), all of them by default; pos_new [B] f32 the position of
        each sequence's first new token; n_new [B] int32 when not every
        sequence has T.  The tokens are appended (len_lh advances) and take
        rows of the decode reserve."""
        p = self.p
        if p.packed_rows == 0:                       # built without the tensor-core decode
            p = kvc.kvc_params.from_buffer_copy(p)
            p.packed_rows = self.Kp.shape[0]
        l0, l1 = layers or (0, p.L)
        _check_chunk(p, l1 - l0, q, k_new, v_new, out,
                     pos_new=(pos_new, (p.B,), torch.float32), n_new=(n_new, (p.B,), torch.int32),
                     lse=(lse, (p.B, l1 - l0, p.H * p.G, *q.shape[3:4]), torch.float32),
                     slopes=(slopes, (p.H * p.G,), torch.float32))
        c = kvc.make_chunk(q.shape[3], l0, l1, n_new=n_new, softcap=softcap, window=window,
                           slopes=slopes)
        need = kvc.kvc_chunk_workspace_bytes(p, c)
        if self._ws_chunk is None or self._ws_chunk.numel() < need:
            if self._ws_chunk is not None:
                self._ws_outgrown.append(self._ws_chunk)
            self._ws_chunk = torch.empty(need, dtype=torch.uint8, device=self.device)
        kvc.kvc_chunk_attn(p, c, q, k_new, v_new, pos_new, self.Kp, self.Vp, self.logm, self.pos,
                           self.len_lh, self.cap_lh, self.off_lh, out, lse, self.len_lh,
                           self._ws_chunk, stream)

    def to_q8(self, reserve: int, pos_next, T: int = 1, **kw):
        """The packed cache in 8 bits (kvc_q8_pack), as a QuantizedCache with room for `reserve`
        more tokens per (b, l, h), in calls of up to T.  pos_next [B]: the position of each sequence's next token
        (n_max at most, unless n_pos says otherwise); further arguments as QuantizedCache's.
        Waits for the device once, for the lengths."""
        kw.setdefault("n_pos", self.p.n_max + int(reserve))
        cache = QuantizedCache(self.p, self.len_lh.cpu() + int(reserve), T, logm=True,
                               device=self.device, **kw)
        cache.pack(self.Kp, self.Vp, self.logm, self.len_lh, self.off_lh, pos_next)
        return cache

    def decode_many(self, q_all, kn_all, vn_all, out_all, pos_all=None, graph=True):
        """T = q_all.shape[0] decode steps back to back (step t reads q_all[t],
        kn_all[t], vn_all[t] and writes out_all[t]).  With graph=True the T calls
        are captured once per set of buffers into a CUDA graph and replayed, so
        the steps pay no per-launch host cost; the cache lengths advance on the
        device either way.  Returns the number of library kernels launched."""
        if not graph:
            n0 = kvc.kvc_launch_count()
            for t in range(q_all.shape[0]):
                self.decode(q_all[t], kn_all[t], vn_all[t], out_all[t],
                            None if pos_all is None else pos_all[t])
            return kvc.kvc_launch_count() - n0
        key = tuple(x.data_ptr() if x is not None else 0
                    for x in (q_all, kn_all, vn_all, out_all, pos_all)) + (q_all.shape[0],)
        g = self._graphs.get(key)
        if g is None:
            g = DecodeGraph(self.p, q_all, kn_all, vn_all, pos_all, self.Kp, self.Vp, self.logm,
                            self.pos, self.len_lh, self.cap_lh, self.off_lh, out_all,
                            self.ws_decode)
            self._graphs[key] = g
        g.replay()
        return g.launches


class DecodeGraph:
    """T kvc_decode_attn calls captured into one CUDA graph.

    The buffers are baked into the graph: replay() runs the T steps on the
    current stream over whatever the buffers then hold.  The library's one-time
    device lookups run before capture (a kvc_device_error call)."""

    def __init__(self, p, q_all, kn_all, vn_all, pos_all, Kp, Vp, logm, pos, len_lh, cap_lh,
                 off_lh, out_all, ws):
        dev = q_all.device
        kvc.kvc_device_error()                       # error-word lookup outside capture
        side = torch.cuda.Stream(device=dev)
        side.wait_stream(torch.cuda.current_stream(dev))
        self.graph = torch.cuda.CUDAGraph()
        n0 = kvc.kvc_launch_count()
        with torch.cuda.graph(self.graph, stream=side):
            for t in range(q_all.shape[0]):
                kvc.kvc_decode_attn(p, q_all[t], kn_all[t], vn_all[t],
                                    None if pos_all is None else pos_all[t], Kp, Vp, logm, pos,
                                    len_lh, cap_lh, off_lh, out_all[t], ws, side)
        self.launches = kvc.kvc_launch_count() - n0
        torch.cuda.current_stream(dev).wait_stream(side)
        # keep the baked buffers alive as long as the graph
        self._keep = (q_all, kn_all, vn_all, pos_all, Kp, Vp, logm, pos, len_lh, cap_lh, off_lh,
                      out_all, ws)

    def replay(self):
        self.graph.replay()


class EvictingCache:
    """NEXT f2: DistillCache per-step top-B eviction with the heuristic score
    (DistillCache Algorithm 1; the score is the attention feature alpha of 3.1.1).

    Every (b, l, h) holds the same tokens of sequence b (its prompt to start
    with) in the same rows of its `cap`-row range at off_lh = (b*L*H + l*H + h)
    * cap.  One step is kvc_decode_attn_lse (append + attend, base-2 LSE per
    query head and, with scores=True, every entry's score) -> kvc_token_alpha
    (from those scores, else recomputed from K) -> kvc_evict_topb (in place);
    every entry keeps log m = 0.  The class only allocates and marshals.
    """

    def __init__(self, p: kvc.kvc_params, K, V, ctx_len: Sequence[int], reserve: int,
                 ratio: float, b_min: int, tensor_cores: bool = True, scores: bool = True):
        B, L, H = p.B, p.L, p.H
        assert K.shape[:3] == (B, L, H) and K.shape == V.shape
        dev = K.device
        self.p, self.ratio, self.b_min = p, float(ratio), int(b_min)
        self.ctx = [int(n) for n in ctx_len]
        self.cap = max(self.ctx) + int(reserve)
        rows = B * L * H * self.cap
        p.packed_rows = rows if tensor_cores else 0
        dt = TORCH_DT[p.dtype]
        self.K = torch.zeros((rows, p.d), dtype=dt, device=dev)
        self.V = torch.zeros((rows, p.d), dtype=dt, device=dev)
        self.pos = torch.zeros((rows,), dtype=torch.float32, device=dev)
        self.logm = torch.zeros((rows,), dtype=torch.float32, device=dev)
        self._prompt = (K, V)
        self.len_lh = torch.zeros((B * L * H,), dtype=torch.int32, device=dev)
        self.cap_lh = torch.full((B * L * H,), self.cap, dtype=torch.int32, device=dev)
        self.off_lh = torch.arange(B * L * H, dtype=torch.int64, device=dev) * self.cap
        self.lse = torch.zeros((B * L * H, p.G), dtype=torch.float32, device=dev)
        # the decode's per-entry scores feed alpha (else alpha recomputes them from K)
        self.scores = (torch.zeros((rows, p.G), dtype=torch.float32, device=dev)
                       if scores else None)
        self.alpha = torch.zeros((B, self.cap), dtype=torch.float32, device=dev)
        self.ws_decode = torch.zeros(kvc.kvc_workspace_bytes(kvc.KVC_WS_DECODE, p),
                                     dtype=torch.uint8, device=dev)
        self.ws_evict = torch.empty(kvc.kvc_evict_workspace_bytes(p, self.cap),
                                    dtype=torch.uint8, device=dev)
        self._graphs = {}
        self.reset()

    def reset(self):
        """Back to the prompt: every (b, l, h) holds the prompt tokens in order."""
        p, (K, V) = self.p, self._prompt
        B, L, H = p.B, p.L, p.H
        Kc = self.K.view(B, L, H, self.cap, p.d)
        Vc = self.V.view(B, L, H, self.cap, p.d)
        Pc = self.pos.view(B, L, H, self.cap)
        for b, n in enumerate(self.ctx):
            assert n <= K.shape[3]
            Kc[b, :, :, :n] = K[b, :, :, :n]
            Vc[b, :, :, :n] = V[b, :, :, :n]
            Pc[b, :, :, :n] = torch.arange(n, dtype=torch.float32, device=K.device)
        lens = np.repeat(np.asarray(self.ctx, np.int32), L * H)
        self.len_lh.copy_(torch.from_numpy(lens))
        self.logm.zero_()

    def step(self, q, k_new, v_new, out, n_seen, pos_new=None, stream=None):
        """One decode step then one eviction; n_seen [B] int64 = tokens seen so far,
        this step's included."""
        kvc.kvc_decode_attn_lse(self.p, q, k_new, v_new, pos_new, self.K, self.V, self.logm,
                                self.pos, self.len_lh, self.cap_lh, self.off_lh, out, self.lse,
                                self.scores, self.ws_decode, stream)
        kvc.kvc_token_alpha(self.p, q, self.K, self.scores, self.len_lh, self.off_lh, self.lse,
                            self.alpha, self.ws_evict, stream)
        kvc.kvc_evict_topb(self.p, self.alpha, n_seen, self.ratio, self.b_min, self.K, self.V,
                           self.pos, self.logm, self.off_lh, self.len_lh, self.ws_evict, stream)

    def run_many(self, q_all, kn_all, vn_all, out_all, nseen_all, pos_all=None, graph=True):
        """T steps back to back (step t reads row t of every *_all tensor); with
        graph=True they are captured once per set of buffers into a CUDA graph
        and replayed.  Returns the library kernels launched."""
        T = q_all.shape[0]
        if not graph:
            n0 = kvc.kvc_launch_count()
            for t in range(T):
                self.step(q_all[t], kn_all[t], vn_all[t], out_all[t], nseen_all[t],
                          None if pos_all is None else pos_all[t])
            return kvc.kvc_launch_count() - n0
        key = tuple(x.data_ptr() if x is not None else 0
                    for x in (q_all, kn_all, vn_all, out_all, nseen_all, pos_all)) + (T,)
        g = self._graphs.get(key)
        if g is None:
            dev = q_all.device
            kvc.kvc_device_error()                   # error-word lookup outside capture
            side = torch.cuda.Stream(device=dev)
            side.wait_stream(torch.cuda.current_stream(dev))
            graph_ = torch.cuda.CUDAGraph()
            n0 = kvc.kvc_launch_count()
            with torch.cuda.graph(graph_, stream=side):
                for t in range(T):
                    self.step(q_all[t], kn_all[t], vn_all[t], out_all[t], nseen_all[t],
                              None if pos_all is None else pos_all[t], side)
            torch.cuda.current_stream(dev).wait_stream(side)
            g = (graph_, kvc.kvc_launch_count() - n0,
                 (q_all, kn_all, vn_all, out_all, nseen_all, pos_all))
            self._graphs[key] = g
        g[0].replay()
        return g[1]

    def entries(self, b: int, l: int, h: int):
        """(K, V, pos) rows the (b, l, h) currently holds, in row order (host copies)."""
        blh = (b * self.p.L + l) * self.p.H + h
        n = int(self.len_lh[blh])
        o = blh * self.cap
        return (self.K[o:o + n].float().cpu().numpy(), self.V[o:o + n].float().cpu().numpy(),
                self.pos[o:o + n].cpu().numpy())


def _check_chunk(p: kvc.kvc_params, layers: int, q, k_new, v_new, out, **others):
    """A chunk's tensors have the cache's type and the shapes the library reads;
    the others are (tensor or None, shape, type)."""
    if q.dim() != 5 or q.shape[3] < 1:
        raise ValueError("q must be [B, layers, H*G, T, d]")
    dt = TORCH_DT[p.dtype]
    want = {"q": (q, p.H * p.G), "k_new": (k_new, p.H), "v_new": (v_new, p.H), "out": (out, p.H * p.G)}
    want = {k: (t, (p.B, layers, heads, q.shape[3], p.d), dt) for k, (t, heads) in want.items()}
    for name, (t, shape, dtype) in {**want, **others}.items():
        if t is not None and (tuple(t.shape) != shape or t.dtype != dtype):
            raise ValueError(f"{name} must be {list(shape)} {dtype}")


class ChunkedCache:
    """A cache of bounded size that a prompt of any length streams through, chunk
    by chunk, and that decoding goes on with.

    Every (b, l, h) owns pages for `budget` entries and one chunk of T tokens.
    A step attends (kvc_chunk_attn), adds the chunk's attention weight to the
    entries' masses (kvc_chunk_mass) and, with evict=True, drops what has least
    of it until `budget` entries are left (kvc_mass_evict), the last `recent`
    positions always staying.  The masses decay once a step, for a chunk of T tokens as
    for a single one (and for a sequence without new tokens).  Nothing waits for the device, so steps can be
    captured into a CUDA graph.  The class only allocates and marshals.
    """

    def __init__(self, p: kvc.kvc_params, budget: int, T: int, page_rows: int = 64,
                 recent: int = 128, decay: float = 1.0, softcap: float = 0.0, window: float = 0.0,
                 slopes=None, device="cuda"):
        if not 0 <= recent <= budget:
            raise ValueError("the protected positions must fit the budget")
        if not 0.0 <= decay <= 1.0:
            raise ValueError("decay must be in 0..1")
        if slopes is not None and (tuple(slopes.shape) != (p.H * p.G,) or slopes.dtype != torch.float32):
            raise ValueError(f"slopes must be [{p.H * p.G}] float32")
        B, L, H = p.B, p.L, p.H
        self.budget, self.recent, self.decay = int(budget), int(recent), float(decay)
        per = -(-(self.budget + int(T)) // page_rows)
        self.cap = per * page_rows
        rows = B * L * H * self.cap
        self.p = kvc.kvc_params.from_buffer_copy(p)
        self.p.packed_rows = rows
        z = dict(device=device)
        dt = TORCH_DT[p.dtype]
        self.K = torch.zeros((rows, p.d), dtype=dt, **z)
        self.V = torch.zeros((rows, p.d), dtype=dt, **z)
        self.logm = torch.zeros((rows,), dtype=torch.float32, **z)
        self.pos = torch.zeros((rows,), dtype=torch.float32, **z)
        self.mass = torch.zeros((rows,), dtype=torch.float32, **z)
        self.table = torch.arange(B * L * H * per, dtype=torch.int32, **z).view(B, L, H, per)
        self.len_lh = torch.zeros((B, L, H), dtype=torch.int32, **z)
        self.len_new = torch.zeros((B, L, H), dtype=torch.int32, **z)
        self.cap_lh = torch.full((B, L, H), self.cap, dtype=torch.int32, **z)
        self.keep_lh = torch.full((B, L, H), self.budget, dtype=torch.int32, **z)
        self.pos_next = torch.zeros((B,), dtype=torch.float32, **z)
        self.n_new = torch.zeros((B,), dtype=torch.int32, **z)
        self.lse = torch.empty((B, L, p.H * p.G, int(T)), dtype=torch.float32, **z)
        self._mods = dict(page_rows=page_rows, page_table=self.table, n_new=self.n_new,
                          softcap=softcap, window=window, slopes=slopes)
        self.T = int(T)
        c = self._chunk(self.T)
        self.ws = torch.empty(max(kvc.kvc_chunk_workspace_bytes(self.p, c),
                                  kvc.kvc_mass_evict_workspace_bytes(self.p, c, self.cap)),
                              dtype=torch.uint8, device=device)

    def _chunk(self, T):
        return kvc.make_chunk(T, 0, self.p.L, **self._mods)

    def step(self, q, k_new, v_new, out, n_new=None, evict=True, stream=None):
        """One chunk of q.shape[3] <= T tokens per sequence (n_new [B] int32 on the
        device when not every sequence has that many): q, out [B, L, H*G, T', d],
        k_new, v_new [B, L, H, T', d].  With a `stream`, it must be torch's current
        one.  A sequence without room for its tokens (evict=False before), or with a
        count above T', is skipped: it takes no token, its masses do not decay, its
        next position stays, and kvc_device_error reports it."""
        _check_chunk(self.p, self.p.L, q, k_new, v_new, out,
                     n_new=(n_new, (self.p.B,), torch.int32))
        if stream is not None and kvc._raw_stream(stream) != kvc._raw_stream(None):
            raise ValueError("the stream must be torch's current one")
        if evict and self.p.B * self.p.L * self.p.H > 65535:
            raise ValueError("the eviction takes up to 65535 (b, l, h)")
        T = q.shape[3]
        if T > self.T:
            raise ValueError(f"a chunk of {T} tokens, the cache was built for {self.T}")
        if n_new is None:
            self.n_new.fill_(T)
        else:
            self.n_new.copy_(n_new)
        c = self._chunk(T)
        lse = self.lse if T == self.T else self.lse.view(-1)[:self.lse.numel() // self.T * T]
        kvc.kvc_chunk_attn(self.p, c, q, k_new, v_new, self.pos_next, self.K, self.V, self.logm,
                           self.pos, self.len_lh, self.cap_lh, None, out, lse, self.len_new,
                           self.ws, stream)
        kvc.kvc_chunk_mass(self.p, c, q, self.K, self.logm, self.pos, self.pos_next, self.len_lh,
                           None, lse, self.decay, self.mass, self.ws, stream, self.cap_lh)
        # what was taken, not what was asked for: units that the device skipped keep their length
        self.pos_next.add_((self.len_new - self.len_lh).flatten(1).amax(1))
        if evict:
            kvc.kvc_mass_evict(self.p, c, self.mass, self.keep_lh, self.recent, self.pos_next,
                               self.K, self.V, self.logm, self.pos, self.len_new, None,
                               self.len_lh, self.cap, self.ws, stream)
        else:
            self.len_lh.copy_(self.len_new)

    def entries(self, b: int, l: int, h: int):
        """(K, V, pos, mass) of the entries (b, l, h) holds, in row order (host copies)."""
        n = int(self.len_lh[b, l, h])
        o = ((b * self.p.L + l) * self.p.H + h) * self.cap
        return tuple(t[o:o + n].float().cpu().numpy() for t in (self.K, self.V, self.pos, self.mass))


class QuantizedCache:
    """A paged cache of e4m3 codes with a power-of-two scale for every page and head
    (kvc_q8_*): half the bytes of a bf16 cache, empty at first or a compressed cache in 8
    bits (Compressor.to_q8).

    A step rotates and appends the new tokens (kvc_q8_append) and attends (kvc_q8_attn); with
    n_sel, every token of every KV head attends over n_sel pages only (kvc_q8_select): the `first`
    pages, the last `recent` ones, and of the others those of largest score.  Every (b, l, h) owns pages
    for `tokens` entries (a number, or [B, L, H] of them in host memory); positions go up to n_pos.  Nothing waits for the device or allocates, so
    steps can be captured into a CUDA graph.  The class only allocates and marshals.
    """

    def __init__(self, p: kvc.kvc_params, tokens, T: int = 1, page_rows: int = 64,
                 n_pos: Optional[int] = None, n_sel: int = 0, first: int = 1, recent: int = 2,
                 logm: bool = False, rotate: bool = True, device="cuda"):
        if n_sel and not (first >= 0 and recent >= 1 and first + recent <= n_sel):
            raise ValueError("the first and recent pages must fit n_sel")
        # what a call of a step would refuse, before there is anything to lose
        if page_rows not in (16, 32, 64, 128):
            raise ValueError("page_rows must be 16, 32, 64 or 128")
        B, L, H = p.B, p.L, p.H
        room = torch.as_tensor(tokens, dtype=torch.int64, device="cpu")
        if room.dim() and tuple(room.shape) != (B, L, H):
            raise ValueError(f"tokens must be a number or {[B, L, H]}")
        if int(room.min()) < 1 or not 1 <= T <= 65536:
            raise ValueError("a cache holds at least one token and takes 1 to 65536 at a time")
        owned = torch.div(room + (page_rows - 1), page_rows, rounding_mode="floor").expand(B, L, H)   # pages
        per, pages = int(owned.max()), int(owned.sum())
        self.T, self.cap, self.page_rows = int(T), per * page_rows, int(page_rows)
        self.n_sel, self.first, self.recent = int(n_sel), int(first), int(recent)
        if pages * page_rows >= 1 << 31 or self.cap > 1 << 27:
            raise ValueError("a cache has fewer than 2^31 rows, and 2^27 at most of one (b, l, h)")
        if n_sel and (n_sel > 32768 or per > 32768):
            raise ValueError("pages are picked from 32768 of a (b, l, h) at most")
        self.p = kvc.kvc_params.from_buffer_copy(p)
        self.p.packed_rows = pages * page_rows
        z = dict(device=device)
        f32, i32, u8 = torch.float32, torch.int32, torch.uint8
        self._first = owned.flatten().cumsum(0).view(B, L, H) - owned     # pages before a (b, l, h)'s own
        column = torch.arange(per)
        self.table = torch.where(column < owned[..., None], self._first[..., None] + column, -1).to(dtype=i32, **z)
        self.n_new = torch.zeros((B,), dtype=i32, **z)
        # (what a call needs depends on its tokens: a few row tiles, or expanded rows)
        few = min(self.T, 64 // p.G + 1)
        need = [kvc.kvc_q8_workspace_bytes(self.p, self._chunk(t), self.n_sel) for t in {self.T, *range(1, few + 1)}]
        if min(need) == 0:
            raise ValueError("the library takes no cache of these sizes")
        self.ws = torch.empty(max(need), dtype=u8, **z)
        self.K = torch.zeros((pages * page_rows, p.d), dtype=u8, **z)
        self.V = torch.zeros((pages * page_rows, p.d), dtype=u8, **z)
        self.k_scale = torch.ones((pages,), dtype=f32, **z)
        self.v_scale = torch.ones((pages,), dtype=f32, **z)
        self.bounds = torch.zeros((pages, 2, p.d), dtype=torch.int8, **z) if n_sel else None
        self.logm = torch.zeros((pages * page_rows,), dtype=f32, **z) if logm else None
        self.x = kvc.make_q8(self.K, self.V, self.k_scale, self.v_scale, self.bounds, self.logm)
        self.len_lh = torch.zeros((B, L, H), dtype=i32, **z)
        self.len_new = torch.zeros((B, L, H), dtype=i32, **z)
        self.cap_lh = (owned * page_rows).to(dtype=i32, **z)
        self.pos_next = torch.zeros((B,), dtype=f32, **z)
        self.rope_cos = self.rope_sin = None
        if rotate:
            n_half = 2 * int(n_pos if n_pos is not None else max(p.n_max, self.cap))
            self.rope_cos = torch.empty((n_half, p.d // 2), dtype=f32, **z)
            self.rope_sin = torch.empty((n_half, p.d // 2), dtype=f32, **z)
            kvc.kvc_rope_table(p.d, p.rope_base, n_half, self.rope_cos, self.rope_sin)
        self.q = torch.empty((B * L * H * p.G * self.T * p.d,), dtype=TORCH_DT[p.dtype], **z)
        self.sel = torch.empty((B * L * H * self.T * max(1, n_sel),), dtype=i32, **z)

    def _chunk(self, T):
        return kvc.make_chunk(T, 0, self.p.L, page_rows=self.page_rows, page_table=self.table, n_new=self.n_new)

    def pack(self, Kp, Vp, logm, len_lh, off_lh, pos_next, stream=None):
        """Replaces the cache by a packed one (its keys are rotated already); pos_next [B]:
        the position of each sequence's next token.  With a `stream`, it must be torch's
        current one."""
        _current_stream_only(stream)
        if tuple(pos_next.shape) != (self.p.B,):
            raise ValueError(f"pos_next must be [{self.p.B}]")
        kvc.kvc_q8_pack(self.p, self._chunk(1), self.x, Kp, Vp, logm, len_lh, off_lh, self.cap_lh, self.len_new,
                        stream)
        self.len_lh.copy_(self.len_new)
        self.pos_next.copy_(pos_next)

    def step(self, q, k_new, v_new, out, n_new=None, lse=None, stream=None):
        """q.shape[3] <= T new tokens per sequence (n_new [B] int32 on the device when not
        every sequence has that many): q, out [B, L, H*G, T', d], k_new, v_new
        [B, L, H, T', d], not rotated yet; lse [B, L, H*G, T'] or None.  With a `stream`, it must be torch's
        current one.  A (b, l, h) without room is skipped: it takes no token, its rows of out
        stay, and kvc_device_error reports it (as it does a count above T', or positions beyond n_pos)."""
        p, T = self.p, q.shape[3] if q.dim() == 5 else 0
        _check_chunk(p, p.L, q, k_new, v_new, out, n_new=(n_new, (p.B,), torch.int32),
                     lse=(lse, (p.B, p.L, p.H * p.G, T), torch.float32))
        _current_stream_only(stream)
        if T > self.T:
            raise ValueError(f"{T} tokens, the cache was built for {self.T}")
        c = self._chunk(T)
        # the attention would refuse these only after the tokens are in the cache
        kvc._q8_ptrs(c, self.x, out, lse)
        if out.data_ptr() % 32:
            raise ValueError("out must begin on a 32-byte boundary")
        if n_new is None:
            self.n_new.fill_(T)
        else:
            self.n_new.copy_(n_new)
        turned = self.q[:q.numel()].view(q.shape)
        kvc.kvc_q8_append(p, c, self.x, self.rope_cos, self.rope_sin, q, k_new, v_new, self.pos_next, turned,
                          self.len_lh, self.cap_lh, self.len_new, stream)
        sel = None
        if self.n_sel:
            sel = self.sel[:p.B * p.L * p.H * T * self.n_sel].view(p.B, p.L, p.H, T, self.n_sel)
            kvc.kvc_q8_select(p, c, self.x, turned, self.len_lh, self.len_new, self.first, self.recent, sel, stream)
        kvc.kvc_q8_attn(p, c, self.x, turned, self.len_lh, self.len_new, sel, out, lse, self.ws, stream)
        # what was taken, not what was asked for: (b, l, h) that the device skipped keep their length
        self.pos_next.add_((self.len_new - self.len_lh).flatten(1).amax(1))
        self.len_lh.copy_(self.len_new)

    def entries(self, b: int, l: int, h: int):
        """(K, V, log m or None) the (b, l, h) holds, in entry order (host copies)."""
        n = int(self.len_lh[b, l, h])
        o = int(self._first[b, l, h]) * self.page_rows
        page = torch.arange(o, o + n, device=self.K.device) // self.page_rows
        K, V = (t[o:o + n].view(torch.float8_e4m3fn).float() * s[page][:, None]
                for t, s in ((self.K, self.k_scale), (self.V, self.v_scale)))
        return K.cpu().numpy(), V.cpu().numpy(), None if self.logm is None else self.logm[o:o + n].cpu().numpy()


def _current_stream_only(stream):
    if stream is not None and kvc._raw_stream(stream) != kvc._raw_stream(None):
        raise ValueError("the stream must be torch's current one")


def pad_bounds(bounds_list, S_max: int) -> np.ndarray:
    """[B, S_max + 1] int32 slot boundaries (rows padded with their last value)."""
    out = np.zeros((len(bounds_list), S_max + 1), dtype=np.int32)
    for b, bd in enumerate(bounds_list):
        bd = np.asarray(bd, dtype=np.int32)
        out[b, :len(bd)] = bd
        out[b, len(bd):] = bd[-1]
    return out
