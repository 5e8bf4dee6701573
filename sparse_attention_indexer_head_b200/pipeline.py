"""One DSA decode/prefill step on the GPU: device buffers plus the C-ABI calls.

PyTorch is used for device memory, pinned host memory and streams only; every
stage runs in libdsa.so:
  dsa_kpool_compress -> dsa_head_gate -> dsa_index_scores -> dsa_topk_expand
  -> dsa_sparse_mla_decode,
or, with the fused indexer, dsa_kpool_compress -> dsa_indexer_select (gate,
scores, top-k and expansion in one launch) -> dsa_sparse_mla_decode.
Cache-side tensors (k, gate logits, validity, latent kv, request offsets and
the layer weights) are device-resident state; query-side tensors (hidden,
indexer queries, MLA queries, query request/position) are the per-step inputs.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Dict, Optional

import numpy as np
import torch

from . import binding as B
from .workloads import INDEX_DIM, INDEX_HEADS, KV_LORA, Workload

QUERY_INPUTS = ("hidden", "q_idx", "q_mla", "q_req", "q_pos")
INDEXER_MAX_POOLS = 32768          # dsa_indexer_select's pool limit
AUTO_FUSED_MAX_QUERIES = 256       # "auto": the fused indexer up to this many queries
PREFIX_MAX_QUERIES = 65535         # dsa_prefix_mla_decode_paged's query limit


def _bf16(a: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16)


def host_tensors(wl: Workload) -> Dict[str, torch.Tensor]:
    """CPU torch views of a workload's arrays (bf16 bit patterns as torch.bfloat16)."""
    return {
        "hidden": torch.from_numpy(wl.hidden),
        "w_gate": torch.from_numpy(wl.w_gate),
        "q_idx": _bf16(wl.q_idx),
        "k": _bf16(wl.k),
        "gate": _bf16(wl.gate),
        "valid": torch.from_numpy(wl.valid),
        "req_start": torch.from_numpy(wl.req_start),
        "ape": torch.from_numpy(wl.ape),
        "ln_w": _bf16(wl.ln_w),
        "ln_b": _bf16(wl.ln_b),
        "q_mla": _bf16(wl.q_mla),
        "kv": _bf16(wl.kv),
        "q_req": torch.from_numpy(wl.q_req),
        "q_pos": torch.from_numpy(wl.q_pos),
    }


@dataclass
class Geometry:
    B: int
    Q: int
    kpool: int
    max_pools: int
    select_k: int
    hm: int
    eps: float
    sm_scale: float
    tail: int = 0           # always_select_tail: kpool - 1 extra slots per index row

    @property
    def W(self) -> int:
        return self.select_k * self.kpool + self.tail


class DecodeStep:
    """Device buffers of one step; ``run()`` enqueues the five calls on a stream."""

    def __init__(self, wl: Workload, device: str = "cuda", inputs: Optional[Dict] = None,
                 always_select_tail: bool = False, fused_indexer: bool = False):
        self.device = torch.device(device)
        # fused_indexer: gate, scores, top-k and expansion in one dsa_indexer_select
        # call (not with always_select_tail, whose tail slots only dsa_topk_expand_tail
        # writes, nor above its pool limit). "auto" takes it for decode-sized batches:
        # its cluster of 8 CTAs a query recomputes the gate and re-reads the request's
        # pooled keys per query, which the separate calls amortise over many queries.
        if fused_indexer == "auto":
            fused_indexer = wl.Q <= AUTO_FUSED_MAX_QUERIES
        self.fused = (bool(fused_indexer) and not always_select_tail
                      and wl.max_pools <= INDEXER_MAX_POOLS)
        self.g = Geometry(wl.B, wl.Q, wl.kpool, wl.max_pools, wl.select_k, wl.hm, wl.eps,
                          wl.sm_scale, wl.kpool - 1 if always_select_tail else 0)
        src = host_tensors(wl) if inputs is None else inputs
        self.t = {k: v.to(self.device) for k, v in src.items()}
        g, dev = self.g, self.device
        self.gate_w = torch.empty(g.Q, INDEX_HEADS, dtype=torch.float32, device=dev)
        self.pool_keys = torch.zeros(g.B, g.max_pools, INDEX_DIM, dtype=torch.bfloat16, device=dev)
        self.pool_idx = torch.empty(g.B, g.max_pools, g.kpool, dtype=torch.int32, device=dev)
        self.pool_valid = torch.empty(g.B, g.max_pools, dtype=torch.uint8, device=dev)
        self.first_valid = torch.empty(g.B, dtype=torch.int32, device=dev)
        self.scores = torch.empty(g.Q, g.max_pools, dtype=torch.float32, device=dev)
        self.cand = torch.empty(g.Q, g.max_pools, dtype=torch.uint8, device=dev)
        self.top_pools = torch.empty(g.Q, g.select_k, dtype=torch.int32, device=dev)
        self.token_ids = torch.empty(g.Q, g.W, dtype=torch.int32, device=dev)
        self.out = torch.empty(g.Q, g.hm, KV_LORA, dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty(g.Q, g.hm, dtype=torch.float32, device=dev)
        ws = B.dsa_sparse_mla_workspace_size(g.Q, g.hm, g.W)
        self.ws = torch.empty(max(ws, 16), dtype=torch.uint8, device=dev)

    # -- the five stages ---------------------------------------------------------------
    def head_gate(self, stream=None):
        g, t = self.g, self.t
        B.dsa_head_gate(t["hidden"], t["w_gate"], self.gate_w, g.Q, t["hidden"].shape[1],
                        INDEX_HEADS, stream)

    def kpool_compress(self, stream=None):
        g, t = self.g, self.t
        B.dsa_kpool_compress(t["k"], t["gate"], t["valid"], t["req_start"], g.B, INDEX_DIM,
                             g.kpool, g.max_pools, t["ape"], t["ln_w"], t["ln_b"], g.eps,
                             self.pool_keys, self.pool_idx, self.pool_valid, self.first_valid,
                             stream)

    def index_scores(self, stream=None):
        g, t = self.g, self.t
        B.dsa_index_scores(t["q_idx"], self.gate_w, t["q_req"], t["q_pos"], g.Q, INDEX_HEADS,
                           INDEX_DIM, self.pool_keys, self.pool_valid, self.first_valid, g.B,
                           g.kpool, g.max_pools, self.scores, self.cand, stream)

    def topk_expand(self, stream=None):
        g, t = self.g, self.t
        if g.tail:
            B.dsa_topk_expand_tail(self.scores, self.cand, self.pool_idx, t["q_req"], t["q_pos"],
                                   self.first_valid, t["valid"], t["req_start"], g.Q, g.B,
                                   g.max_pools, g.kpool, g.select_k, self.top_pools,
                                   self.token_ids, stream)
        else:
            B.dsa_topk_expand(self.scores, self.cand, self.pool_idx, t["q_req"], g.Q, g.B,
                              g.max_pools, g.kpool, g.select_k, self.top_pools, self.token_ids,
                              stream)

    def sparse_mla(self, stream=None):
        g, t = self.g, self.t
        B.dsa_sparse_mla_decode(t["q_mla"], t["kv"], t["kv"].shape[0], t["req_start"], t["q_req"],
                                self.token_ids,
                                g.Q, g.B, g.hm, g.W, KV_LORA, 0, g.sm_scale, self.out, self.lse,
                                self.ws, self.ws.numel(), stream)

    def indexer(self, stream=None):
        """a1 + a4 + a5 + a6 in one launch (dsa_indexer_select)."""
        g, t = self.g, self.t
        B.dsa_indexer_select(t["hidden"], t["w_gate"], t["hidden"].shape[1], t["q_idx"], t["q_req"],
                             t["q_pos"], g.Q, INDEX_HEADS, INDEX_DIM, self.pool_keys,
                             self.pool_valid, self.first_valid, self.pool_idx, g.B, g.kpool,
                             g.max_pools, g.select_k, self.gate_w, self.scores, self.cand,
                             self.top_pools, self.token_ids, stream)

    def stages(self):
        """Names of the stage methods run() calls, in order."""
        if self.fused:
            return ["kpool_compress", "indexer", "sparse_mla"]
        # compress first: the small head-gate grid then overlaps compress's tail
        # (every kernel is launched with programmatic dependent launch).
        return ["kpool_compress", "head_gate", "index_scores", "topk_expand", "sparse_mla"]

    def run(self, stream=None):
        for name in self.stages():
            getattr(self, name)(stream)

    # -- incremental decode: the step's new token rows update the pooled-key cache -------
    def stage_new_tokens(self, k_new=None, gate_new=None, valid_new=None, tok_req=None,
                         tok_pos=None):
        """Device buffers of a step's new indexer rows and the token ranges they change.

        Default: one new token per request, its last row (position T_b - 1), with
        the k and gate values the cache already holds there, so a step that
        stores it leaves the cache as it was and its outputs can be compared
        with the full step's. Requests with no rows get none.
        """
        g, t, dev = self.g, self.t, self.device
        rs = t["req_start"].to("cpu").numpy().astype(np.int64)
        lengths = rs[1:] - rs[:-1]
        if tok_req is None:
            have = np.nonzero(lengths > 0)[0]
            tok_req = have.astype(np.int32)
            tok_pos = (lengths[have] - 1).astype(np.int32)
            rows = torch.from_numpy(rs[have] + tok_pos).to(dev)
            k_new = t["k"].index_select(0, rows)
            gate_new = t["gate"].index_select(0, rows)
            valid_new = t["valid"].index_select(0, rows)
        tok_req = np.asarray(tok_req, np.int32)
        tok_pos = np.asarray(tok_pos, np.int32)
        begin = np.full(g.B, 0, np.int32)
        end = np.full(g.B, 0, np.int32)
        for b in range(g.B):                   # the smallest range holding b's new rows
            mine = tok_pos[tok_req == b]
            if mine.size:
                begin[b], end[b] = mine.min(), mine.max() + 1
        self.new = {
            "k": torch.as_tensor(k_new).to(dev), "gate": torch.as_tensor(gate_new).to(dev),
            "valid": None if valid_new is None else torch.as_tensor(valid_new).to(dev),
            "tok_req": torch.from_numpy(tok_req).to(dev), "tok_pos": torch.from_numpy(tok_pos).to(dev),
            "n": int(tok_req.shape[0]),
            "tok_begin": torch.from_numpy(begin).to(dev), "tok_end": torch.from_numpy(end).to(dev),
        }

    def indexer_store(self, stream=None):
        g, t, n = self.g, self.t, self.new
        B.dsa_indexer_store(n["k"], n["gate"], n["valid"], n["tok_req"], n["tok_pos"], n["n"],
                            INDEX_DIM, t["req_start"], g.B, t["k"], t["gate"], t["valid"], stream)

    def kpool_compress_tokens(self, stream=None):
        g, t, n = self.g, self.t, self.new
        B.dsa_kpool_compress_tokens(t["k"], t["gate"], t["valid"], t["req_start"], g.B, INDEX_DIM,
                                    g.kpool, g.max_pools, t["ape"], t["ln_w"], t["ln_b"], g.eps,
                                    n["tok_begin"], n["tok_end"], self.pool_keys, self.pool_idx,
                                    self.pool_valid, self.first_valid, stream)

    def run_incremental(self, stream=None):
        """A decode step that stores the new rows and recomputes only their pools.

        The pooled-key outputs must already hold the compress result of the
        cache before the new rows (run() or kpool_compress() once).
        """
        self.indexer_store(stream)
        self.kpool_compress_tokens(stream)
        for name in self.stages()[1:]:
            getattr(self, name)(stream)

    def kernels_per_step(self) -> int:
        """Launches of run(): compress, then gate, scores and topk+expand (or the one fused
        indexer), and the MLA's one or two kernels (split kernel, plus the combine when
        splits merge in the workspace)."""
        g = self.g
        return len(self.stages()) - 1 + B.dsa_sparse_mla_launch_count(g.Q, g.hm, g.W)

    def kernels_per_step_incremental(self) -> int:
        """Launches of run_incremental(): store (when there are new rows), token-range
        compress, the indexer stage(s) and the MLA's kernels."""
        return (1 if self.new["n"] > 0 else 0) + self.kernels_per_step()

    def outputs_numpy(self) -> Dict[str, np.ndarray]:
        def u16(x):
            return x.view(torch.int16).cpu().numpy().view(np.uint16)
        return {
            "gate_w": self.gate_w.cpu().numpy(),
            "pool_keys": u16(self.pool_keys),
            "pool_idx": self.pool_idx.cpu().numpy(),
            "pool_valid": self.pool_valid.cpu().numpy(),
            "first_valid": self.first_valid.cpu().numpy(),
            "scores": self.scores.cpu().numpy(),
            "cand": self.cand.cpu().numpy(),
            "top_pools": self.top_pools.cpu().numpy(),
            "token_ids": self.token_ids.cpu().numpy(),
            "out": u16(self.out),
            "lse": self.lse.cpu().numpy(),
        }


class StreamedDecode:
    """Decode steps served from and to pinned host memory.

    Each slot owns a pinned host input buffer (the query inputs packed, see
    `write_inputs`), device buffers and a pinned host output buffer, and a CUDA
    graph that copies the inputs host -> device, runs the five calls and copies
    the output device -> host, on the slot's own stream. Steps rotate over the
    slots, so consecutive steps run on different streams and overlap on the
    GPU (their copies and kernels interleave). Step i uses slot i % slots: its
    inputs must be in that slot's buffer when it is submitted, and the buffer
    may be refilled for step i + slots once result(i) has returned.
    """

    def __init__(self, wl: Workload, device: str = "cuda", slots: int = 2,
                 inputs: Optional[Dict] = None, fused_indexer: bool = False):
        self.device = torch.device(device)
        self.steps = [DecodeStep(wl, device=device, inputs=inputs, fused_indexer=fused_indexer)
                      for _ in range(slots)]
        # A slot's query inputs live in one device buffer: one copy per step.
        self.layout, nbytes = {}, 0
        for name in QUERY_INPUTS:
            t = self.steps[0].t[name]
            nbytes = (nbytes + 255) // 256 * 256
            self.layout[name] = (nbytes, t.dtype, tuple(t.shape))
            nbytes += t.numel() * t.element_size()
        self.nbytes = nbytes
        self.dev_in, self.in_host, self.out_host, self.streams = [], [], [], []
        for st in self.steps:
            buf = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
            host = torch.zeros(nbytes, dtype=torch.uint8).pin_memory()
            for name, (off, dtype, shape) in self.layout.items():
                view = self._view(buf, off, dtype, shape)
                view.copy_(st.t[name])
                self._view(host, off, dtype, shape).copy_(st.t[name].cpu())
                st.t[name] = view
            self.dev_in.append(buf)
            self.in_host.append(host)
            self.out_host.append(torch.empty(st.out.shape, dtype=st.out.dtype).pin_memory())
            self.streams.append(torch.cuda.Stream(device=self.device))
        self.graphs = []
        for k, st in enumerate(self.steps):
            with torch.cuda.stream(self.streams[k]):
                st.run()                                  # sets kernel attributes eagerly
            self.streams[k].synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=self.streams[k]):
                self.dev_in[k].copy_(self.in_host[k], non_blocking=True)
                st.run()
                self.out_host[k].copy_(st.out, non_blocking=True)
            self.graphs.append(g)
        torch.cuda.synchronize(self.device)
        self.done = [torch.cuda.Event() for _ in self.steps]
        self.submitted = 0

    @staticmethod
    def _view(buf: torch.Tensor, off: int, dtype, shape) -> torch.Tensor:
        n = 1
        for d in shape:
            n *= d
        size = n * torch.empty((), dtype=dtype).element_size()
        return buf[off:off + size].view(dtype).view(shape)

    def slot(self, i: int) -> int:
        return i % len(self.steps)

    def write_inputs(self, i: int, host_inputs: Dict[str, torch.Tensor]) -> None:
        """Pack step i's query inputs (names of QUERY_INPUTS) into its slot's buffer."""
        buf = self.in_host[self.slot(i)]
        for name, (off, dtype, shape) in self.layout.items():
            self._view(buf, off, dtype, shape).copy_(host_inputs[name])

    def submit(self) -> int:
        """Enqueue the next step on its slot's stream; returns its index."""
        i = self.submitted
        k = self.slot(i)
        with torch.cuda.stream(self.streams[k]):
            self.graphs[k].replay()
            self.done[k].record(self.streams[k])
        self.submitted += 1
        return i

    def result(self, i: int) -> torch.Tensor:
        """Step i's output [Q, Hm, 512] bf16 on the host (step i must be among the
        last `slots` submitted)."""
        if not (self.submitted - len(self.steps) <= i < self.submitted):
            raise ValueError("step is not among the slots in flight")
        self.done[self.slot(i)].synchronize()
        return self.out_host[self.slot(i)]

    def kernels_per_step(self) -> int:
        return self.steps[0].kernels_per_step()


def _operand(x: torch.Tensor, device: torch.device, dtype: torch.dtype) -> torch.Tensor:
    """x as the entry points read it: of that type, on the device, its elements in order from a
    16-byte aligned address (x itself where it is so already)."""
    x = x.to(device, dtype).contiguous()
    return x if x.data_ptr() % 16 == 0 else x.clone()


def _torch_stream(s) -> torch.cuda.Stream:
    """A stream as torch's: a handle (0 is the default stream) or an object that has one."""
    if isinstance(s, torch.cuda.Stream):
        return s
    handle = s if isinstance(s, int) else s.cuda_stream
    return torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()


class PrefixDecode:
    """Dense MLA over a paged latent cache for a batch whose requests share a prefix.

    Owns the cache (bf16, or E4M3 with one scale), the page tables and the lengths on the
    device. ``fill_prefix`` appends the shared prefix's latent rows once; ``step`` appends
    one new row a request (normalised, rotated at its position; dsa_latent_append_paged),
    rotates the step's query heads in the same launch and attends over prefix and own
    tokens (dsa_prefix_mla_decode_paged): all requests in step, from the prefix's end on.
    Batches of ragged lengths, several new tokens a request or prompts of its own call the
    two entry points themselves. A step whose call fails is not taken. With ``graph`` the two calls are captured at the
    first step and replayed: the lengths are device data, and every page a request can
    come to hold is in its table from the start.
    """

    def __init__(self, requests: int, heads: int, max_own: int, prefix_len: int, *,
                 norm_w: Optional[torch.Tensor], cos_sin: Optional[torch.Tensor] = None,
                 interleaved: bool = True, page: int = 64, fp8: bool = False, kv_scale: float = 1.0,
                 eps: float = 1e-6, sm_scale: float = KV_LORA ** -0.5, graph: bool = False,
                 device: str = "cuda"):
        if norm_w is not None and tuple(norm_w.shape) != (KV_LORA,):
            raise ValueError(f"norm_w is {tuple(norm_w.shape)}, not ({KV_LORA},)")
        if min(requests, max_own, prefix_len) < 0 or page < 1:
            raise ValueError("requests, max_own and prefix_len are not negative, page is positive")
        self.max_len = prefix_len + max_own
        if cos_sin is not None and (cos_sin.dim() != 2 or cos_sin.shape[0] < self.max_len):
            raise ValueError("cos_sin is a table with a row for every position that the sequences may come to hold")
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError(f"no path on {self.device}")
        self.requests, self.heads, self.page, self.prefix_len = requests, heads, page, prefix_len
        self.rope = 0 if cos_sin is None else int(cos_sin.shape[1])
        self.width = KV_LORA + self.rope
        self.fp8, self.kv_scale, self.eps, self.sm_scale = fp8, kv_scale, eps, sm_scale
        self.interleaved, self.graph = interleaved, graph
        n_prefix, whole, n_all = -(-prefix_len // page), prefix_len // page, -(-self.max_len // page)
        own = n_all - whole
        self.kv_rows = (n_prefix + requests * own) * page
        self._refuse(n_prefix, n_all, 0 if cos_sin is None else cos_sin.shape[0])
        if self.device.index is None:         # the device of its tensors, whichever is current at a later call
            self.device = torch.device("cuda", torch.cuda.current_device())
        dev = dict(device=self.device)
        self.norm_w = None if norm_w is None else _operand(norm_w, self.device, torch.bfloat16)
        self.cos_sin = None if cos_sin is None else _operand(cos_sin, self.device, torch.float32)
        # pages: the prefix's, then each request's own from the page that the prefix ends in
        pages = torch.arange(n_prefix + requests * own, dtype=torch.int32)
        self.prefix_table = pages[:max(1, n_prefix)].contiguous().to(self.device)
        table = torch.full((requests, max(1, n_all)), -1, dtype=torch.int32)
        if own:
            table[:, whole:] = pages[n_prefix:].view(requests, own)
        self.block_table = table.to(self.device)
        self.cache = torch.zeros(self.kv_rows, self.width, dtype=torch.uint8 if fp8 else torch.bfloat16, **dev)
        i32 = dict(dtype=torch.int32, device=self.device)
        self.prefix_tokens = torch.tensor([prefix_len], **i32)
        self.prefix_req = torch.zeros(prefix_len, **i32)
        self.prefix_pos = torch.arange(prefix_len, **i32)
        self.seq_len = torch.full((requests,), prefix_len, **i32)
        self.q_req = torch.arange(requests, **i32)
        self.q_pos = self.seq_len - 1
        self.kv_new = torch.zeros(requests, self.width, dtype=torch.bfloat16, **dev)
        self.q = torch.zeros(requests, heads, self.width, dtype=torch.bfloat16, **dev)
        self.out = torch.empty(requests, heads, KV_LORA, dtype=torch.bfloat16, **dev)
        self.lse = torch.empty(requests, heads, dtype=torch.float32, **dev)
        self.ws = torch.empty(max(16, B.dsa_prefix_mla_workspace_size(requests, heads)), dtype=torch.uint8, **dev)
        self.tokens = 0                       # own tokens of every request so far
        self._captured = None

    def _refuse(self, n_prefix: int, n_all: int, positions: int) -> None:
        """What the calls of a step would refuse, before anything is allocated: the entry points
        check a call's sizes and scales before they find that it has nothing to do."""
        scale = (self.kv_scale,) if self.fp8 else ()
        append = B.dsa_latent_append_paged_fp8 if self.fp8 else B.dsa_latent_append_paged
        attend = B.dsa_prefix_mla_decode_paged_fp8 if self.fp8 else B.dsa_prefix_mla_decode_paged
        if self.requests > PREFIX_MAX_QUERIES:
            raise ValueError(f"{self.requests} requests: a step takes at most {PREFIX_MAX_QUERIES}")
        append(None, self.width, None, self.eps, None, positions, int(self.interleaved), None, None, 0, KV_LORA, self.rope,
               None, self.requests, n_all, self.page, None, *scale, self.kv_rows)
        attend(None, None, *scale, self.kv_rows, None, n_prefix, None, None, n_all, self.page, None, None, None, 0,
               self.requests, self.heads, KV_LORA, self.rope, self.sm_scale, None, None, None, 0)

    def _append(self, kv_new, tok_req, tok_pos, table, n_req, q=None, stream=None):
        cs, queries = self.cos_sin, ()
        if q is not None and self.rope:       # rotated in place, behind the latent columns
            queries = (q[..., KV_LORA:], q.stride(0), q.stride(1), self.heads, q)
        shape = (kv_new.stride(0), self.norm_w, self.eps, cs, 0 if cs is None else cs.shape[0],
                 int(self.interleaved), tok_req, tok_pos, kv_new.shape[0], KV_LORA, self.rope, table,
                 n_req, table.shape[-1], self.page)
        if self.fp8:
            B.dsa_latent_append_paged_fp8(kv_new, *shape, self.cache, self.kv_scale, self.kv_rows, *queries,
                                          stream=stream)
        else:
            B.dsa_latent_append_paged(kv_new, *shape, self.cache, self.kv_rows, *queries, stream=stream)

    @staticmethod
    def _check(name: str, x: torch.Tensor, shape) -> None:
        if tuple(x.shape) != shape or x.dtype != torch.bfloat16:
            raise ValueError(f"{name} is {x.dtype} {tuple(x.shape)}, not bfloat16 {shape}")

    @torch.no_grad()
    def fill_prefix(self, kv_new: torch.Tensor, stream=None) -> None:
        """Append the prefix's rows: kv_new bf16 [prefix_len, 512 + rope], as projected. On another
        ``stream`` than the current one it runs behind the current stream's work so far, and the
        current stream's next work behind it."""
        self._check("kv_new", kv_new, (self.prefix_len, self.width))
        if kv_new.device != self.cache.device or kv_new.stride(1) != 1:
            raise ValueError("kv_new must lie on the cache's device, the channels of a row together")
        with torch.cuda.device(self.device):
            here = torch.cuda.current_stream()
            side = here if stream is None else _torch_stream(stream)
            if side.cuda_stream != here.cuda_stream:
                side.wait_stream(here)
            self._append(kv_new, self.prefix_req, self.prefix_pos, self.prefix_table, 1, stream=side)
            if side.cuda_stream != here.cuda_stream:
                here.wait_stream(side)

    def _calls(self, stream=None):
        self._append(self.kv_new, self.q_req, self.q_pos, self.block_table, self.requests, self.q, stream)
        where = (self.prefix_table, self.prefix_table.numel(), self.prefix_tokens, self.block_table,
                 self.block_table.shape[1], self.page, self.seq_len, self.q_req, self.q_pos, self.requests,
                 self.requests, self.heads, KV_LORA, self.rope, self.sm_scale, self.out, self.lse, self.ws,
                 self.ws.numel(), stream)
        if self.fp8:
            B.dsa_prefix_mla_decode_paged_fp8(self.q, self.cache, self.kv_scale, self.kv_rows, *where)
        else:
            B.dsa_prefix_mla_decode_paged(self.q, self.cache, self.kv_rows, *where)

    @torch.no_grad()
    def step(self, kv_new: torch.Tensor, q: torch.Tensor) -> torch.Tensor:
        """One token a request: kv_new bf16 [requests, 512 + rope] as projected, q bf16 [requests,
        heads, 512 + rope] with its last rope columns not yet rotated, both on the device or in
        host memory (which has been read when the call returns). Returns the output [requests,
        heads, 512] (its buffer, overwritten by the next step)."""
        if self.prefix_len + self.tokens >= self.max_len:
            raise ValueError("the requests' pages are full")
        self._check("kv_new", kv_new, tuple(self.kv_new.shape))
        self._check("q", q, tuple(self.q.shape))
        with torch.cuda.device(self.device):
            return self._step(kv_new, q)

    def _step(self, kv_new: torch.Tensor, q: torch.Tensor) -> torch.Tensor:
        for mine, x in ((self.kv_new, kv_new), (self.q, q)):
            # host memory has been read when the call returns (a caller's capture reads it at every replay)
            mine.copy_(x, non_blocking=x.is_cuda or torch.cuda.is_current_stream_capturing())
        self.seq_len += 1
        self.q_pos += 1
        try:
            self._launch()
        except BaseException:
            self.seq_len -= 1                 # the step was not taken: the next one is for the same token
            self.q_pos -= 1
            raise
        self.tokens += 1
        return self.out

    def _launch(self) -> None:
        if not self.graph:
            self._calls()
            return
        if self._captured is None:
            before = self.q.clone()
            self._calls()                                  # sets kernel attributes eagerly
            # the eager step rotated q in place: the replay below starts from what came in
            self.q.copy_(before)
            torch.cuda.synchronize(self.device)
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured):
                self._calls()
            self._captured = captured
        self._captured.replay()
