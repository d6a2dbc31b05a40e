"""Composition of the hot-path calls for the three workload shapes, on caller-provided CUDA
tensors: a CSA decode step, an HCA layer (prefill chunk or decode), and a CSA/HCA layer pair
over a chunked prefill; and for ragged batches the page bookkeeping of a batch and the layers over
its paged 8-bit caches.  Owns the intermediate buffers (scores, indices, workspaces) so a step
allocates nothing; every step is a sequence of libhcl calls on one stream."""
import contextlib
import math

import torch

from . import api
from .api import HCL_BF16, HCL_FP32, HCL_MXFP4, KV


class CsaDecode:
    """One query per sequence: [quantise q_I] -> index scores -> top-k -> sparse attention.

    q [B,1,H,d] bf16; qI [B,1,HI,dI] bf16; w [B,1,HI] fp32; keys: bf16 [B,cap,dI], or MXFP4
    packed [B,cap,dI/2] + kI_sf [B,cap,dI/32]; kvc / raw: api.KV stores; q_pos [B,1] int32."""

    def __init__(self, q, qI, w, kI, kvc: KV, Nc, raw: KV, L, W, q_pos, m=4, k=1024,
                 op_fmt=HCL_BF16, score_fmt=HCL_FP32, kI_sf=None, sink=None, q_gamma=None,
                 q_eps=1e-6):
        self.q, self.qI, self.w, self.kI, self.kI_sf = q, qI, w, kI, kI_sf
        self.q_gamma, self.q_eps = q_gamma, q_eps
        self.kvc, self.raw, self.Nc, self.L, self.W, self.q_pos = kvc, raw, Nc, L, W, q_pos
        self.m, self.k, self.op_fmt, self.score_fmt, self.sink = m, k, op_fmt, score_fmt, sink
        B, _, H, d = q.shape
        HI, dI = qI.shape[-2], qI.shape[-1]
        dev = q.device
        self.B, self.H, self.HI = B, H, HI
        if op_fmt == HCL_MXFP4:
            self.qI_packed = torch.empty(B, 1, HI, dI // 2, dtype=torch.uint8, device=dev)
            self.qI_sf = torch.empty(B, 1, HI, dI // 32, dtype=torch.uint8, device=dev)
        sdt = torch.bfloat16 if score_fmt == HCL_BF16 else torch.float32
        self.scores = torch.empty(B, 1, Nc, dtype=sdt, device=dev)
        self.idx = torch.empty(B, 1, k, dtype=torch.int32, device=dev)
        self.out = torch.empty(B, 1, H, d, dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty(B, 1, H, dtype=torch.float32, device=dev)
        n = api.csa_sparse_attn_workspace_bytes(B, 1, H, k, W)
        self.attn_ws = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
        n = api.decode_step_workspace_bytes(B, H, HI, Nc, k, W, op_fmt, score_fmt)
        self.step_ws = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def launches_per_step(self, fused=True):
        """Kernels one step launches: the fused C-ABI step as the library reports it, or with
        step_parts() indexer, top-k, attention (+ split merge) and, for MXFP4 keys, a separate
        q_I quantisation."""
        if fused:
            return api.lib().hcl_csa_decode_step_kernels(self.B, self.H, self.HI, self.Nc, self.k,
                                                         self.W, self.op_fmt, self.score_fmt,
                                                         self.kvc.fmt)
        n = 3 + (1 if self.op_fmt == HCL_MXFP4 else 0)
        need = api.csa_sparse_attn_workspace_bytes(self.B, 1, self.H, self.k, self.W)
        return n + (1 if need else 0)

    def step_parts(self, stream=None):
        """The four calls one by one, keeping the intermediates (scores, idx)."""
        qI, qI_sf = self.qI, None
        if self.op_fmt == HCL_MXFP4:
            api.hcl_quant_mxfp4(self.qI, self.qI_packed, self.qI_sf, stream=stream)
            qI, qI_sf = self.qI_packed, self.qI_sf
        api.hcl_csa_index_scores(self.op_fmt, qI, self.w, self.kI, self.q_pos, self.m, self.scores,
                                 Nc=self.Nc, qI_sf=qI_sf, kI_sf=self.kI_sf, status=self.status,
                                 stream=stream)
        api.hcl_csa_topk(self.scores, self.q_pos, self.m, self.k, self.idx, status=self.status,
                         stream=stream)
        api.hcl_csa_sparse_attn(self.q, self.kvc, self.Nc, self.idx, self.raw, self.L, self.W,
                                self.q_pos, self.out, lse=self.lse, sink=self.sink,
                                ws=self.attn_ws, status=self.status, q_gamma=self.q_gamma,
                                q_eps=self.q_eps, stream=stream)
        return self.out

    def step(self, stream=None):
        """The fused C-ABI decode step (same kernels, one call)."""
        api.hcl_csa_decode_step(self.q, self.qI, self.w, self.op_fmt, self.kI, self.kvc, self.Nc,
                                self.m, self.k, self.raw, self.L, self.W, self.q_pos, self.out,
                                score_fmt=self.score_fmt, kI_sf=self.kI_sf, lse=self.lse,
                                idx_out=self.idx, sink=self.sink, ws=self.step_ws,
                                status=self.status, q_gamma=self.q_gamma, q_eps=self.q_eps,
                                stream=stream)
        return self.out


class HcaLayer:
    """HCA attention over the compressed entries plus the raw window for Tq queries per
    sequence (a prefill chunk, or Tq = 1 for decode); optionally compresses entries first."""

    def __init__(self, q, kvh: KV, Nh, mh, raw: KV, L, W, q_pos, sink=None, q_gamma=None,
                 q_eps=1e-6):
        self.q, self.kvh, self.Nh, self.mh, self.raw, self.L, self.W = q, kvh, Nh, mh, raw, L, W
        self.q_pos, self.sink, self.q_gamma, self.q_eps = q_pos, sink, q_gamma, q_eps
        B, Tq, H, d = q.shape
        self.out = torch.empty(B, Tq, H, d, dtype=torch.bfloat16, device=q.device)
        self.lse = torch.empty(B, Tq, H, dtype=torch.float32, device=q.device)
        n = api.hca_dense_attn_workspace_bytes(B, Tq, H, Nh, W)
        self.ws = torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)
        self.status = torch.zeros(1, dtype=torch.int32, device=q.device)

    def step(self, stream=None):
        api.hcl_hca_dense_attn(self.q, self.kvh, self.Nh, self.mh, self.raw, self.L, self.W,
                               self.q_pos, self.out, lse=self.lse, sink=self.sink, ws=self.ws,
                               status=self.status, q_gamma=self.q_gamma, q_eps=self.q_eps,
                               stream=stream)
        return self.out


class PairPrefill:
    """Alternating CSA/HCA layer pair over a chunk of new tokens appended to a context:
    compress the new CSA and HCA entries, score all CSA entries for every new query, top-k,
    CSA sparse attention, HCA dense attention.

    raw_kv / gate [1, L, d] bf16 (context + chunk); entries before the chunk are expected in
    comp_csa / comp_hca already (bf16 [1, cap, d]); qI [1,Tq,HI,dI] bf16, w [1,Tq,HI];
    q_csa / q_hca [1,Tq,H,d]; kI [1,Nc,dI] bf16."""

    def __init__(self, raw_kv, gate, bias_csa, bias_hca, comp_csa, comp_hca, q_csa, q_hca, qI, w,
                 kI, q_pos, chunk_begin, m=4, mh=128, k=1024, W=128, score_fmt=HCL_BF16):
        self.raw_kv, self.gate, self.bias_csa, self.bias_hca = raw_kv, gate, bias_csa, bias_hca
        self.comp_csa, self.comp_hca, self.q_csa, self.q_hca = comp_csa, comp_hca, q_csa, q_hca
        self.qI, self.w, self.kI, self.q_pos = qI, w, kI, q_pos
        self.m, self.mh, self.k, self.W, self.score_fmt = m, mh, k, W, score_fmt
        B, L, d = raw_kv.shape
        Tq, H = q_csa.shape[1], q_csa.shape[2]
        self.L = L
        self.Nc = -(-L // m)
        self.Nh = -(-L // mh)
        self.csa_begin = chunk_begin // m
        self.hca_begin = chunk_begin // mh
        dev = raw_kv.device
        sdt = torch.bfloat16 if score_fmt == HCL_BF16 else torch.float32
        self.scores = torch.empty(B, Tq, self.Nc, dtype=sdt, device=dev)
        self.idx = torch.empty(B, Tq, k, dtype=torch.int32, device=dev)
        self.raw = KV(raw_kv)
        self.kvc = KV(comp_csa)
        self.kvh = KV(comp_hca)
        self.out_csa = torch.empty(B, Tq, H, d, dtype=torch.bfloat16, device=dev)
        self.lse_csa = torch.empty(B, Tq, H, dtype=torch.float32, device=dev)
        n = api.csa_sparse_attn_workspace_bytes(B, Tq, H, k, W)
        self.ws_csa = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
        self.hca = HcaLayer(q_hca, self.kvh, self.Nh, mh, self.raw, L, W, q_pos)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def compress_prior(self, stream=None):
        """Entries of the context before the chunk (set-up, not part of a step)."""
        if self.csa_begin:
            api.hcl_csa_compress(self.raw_kv, self.gate, self.bias_csa, self.m, self.comp_csa,
                                 0, self.csa_begin, stream=stream)
        if self.hca_begin:
            api.hcl_hca_compress(self.raw_kv, self.gate, self.bias_hca, self.mh, self.comp_hca,
                                 0, self.hca_begin, stream=stream)

    def step(self, stream=None):
        api.hcl_csa_compress(self.raw_kv, self.gate, self.bias_csa, self.m, self.comp_csa,
                             self.csa_begin, self.Nc, stream=stream)
        api.hcl_hca_compress(self.raw_kv, self.gate, self.bias_hca, self.mh, self.comp_hca,
                             self.hca_begin, self.Nh, stream=stream)
        api.hcl_csa_index_scores(HCL_BF16, self.qI, self.w, self.kI, self.q_pos, self.m,
                                 self.scores, Nc=self.Nc, status=self.status, stream=stream)
        api.hcl_csa_topk(self.scores, self.q_pos, self.m, self.k, self.idx, status=self.status,
                         stream=stream)
        api.hcl_csa_sparse_attn(self.q_csa, self.kvc, self.Nc, self.idx, self.raw, self.L, self.W,
                                self.q_pos, self.out_csa, lse=self.lse_csa, ws=self.ws_csa,
                                status=self.status, stream=stream)
        self.hca.step(stream=stream)
        return self.out_csa, self.hca.out

    def launches_per_step(self):
        n = 6
        if api.csa_sparse_attn_workspace_bytes(*self.idx.shape[:2], self.q_csa.shape[2], self.k, self.W):
            n += 1
        if api.hca_dense_attn_workspace_bytes(*self.q_hca.shape[:3], self.Nh, self.W):
            n += 1
        return n


class PagedBatch:
    """The page bookkeeping of a ragged batch, shared by all layers whose caches hold the same rows:
    block tables, free pages and, for each step, slots and positions of the new rows.

    B requests of up to max_pages pages of `page` rows, n_pages pages in all; T: the most new rows
    of a step.  Nothing here reads the device back, so a step can be captured and replayed."""

    def __init__(self, B, page, max_pages, n_pages, T, device="cuda"):
        def i32(*shape, value=0):
            return torch.full(shape, value, dtype=torch.int32, device=device)

        self.B, self.page, self.T = B, page, T
        self.seq_len, self.start, self._keep, self._zero = i32(B), i32(B), i32(B), i32(1)
        self.table = i32(B, max_pages, value=-1)
        self.free_list = torch.arange(n_pages - 1, -1, -1, dtype=torch.int32, device=device)
        self.n_free = i32(1, value=n_pages)
        self.cu_new, self.pos, self.slot = i32(B + 1), i32(T), i32(T)
        self.status = i32(1)

    def plan(self, new_len, keep=None, stream=None):
        """One step: of each request keep[b] rows stay (default: all; 0 for a new request in the
        row) and new_len[b] rows (int32 [B]) are added.  Afterwards start holds the first new
        row's position, slot and pos the new rows' places (-1 behind the last), seq_len the
        lengths.  The status word has HCL_ERR_NO_PAGES where a request did not get its rows, and
        HCL_ERR_DEVICE_FAULT where keep was out of range: it counts as the nearest length that the
        request can keep."""
        with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
            if keep is None:
                self.start.copy_(self.seq_len)
            else:
                self._keep.copy_(keep)
                torch.clamp(self._keep, min=self._zero, max=self.seq_len, out=self.start)
        api.hcl_page_plan(self.start if keep is None else self._keep, new_len, self.seq_len, self.table,
                          self.free_list, self.n_free, self.page, self.cu_new, self.pos, self.slot,
                          status=self.status, stream=stream)


class PagedAttnLayer:
    """One attention layer over a paged 8-bit cache: the step's new rows are written, then its
    queries attend (causal; with W only over the last W rows; with m over entries of m tokens).

    shared: rows are both key and value (H query heads on Hkv of them).  max_T: the most query rows
    of a call (default: the batch's T).  The workspace is the layer's: two calls of attend on one
    layer must not overlap."""

    def __init__(self, batch: PagedBatch, n_pages, H, Hkv, d, shared=False, m=1, W=0, sink=None,
                 device="cuda", max_T=None):
        self.batch, self.m, self.W, self.sink, self.H = batch, m, W, sink, H
        self.store = api.PagedKV.empty(n_pages, Hkv, batch.page, d, shared=shared, device=device)
        n = api.paged_attn_workspace_bytes(batch.T if max_T is None else max_T, H, Hkv, d)
        self.ws = torch.empty(max(n, 16), dtype=torch.uint8, device=device)

    def write(self, k_new, v_new=None, stream=None):
        """k_new, v_new bf16 [T, Hkv, d], the rows of the batch's last plan."""
        api.hcl_paged_write(k_new, v_new, self.batch.slot, self.store, status=self.batch.status,
                            stream=stream)

    def attend(self, q, out, lse=None, max_q=None, cu_q=None, q_start=None, sink=None, stream=None):
        """q bf16 [T, H, d]: the plan's new rows, unless cu_q and q_start say otherwise.  out bf16, or
        fp32 (a part that hcl_lse_merge joins with others)."""
        b = self.batch
        attn = api.hcl_paged_attn_f32 if out.dtype == torch.float32 else api.hcl_paged_attn
        return attn(q, b.cu_new if cu_q is None else cu_q, b.start if q_start is None else q_start,
                    self.store, b.table, b.seq_len, out, lse=lse, m=self.m, W=self.W, max_q=max_q,
                    sink=self.sink if sink is None else sink, ws=self.ws, status=b.status,
                    stream=stream)

    def step(self, q, k_new, v_new, out, lse=None, max_q=None, stream=None):
        self.write(k_new, v_new, stream=stream)
        return self.attend(q, out, lse=lse, max_q=max_q, stream=stream)


class PagedHcaLayer:
    """HCA attention of a ragged batch over two paged 8-bit caches: the compressed entries (mh
    tokens each, dense) and the raw rows (a sliding window of W), whose partial results merge by
    log-sum-exp with the sink.  Rows are both key and value, one for all H heads.

    raw and entries are PagedBatch's, planned for tokens and for completed entries; the rows of
    both are written with raw_layer.write and entry_layer.write before attend.  The workspaces and
    partial results are the layer's: two calls of attend on one layer must not overlap."""

    def __init__(self, raw: PagedBatch, entries: PagedBatch, n_raw_pages, n_entry_pages, H, d, mh=128,
                 W=128, sink=None, device="cuda"):
        self.raw, self.entries, self.sink = raw, entries, sink
        self.raw_layer = PagedAttnLayer(raw, n_raw_pages, H, 1, d, shared=True, W=W, device=device)
        # (its queries are the raw batch's)
        self.entry_layer = PagedAttnLayer(entries, n_entry_pages, H, 1, d, shared=True, m=mh,
                                          device=device, max_T=raw.T)
        # (fp32: the parts may cancel, and out is rounded once)
        self.o_parts = torch.zeros(2, raw.T, H, d, dtype=torch.float32, device=device)
        self.lse_parts = torch.empty(2, raw.T, H, dtype=torch.float32, device=device)

    def attend(self, q, out, lse=None, max_q=None, stream=None):
        """q bf16 [T, H, d], the raw batch's new rows (T: its capacity).  Rows of out behind the
        last request's become zeros."""
        b = self.raw
        # rows that belong to no request, or to one only in an earlier step, weigh nothing
        with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
            self.lse_parts.fill_(-math.inf)
        for i, layer in enumerate((self.entry_layer, self.raw_layer)):
            layer.attend(q, self.o_parts[i], lse=self.lse_parts[i], max_q=max_q, cu_q=b.cu_new,
                         q_start=b.start, stream=stream)
        api.hcl_lse_merge(self.o_parts, self.lse_parts, out, lse_out=lse, sink=self.sink, stream=stream)
        return out
