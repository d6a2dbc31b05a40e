"""Python binding of libhcl with the C ABI's names; torch tensors in, argument marshalling only.

Every function takes CUDA tensors (device memory owned by the caller) and enqueues the
corresponding libhcl call on the current torch stream (or `stream`).  No arithmetic of the
method happens here.  Formats: HCL_BF16 / HCL_FP32 / HCL_FP8SPLIT / HCL_MXFP4.
"""
import contextlib
import ctypes
import math

import torch

from . import _lib
from ._lib import (HCL_BF16, HCL_FP32, HCL_FP8SPLIT, HCL_MXFP4, check, hcl_kv_t, hcl_paged_kv_t,
                   lib)

__all__ = ["KV", "hcl_csa_compress", "hcl_hca_compress", "hcl_quant_kv_fp8", "hcl_quant_mxfp4",
           "hcl_csa_index_scores", "hcl_csa_topk", "hcl_csa_sparse_attn", "hcl_hca_dense_attn",
           "hcl_csa_decode_step", "hcl_cache_append", "PagedKV", "hcl_page_plan", "hcl_paged_write",
           "hcl_paged_attn", "hcl_paged_attn_f32", "paged_attn_workspace_bytes", "hcl_selftest_bounded_wait", "HCL_BF16",
           "HCL_FP32", "HCL_FP8SPLIT", "HCL_MXFP4"]


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libhcl takes CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("libhcl takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


class KV:
    """A KV store (see hcl_kv_t): bf16 rows [B, cap, d], or split rows: e4m3 codes
    [B, cap, d/2] (uint8), fp32 scale [B, cap], bf16 RoPE half [B, cap, d/2]."""

    def __init__(self, data, scale=None, rope=None):
        self.data, self.scale, self.rope = data, scale, rope
        self.fmt = HCL_FP8SPLIT if scale is not None else HCL_BF16
        self.cap = data.shape[1]
        self._c = hcl_kv_t(self.fmt, self.cap, _ptr(data).value, None if scale is None else _ptr(scale).value,
                           None if rope is None else _ptr(rope).value)

    def ref(self):
        return ctypes.byref(self._c)


def _fmt_of(t):
    return HCL_FP32 if t.dtype == torch.float32 else HCL_BF16


def hcl_csa_compress(kv, gate, bias, m, out, entry_begin=0, entry_end=None, gamma=None,
                     eps=1e-6, stream=None):
    """gamma (fp32 [d] CUDA tensor): RMSNorm each pooled entry (x / rms(x) * gamma)."""
    B, L, d = kv.shape
    if entry_end is None:
        entry_end = -(-L // m)
    check(lib().hcl_csa_compress(_ptr(kv), _ptr(gate), _ptr(bias), B, L, d, m, entry_begin,
                                 entry_end, _ptr(out), _fmt_of(out), out.shape[1], _ptr(gamma),
                                 eps, _stream(stream)))
    return out


def hcl_hca_compress(kv, gate, bias, m, out, entry_begin=0, entry_end=None, gamma=None,
                     eps=1e-6, stream=None):
    B, L, d = kv.shape
    if entry_end is None:
        entry_end = -(-L // m)
    check(lib().hcl_hca_compress(_ptr(kv), _ptr(gate), _ptr(bias), B, L, d, m, entry_begin,
                                 entry_end, _ptr(out), _fmt_of(out), out.shape[1], _ptr(gamma),
                                 eps, _stream(stream)))
    return out


def hcl_quant_kv_fp8(kv, nope, scale, rope, stream=None):
    d = kv.shape[-1]
    rows = kv.numel() // d
    check(lib().hcl_quant_kv_fp8(_ptr(kv), rows, d, _ptr(nope), _ptr(scale), _ptr(rope),
                                 _stream(stream)))


def hcl_quant_mxfp4(x, packed, sf, stream=None):
    cols = x.shape[-1]
    rows = x.numel() // cols
    check(lib().hcl_quant_mxfp4(_ptr(x), rows, cols, _ptr(packed), _ptr(sf), _stream(stream)))


def hcl_csa_index_scores(op_fmt, qI, w, kI, q_pos, m, scores, Nc=None, qI_sf=None, kI_sf=None,
                         status=None, stream=None):
    B, Tq, HI = w.shape
    dI = qI.shape[-1] * (2 if op_fmt == HCL_MXFP4 else 1)
    cap = kI.shape[1]
    Nc = cap if Nc is None else Nc
    check(lib().hcl_csa_index_scores(op_fmt, _ptr(qI), _ptr(qI_sf), _ptr(w), _ptr(kI), _ptr(kI_sf),
                                     B, Tq, HI, dI, Nc, cap, _ptr(q_pos), m, _ptr(scores),
                                     _fmt_of(scores), _ptr(status), _stream(stream)))
    return scores


def hcl_csa_topk(scores, q_pos, m, k, idx, status=None, stream=None):
    B, Tq, Nc = scores.shape
    fmt = _fmt_of(scores)
    wsb = lib().hcl_csa_topk_workspace_bytes(B, Tq, Nc, k, fmt)
    ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=scores.device) if wsb else None
    check(lib().hcl_csa_topk(_ptr(scores), fmt, B, Tq, Nc, _ptr(q_pos), m, k, _ptr(idx), _ptr(ws),
                             wsb, _ptr(status), _stream(stream)))
    return idx


def csa_sparse_attn_workspace_bytes(B, Tq, H, k, W):
    return lib().hcl_csa_sparse_attn_workspace_bytes(B, Tq, H, k, W)


def hcl_csa_sparse_attn(q, kvc: KV, Nc, idx, raw: KV, L, W, q_pos, out, lse=None, scale=None,
                        sink=None, ws=None, status=None, q_gamma=None, q_eps=1e-6, stream=None):
    B, Tq, H, d = q.shape
    k = idx.shape[-1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    need = csa_sparse_attn_workspace_bytes(B, Tq, H, k, W)
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    check(lib().hcl_csa_sparse_attn(_ptr(q), B, Tq, H, d, kvc.ref(), Nc, _ptr(idx), k, raw.ref(),
                                    L, W, _ptr(q_pos), scale, _ptr(sink), _ptr(q_gamma), q_eps,
                                    _ptr(out), _ptr(lse),
                                    _ptr(ws), 0 if ws is None else ws.numel(), _ptr(status),
                                    _stream(stream)))
    return out


def hca_dense_attn_workspace_bytes(B, Tq, H, Nh, W):
    return lib().hcl_hca_dense_attn_workspace_bytes(B, Tq, H, Nh, W)


def hcl_hca_dense_attn(q, kvh: KV, Nh, mh, raw: KV, L, W, q_pos, out, lse=None, scale=None,
                       sink=None, ws=None, status=None, q_gamma=None, q_eps=1e-6, stream=None):
    B, Tq, H, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    need = hca_dense_attn_workspace_bytes(B, Tq, H, Nh, W)
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    check(lib().hcl_hca_dense_attn(_ptr(q), B, Tq, H, d, kvh.ref(), Nh, mh, raw.ref(), L, W,
                                   _ptr(q_pos), scale, _ptr(sink), _ptr(q_gamma), q_eps, _ptr(out),
                                   _ptr(lse), _ptr(ws),
                                   0 if ws is None else ws.numel(), _ptr(status), _stream(stream)))
    return out


def decode_step_workspace_bytes(B, H, HI, Nc, k, W, op_fmt, score_fmt):
    return lib().hcl_csa_decode_step_workspace_bytes(B, H, HI, Nc, k, W, op_fmt, score_fmt)


def hcl_csa_decode_step(q, qI, w, op_fmt, kI, kvc: KV, Nc, m, k, raw: KV, L, W, q_pos, out,
                        score_fmt=HCL_FP32, kI_sf=None, lse=None, idx_out=None, scale=None,
                        sink=None, ws=None, status=None, q_gamma=None, q_eps=1e-6, stream=None):
    """One CSA decode step (Tq = 1): MXFP4-quantise qI (MXFP4 keys only), score, top-k, attend."""
    B, _, H, d = q.shape
    HI, dI = qI.shape[-2], qI.shape[-1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    need = decode_step_workspace_bytes(B, H, HI, Nc, k, W, op_fmt, score_fmt)
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    check(lib().hcl_csa_decode_step(_ptr(q), _ptr(qI), _ptr(w), op_fmt, _ptr(kI), _ptr(kI_sf),
                                    kI.shape[1], score_fmt, B, H, HI, dI, d, kvc.ref(), Nc, m, k,
                                    raw.ref(), L, W, _ptr(q_pos), scale, _ptr(sink), _ptr(q_gamma),
                                    q_eps, _ptr(out), _ptr(lse), _ptr(idx_out), _ptr(ws), ws.numel(),
                                    _ptr(status),
                                    _stream(stream)))
    return out


def hcl_cache_append(kv_new, gate_new, t_new, stage_kv, stage_gate, raw: KV, kvc: KV = None,
                     bias_csa=None, m=4, kI_new=None, kI=None, kI_sf=None, kvh: KV = None,
                     bias_hca=None, mh=128, gamma=None, eps=1e-6, stream=None):
    """Append one token per sequence (kv_new / gate_new bf16 [B, d], t_new int32 [B]) to one
    layer's cache: staging rings, raw window store, and the CSA (kvc, index keys kI: bf16
    [B, cap, dI], or MXFP4 packed uint8 [B, cap, dI/2] with kI_sf) or HCA (kvh) entry it
    completes."""
    B, d = kv_new.shape
    kI_fmt = HCL_MXFP4 if kI_sf is not None else HCL_BF16
    dI = 0 if kI is None else (kI.shape[-1] * (2 if kI_fmt == HCL_MXFP4 else 1))
    check(lib().hcl_cache_append(_ptr(kv_new), _ptr(gate_new), _ptr(kI_new), _ptr(t_new), B, d, dI,
                                 _ptr(stage_kv), _ptr(stage_gate), stage_kv.shape[1], raw.ref(),
                                 None if kvc is None else kvc.ref(), _ptr(bias_csa), m, kI_fmt,
                                 _ptr(kI), _ptr(kI_sf), 0 if kI is None else kI.shape[1],
                                 None if kvh is None else kvh.ref(), _ptr(bias_hca), mh,
                                 _ptr(gamma), eps, None, _stream(stream)))


def hcl_cp_candidates(scores, idx, e0, cand_scores, cand_idx, status=None, stream=None):
    """Local top-k (idx [B, 1, k]) over a rank's scores [B, 1, Nc_local] -> (fp32 score, global
    index) candidates [B, k]."""
    B, _, Nc_local = scores.shape
    k = idx.shape[-1]
    check(lib().hcl_cp_candidates(_ptr(scores), _fmt_of(scores), _ptr(idx), B, Nc_local, k, e0,
                                  _ptr(cand_scores), _ptr(cand_idx), _ptr(status), _stream(stream)))


def hcl_cp_own(pos, gathered_idx, e0, e1, sel_out, own_out, stream=None):
    """pos [B, 1, k] selected positions in the gathered list gathered_idx [B, n] -> global
    selection sel_out [B, 1, k] and this rank's local share own_out [B, 1, k]."""
    B, n = gathered_idx.shape
    k = pos.shape[-1]
    check(lib().hcl_cp_own(_ptr(pos), _ptr(gathered_idx), B, n, k, e0, e1, _ptr(sel_out),
                           _ptr(own_out), _stream(stream)))


def hcl_lse_merge(o_parts, lse_parts, out, lse_out=None, sink=None, stream=None):
    """o_parts bf16 or fp32 [G, B, Tq, H, d], lse_parts fp32 [G, B, Tq, H] -> out bf16 [B, Tq, H, d]."""
    G = o_parts.shape[0]
    H, d = o_parts.shape[-2], o_parts.shape[-1]
    rows = lse_parts[0].numel()
    if o_parts.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("o_parts must be bf16 or fp32")
    merge = lib().hcl_lse_merge_f32 if o_parts.dtype == torch.float32 else lib().hcl_lse_merge
    check(merge(_ptr(o_parts), _ptr(lse_parts), G, rows, d, H, _ptr(sink), _ptr(out), _ptr(lse_out),
                _stream(stream)))


# The paged cache's calls are made once per layer and step, on small batches too, so their checks
# are kept to a few attribute reads per tensor.


def _stream_on(stream, dev):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _i32(t, name, dev, n=None):
    """The address of a contiguous int32 tensor on device `dev` (n: its element count)."""
    if t.dtype is not torch.int32 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current CUDA device")
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, not {t.numel()}")
    return t.data_ptr()


def _dense(t, name, dev, dtype, shape):
    """The address of a contiguous tensor of the given type and shape on device `dev`."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current CUDA device")
    return t.data_ptr()


def _rows(t, name, dev, heads, d):
    """(address, token stride in elements) of bf16 rows [T, heads, d] whose heads lie together:
    a whole tensor, or a slice of wider rows such as a fused projection's output."""
    if t.dtype is not torch.bfloat16 or t.dim() != 3 or t.shape[1:] != (heads, d):
        raise ValueError(f"{name} must be bf16 [T, {heads}, {d}]")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current CUDA device")
    s = t.stride()
    if s[2] != 1 or (heads > 1 and s[1] != d):
        raise ValueError(f"{name}: the heads of a token must lie together")
    return t.data_ptr(), (s[0] if t.shape[0] > 1 else heads * d)


class PagedKV:
    """A paged 8-bit store (see hcl_paged_kv_t): E4M3 codes k, v uint8 [n_pages, Hkv, page, d]
    and fp32 scales [n_pages, Hkv].  Without v each row is both key and value."""

    def __init__(self, k, k_scale, v=None, v_scale=None):
        if (v is None) != (v_scale is None):
            raise ValueError("v and v_scale go together")
        if k.dim() != 4:
            raise ValueError("k must be codes [n_pages, Hkv, page, d]")
        n, Hkv, page, d = k.shape
        dev = torch.cuda.current_device()
        ptr = []
        for name, codes, scale in (("k", k, k_scale), ("v", v, v_scale)):
            ptr.append(None if codes is None else _dense(codes, name, dev, torch.uint8, k.shape))
            ptr.append(None if codes is None else
                       _dense(scale, name + "_scale", dev, torch.float32, (n, Hkv)))
        self.k, self.k_scale, self.v, self.v_scale = k, k_scale, v, v_scale
        self.n_pages, self.Hkv, self.page, self.d, self.dev = n, Hkv, page, d, dev
        self._c = hcl_paged_kv_t(page, n, Hkv, d, ptr[0], ptr[2], ptr[1], ptr[3])
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, n_pages, Hkv, page, d, shared=False, device="cuda"):
        """A new store; shared: rows are both key and value."""
        def plane():
            return (torch.empty(n_pages, Hkv, page, d, dtype=torch.uint8, device=device),
                    torch.ones(n_pages, Hkv, dtype=torch.float32, device=device))
        return cls(*plane()) if shared else cls(*plane(), *plane())

    def ref(self, dev):
        if self.dev != dev:
            raise ValueError("the store must be on the current CUDA device")
        return self._ref


def hcl_page_plan(keep, new_len, seq_len, table, free_list, n_free, page, cu_new, pos, slot,
                  status=None, stream=None):
    """Block tables and slot maps of one step, in place (see hcl.h): keep, new_len, seq_len int32
    [B]; table int32 [B, max_pages]; free_list int32 [n_pages], n_free int32 [1]; cu_new int32
    [B + 1]; pos, slot int32 [T]."""
    B, max_pages = table.shape
    T = slot.numel()
    dev = torch.cuda.current_device()
    check(lib().hcl_page_plan(
        _i32(keep, "keep", dev, B), _i32(new_len, "new_len", dev, B), B, page,
        _i32(seq_len, "seq_len", dev, B), _i32(table, "table", dev), max_pages,
        _i32(free_list, "free_list", dev), free_list.numel(), _i32(n_free, "n_free", dev, 1), T,
        _i32(cu_new, "cu_new", dev, B + 1), _i32(pos, "pos", dev, T), _i32(slot, "slot", dev),
        None if status is None else _i32(status, "status", dev), _stream_on(stream, dev)))


def hcl_paged_write(k_new, v_new, slot, store: PagedKV, status=None, stream=None):
    """Quantise new rows (bf16 [T, Hkv, d]; v_new None for a store without v) into their slots."""
    T = slot.numel()
    dev = torch.cuda.current_device()
    k, ks = _rows(k_new, "k_new", dev, store.Hkv, store.d)
    v, vs = (None, 0) if v_new is None else _rows(v_new, "v_new", dev, store.Hkv, store.d)
    if k_new.shape[0] != T or (v_new is not None and v_new.shape[0] != T):
        raise ValueError("k_new, v_new and slot must have as many rows")
    check(lib().hcl_paged_write(k, ks, v, vs, _i32(slot, "slot", dev), T, store.ref(dev),
                                None if status is None else _i32(status, "status", dev),
                                _stream_on(stream, dev)))


def paged_attn_workspace_bytes(T, H, Hkv, d):
    return lib().hcl_paged_attn_workspace_bytes(T, H, Hkv, d)


def hcl_paged_attn(q, cu_q, q_start, store: PagedKV, table, kv_len, out, lse=None, m=1, W=0,
                   max_q=None, scale=None, sink=None, ws=None, status=None, stream=None):
    """Attention of ragged queries (bf16 [T, H, d], request b's rows cu_q[b] .. cu_q[b + 1] - 1,
    the first at position q_start[b]) over the pages that table int32 [B, max_pages] lists."""
    return _paged_attn(lib().hcl_paged_attn, torch.bfloat16, q, cu_q, q_start, store, table, kv_len, out, lse, m, W,
                       max_q, scale, sink, ws, status, stream)


def hcl_paged_attn_f32(q, cu_q, q_start, store: PagedKV, table, kv_len, out, lse=None, m=1, W=0,
                       max_q=None, scale=None, sink=None, ws=None, status=None, stream=None):
    """hcl_paged_attn with out fp32 [T, H, d]: a part to merge with others (hcl_lse_merge)."""
    return _paged_attn(lib().hcl_paged_attn_f32, torch.float32, q, cu_q, q_start, store, table, kv_len, out, lse, m, W,
                       max_q, scale, sink, ws, status, stream)


def _paged_attn(call, out_dtype, q, cu_q, q_start, store, table, kv_len, out, lse, m, W, max_q, scale, sink, ws,
                status, stream):
    T, H, d = q.shape
    B, max_pages = table.shape
    dev = torch.cuda.current_device()
    qp, qs = _rows(q, "q", dev, H, store.d)
    if ws is None:
        need = paged_attn_workspace_bytes(T, H, store.Hkv, d)
        if need:
            # (from the launching stream's pool: a block of another stream's may still be in use there)
            with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
                ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws must be contiguous, on the current CUDA device")
    check(call(
        qp, qs, T, H, _i32(cu_q, "cu_q", dev, B + 1), _i32(q_start, "q_start", dev, B), B,
        store.ref(dev), _i32(table, "table", dev), max_pages, _i32(kv_len, "kv_len", dev, B),
        T if max_q is None else max_q, m, W, 1.0 / math.sqrt(d) if scale is None else scale,
        None if sink is None else _dense(sink, "sink", dev, torch.float32, (H,)),
        _dense(out, "out", dev, out_dtype, q.shape),
        None if lse is None else _dense(lse, "lse", dev, torch.float32, (T, H)),
        None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel() * ws.element_size(),
        None if status is None else _i32(status, "status", dev), _stream_on(stream, dev)))
    return out


def hcl_selftest_bounded_wait(status, limit_us=1000, stream=None):
    check(lib().hcl_selftest_bounded_wait(_ptr(status), limit_us, _stream(stream)))
