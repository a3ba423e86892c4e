"""The operators of a decode block around the routed layer, on torch tensors:
the fused block norm, the paged key-value cache (append and attention) and the
linear product with 4-bit weights; and :class:`DecodeBlock`, which runs them
together with a :class:`~.layer.MoELayer`.  Marshalling only: every computation
runs in libmoe.so (formulas, limits and errors in include/moe.h).

Tensors lie on the current device.  ``stream`` is a torch stream or a
cudaStream_t (default: the current stream); outputs that a call makes belong to
that stream.  Wrong shapes, types or strides are ValueErrors; what the library
refuses is a :class:`~.moe.MoeError`.
"""
from __future__ import annotations

import torch

from . import moe
from .layer import MoELayer, _ptr, _stream

_DT = {torch.bfloat16: moe.MOE_DT_BF16, torch.float32: moe.MOE_DT_F32,
       torch.float16: moe.MOE_DT_F16, torch.float8_e4m3fn: moe.MOE_DT_E4M3}
_KINDS = {"rms": moe.MOE_NORM_RMS, "layer": moe.MOE_NORM_LAYER}
_FORMATS = {"u4": moe.MOE_W4_U4, "e2m1": moe.MOE_W4_E2M1}
_device, _current = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _handle(stream) -> int:
    """cudaStream_t of `stream`, of the current stream for None."""
    return _current(_device()) if stream is None else _stream(stream)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """An output that belongs to the stream that will write it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(s):
        return torch.empty(shape, dtype=dtype, device=device)


# The checks raise with a text that is put together only then: a call's own
# time is a few microseconds.
def _rows(t: torch.Tensor, T: int, H: int, name: str) -> int:
    """t as T contiguous rows of H values: their stride."""
    if t.shape != (T, H) or not t.is_cuda:
        raise ValueError(f"{name}: [{T}, {H}] on the GPU is wanted, got {tuple(t.shape)} on {t.device}")
    row, one = t.stride()
    if one != 1 and H != 1:
        raise ValueError(f"{name}: contiguous rows are wanted")
    return row if T > 1 or row >= H else H


def _vector(t: torch.Tensor, n: int, dtype, name: str) -> int:
    if t.shape != (n,) or t.dtype is not dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous [{n}] of {dtype} on the GPU is wanted")
    return t.data_ptr()


def _ints(t: torch.Tensor, dims: int, name: str) -> None:
    if t.dtype is not torch.int32 or t.dim() != dims or not t.is_cuda or (
            t.stride(-1) != 1 and t.numel() > 1 and t.shape[-1] > 1):
        raise ValueError(f"{name}: int32 with {dims} dimensions and contiguous rows on the GPU is wanted")


def block_norm(x, y=None, *, w_pre=None, w_post=None, b_pre=None, b_post=None, post_norm=None,
               gate=None, gate_sigmoid=False, res_scale=1.0, branch_scale=1.0, eps=1e-5,
               kind="rms", w_offset=0.0, r=None, h=None, need_r=True, need_h=True, h_dtype=None,
               stream=None):
    """r = res_scale * x + branch_scale * gate * N(y; w_post), h = N(r; w_pre)
    (moe_block_norm).

    x [T, H] is the residual stream, y [T, H] the block's output (None: no
    block has run yet).  The output of the block is normalised when w_post or
    b_post is given or ``post_norm`` is set.  gate: [H], [T, 1] or [T, H].
    Weights are fp32 or of y's type, all alike.  r and h are written in place
    when given (r may be x, h may be y); need_r / need_h False leaves one out.
    Returns (r, h), None for the one left out."""
    T, H = x.shape
    ldx = _rows(x, T, H, "x")
    stream_type, branch = x.dtype, h_dtype
    ldy = ldr = ldh = py = pr = ph = 0
    if y is not None:
        ldy, py, branch = _rows(y, T, H, "y"), y.data_ptr(), y.dtype
    if h is not None:
        if y is not None and h.dtype is not branch:
            raise ValueError("h: y's type is wanted")
        branch = h.dtype
    elif branch is None:
        branch = stream_type
    if r is not None:
        if r.dtype is not stream_type:
            raise ValueError("r: x's type is wanted")
        ldr, pr = _rows(r, T, H, "r"), r.data_ptr()
    elif need_r:
        r = _empty((T, H), stream_type, x.device, stream)
        ldr, pr = H, r.data_ptr()
    if h is not None:
        ldh, ph = _rows(h, T, H, "h"), h.data_ptr()
    elif need_h:
        h = _empty((T, H), branch, x.device, stream)
        ldh, ph = H, h.data_ptr()
    weight, post, post_b, pre, pre_b = None, 0, 0, 0, 0
    if w_pre is not None:
        weight = w_pre.dtype
        pre = _vector(w_pre, H, weight, "w_pre")
    if w_post is not None:
        weight = weight or w_post.dtype
        post = _vector(w_post, H, weight, "w_post")
    if b_pre is not None:
        weight = weight or b_pre.dtype
        pre_b = _vector(b_pre, H, weight, "b_pre")
    if b_post is not None:
        weight = weight or b_post.dtype
        post_b = _vector(b_post, H, weight, "b_post")
    if post_norm is None:
        post_norm = post or post_b
    row = col = pg = 0
    if gate is not None:
        shape = gate.shape
        if gate.dtype is not branch or not gate.is_cuda or shape not in ((H,), (T, 1), (T, H)):
            raise ValueError(f"gate: [{H}], [{T}, 1] or [{T}, {H}] of {branch} on the GPU is wanted")
        pg = gate.data_ptr()
        if len(shape) == 2:
            row = gate.stride(0)
        if shape[-1] == H:
            col = 1
            if H > 1 and gate.stride(-1) != 1:
                raise ValueError("gate: contiguous rows are wanted")
    if kind not in _KINDS:
        raise ValueError(f"kind: one of {sorted(_KINDS)} is wanted")
    a = moe.moe_block_norm_args(
        T, H, _KINDS[kind], _DT.get(stream_type, -1), _DT.get(branch, -1),
        moe.MOE_DT_F32 if weight is None else _DT.get(weight, -1), x.data_ptr(), ldx, py, ldy, pg, row, col,
        1 if gate_sigmoid else 0, 1 if post_norm else 0, post, post_b, pre, pre_b,
        res_scale, branch_scale, eps, w_offset, pr, ldr, ph, ldh)
    moe.moe_block_norm(a, _handle(stream))
    return r, h


class PagedKVCache:
    """Keys and values of many sequences in two pools of pages, each
    [n_pages, Hkv, page_size, D] (any strides with contiguous D values): the
    16-bit type of the queries, or torch.float8_e4m3fn with k_scale / v_scale
    [Hkv] fp32.  Holds the pools, the attention's workspace and a sticky status
    word; calls on one handle must not overlap on the GPU."""

    def __init__(self, k_pages, v_pages, k_scale=None, v_scale=None):
        if not (k_pages.dim() == 4 and k_pages.shape == v_pages.shape and k_pages.is_cuda and
                v_pages.is_cuda and k_pages.dtype == v_pages.dtype and k_pages.dtype in _DT and
                k_pages.stride() == v_pages.stride() and k_pages.stride(3) == 1):
            raise ValueError("pools: two alike [n_pages, Hkv, page_size, D] on the GPU are wanted")
        self.k_pages, self.v_pages, self.k_scale, self.v_scale = k_pages, v_pages, k_scale, v_scale
        n_pages, self.Hkv, self.page_size, self.D = k_pages.shape
        e4m3 = k_pages.dtype == torch.float8_e4m3fn
        if not e4m3 and (k_scale is not None or v_scale is not None):
            raise ValueError("scales: only for 8-bit pools")
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is not None:
                _vector(t, self.Hkv, torch.float32, name)
        self.view = moe.kvcache_view(
            k_pages.data_ptr(), v_pages.data_ptr(), k_pages.stride(0), k_pages.stride(1),
            k_pages.stride(2), n_pages, self.page_size, self.Hkv, self.D, _DT[k_pages.dtype],
            _ptr(k_scale), _ptr(v_scale))
        # enough for any number of query heads; its first 4096 bytes start at zero
        self._bytes = moe.kvcache_attend_workspace_bytes(16 * self.Hkv, self.Hkv, self.D)
        self._ws = torch.empty(max(self._bytes, 4096), dtype=torch.uint8, device=k_pages.device)
        self._ws[:4096].zero_()
        self._status = torch.zeros(1, dtype=torch.int32, device=k_pages.device)
        torch.cuda.current_stream().synchronize()
        self._append = moe.kvcache_append_args(c=self.view)
        self._append.status = self._status.data_ptr()
        self._attend = moe.kvcache_attend_args(c=self.view)
        self._attend.workspace, self._attend.workspace_bytes = self._ws.data_ptr(), self._bytes
        self._attend.status = self._status.data_ptr()

    @classmethod
    def create(cls, n_pages: int, page_size: int, Hkv: int, D: int, dtype=torch.bfloat16,
               k_scale=None, v_scale=None, device="cuda") -> "PagedKVCache":
        """New pools (zeros)."""
        k, v = (torch.zeros((n_pages, Hkv, page_size, D), dtype=dtype, device=device)
                for _ in range(2))
        return cls(k, v, k_scale, v_scale)

    def _heads(self, t, N, name):
        """Row and head strides of t, [N, heads, D]."""
        shape, st = t.shape, t.stride()
        if len(shape) != 3 or shape[0] != N or shape[2] != self.D or st[2] != 1 or not t.is_cuda:
            raise ValueError(f"{name}: [{N}, heads, {self.D}] on the GPU is wanted")
        return st[0], st[1]

    def append(self, k, v, page_table, pos, seq=None, q=None, cos=None, sin=None,
               interleaved=False, q_out=None, stream=None):
        """Stores k, v [N, Hkv, D] of N new tokens at positions pos [N] of
        sequences seq [N] (None: token n of sequence n), rotating k and q
        [N, Hq, D] by cos / sin [max_pos, rot / 2] when given
        (kvcache_append).  Returns the rotated q (None without q)."""
        _ints(pos, 1, "pos")
        _ints(page_table, 2, "page_table")
        N, a = pos.shape[0], self._append
        dtype = k.dtype
        if k.shape[1] != self.Hkv or v.shape[1] != self.Hkv or v.dtype is not dtype:
            raise ValueError(f"k, v: {self.Hkv} heads of one type are wanted")
        a.k_row, a.k_head = self._heads(k, N, "k")
        a.v_row, a.v_head = self._heads(v, N, "v")
        a.N, a.dtype, a.k, a.v = N, _DT.get(dtype, -1), k.data_ptr(), v.data_ptr()
        if q is not None:
            a.q_row, a.q_head = self._heads(q, N, "q")
            if q.dtype is not dtype:
                raise ValueError("q: the type of k is wanted")
            if q_out is None:
                q_out = _empty(q.shape, dtype, q.device, stream)
            elif q_out.shape != q.shape or q_out.dtype is not dtype:
                raise ValueError("q_out: q's shape and type are wanted")
            a.q_out_row, a.q_out_head = self._heads(q_out, N, "q_out")
            a.Hq, a.q, a.q_out = q.shape[1], q.data_ptr(), q_out.data_ptr()
        else:
            if q_out is not None:
                raise ValueError("q_out without q")
            a.Hq, a.q, a.q_out = 0, None, None
        if seq is not None:
            _ints(seq, 1, "seq")
            if seq.shape[0] != N:
                raise ValueError(f"seq: [{N}] is wanted")
            a.seq = seq.data_ptr()
        else:
            a.seq = None
        a.pos, a.page_table, a.table_ld = pos.data_ptr(), page_table.data_ptr(), page_table.stride(0)
        a.n_seqs, a.max_pages = page_table.shape
        if cos is None and sin is None:
            a.cos, a.sin, a.rot, a.max_pos = None, None, 0, 0
        else:
            if cos is None or sin is None or cos.dim() != 2 or cos.shape != sin.shape or not (
                    cos.dtype is sin.dtype is torch.float32 and cos.is_cuda and sin.is_cuda and
                    cos.is_contiguous() and sin.is_contiguous()):
                raise ValueError("cos, sin: both contiguous fp32 [max_pos, rot / 2] on the GPU are wanted")
            a.cos, a.sin = cos.data_ptr(), sin.data_ptr()
            a.max_pos, half = cos.shape
            a.rot = 2 * half
        a.interleaved = 1 if interleaved else 0
        moe.kvcache_append(a, _handle(stream))
        return q_out

    def attend(self, q, page_table, seq_lens, scale=None, window=0, softcap=0.0, out=None,
               lse=None, return_lse=False, stream=None):
        """Attention of one new token per sequence: q [B, Hq, D] over the first
        seq_lens [B] cached tokens (kvcache_attend).  scale defaults to
        D ** -0.5; window > 0 reads the last `window` positions only.  Returns
        out, or (out, lse [B, Hq] fp32) with return_lse or lse given."""
        shape, dtype, a = q.shape, q.dtype, self._attend
        B = shape[0]
        a.q_row, a.q_head = self._heads(q, B, "q")
        _ints(page_table, 2, "page_table")
        _ints(seq_lens, 1, "seq_lens")
        rows, a.max_pages = page_table.shape
        if rows != B or seq_lens.shape[0] != B:
            raise ValueError(f"page_table, seq_lens: {B} rows are wanted")
        if out is None:
            out = _empty(shape, dtype, q.device, stream)
        elif out.shape != shape or out.dtype is not dtype:
            raise ValueError("out: q's shape and type are wanted")
        a.out_row, a.out_head = self._heads(out, B, "out")
        if lse is not None:
            if lse.dtype is not torch.float32 or lse.shape != shape[:2] or not (
                    lse.is_cuda and lse.is_contiguous()):
                raise ValueError("lse: contiguous fp32 [B, Hq] on the GPU is wanted")
        elif return_lse:
            lse = _empty(shape[:2], torch.float32, q.device, stream)
        a.lse = None if lse is None else lse.data_ptr()
        a.B, a.Hq, a.dtype, a.q, a.out = B, shape[1], _DT.get(dtype, -1), q.data_ptr(), out.data_ptr()
        a.page_table, a.table_ld, a.seq_lens = (page_table.data_ptr(), page_table.stride(0),
                                                seq_lens.data_ptr())
        a.scale = self.D ** -0.5 if scale is None else scale
        a.softcap, a.window = softcap, window
        moe.kvcache_attend(a, _handle(stream))
        return out if lse is None else (out, lse)

    def read_status(self, stream=None) -> int:
        """Synchronises, returns the sticky device status and clears it."""
        s = torch.cuda.current_stream() if stream is None else stream
        if isinstance(s, int):
            s = torch.cuda.ExternalStream(s)
        with torch.cuda.stream(s):
            value = int(self._status.item())
            if value:
                self._status.zero_()
                s.synchronize()
        return value


class W4Linear:
    """y = x W^T + bias with 4-bit weights (moe_w4_linear): codes [N, K / 2]
    uint8 (value 2j in the low nibble), scales [N, K / group] of x's type;
    fmt "u4" (minus zeros, [N, ceil(K / group / 2)] uint8 nibbles, or 8) or
    "e2m1".  Holds its tensors; no workspace."""

    def __init__(self, codes, scales, group: int, zeros=None, bias=None, fmt="u4"):
        if fmt not in _FORMATS:
            raise ValueError(f"fmt: one of {sorted(_FORMATS)} is wanted")
        if codes.dtype is not torch.uint8 or codes.dim() != 2 or not (
                codes.is_cuda and codes.is_contiguous()):
            raise ValueError("codes: contiguous uint8 [N, K / 2] on the GPU are wanted")
        self.N, self.K = codes.shape[0], 2 * codes.shape[1]
        if group <= 0 or self.K % group:
            raise ValueError(f"group: a divisor of {self.K} is wanted")
        G = self.K // group
        if scales.shape != (self.N, G) or not (scales.is_cuda and scales.is_contiguous()):
            raise ValueError(f"scales: contiguous [{self.N}, {G}] on the GPU are wanted")
        if zeros is not None and (zeros.dtype is not torch.uint8 or zeros.shape != (self.N, (G + 1) // 2)
                                  or not (zeros.is_cuda and zeros.is_contiguous())):
            raise ValueError(f"zeros: contiguous uint8 [{self.N}, {(G + 1) // 2}] on the GPU are wanted")
        if bias is not None:
            _vector(bias, self.N, scales.dtype, "bias")
        self.codes, self.scales, self.zeros, self.bias = codes, scales, zeros, bias
        self.dtype = scales.dtype
        self._args = moe.moe_w4_linear_args(
            0, self.N, self.K, group, _DT.get(scales.dtype, -1), _FORMATS[fmt], None, 0,
            codes.data_ptr(), scales.data_ptr(), _ptr(zeros), _ptr(bias), None, 0)

    def forward(self, x, y=None, stream=None) -> torch.Tensor:
        """x [T, K] -> y [T, N]."""
        if x.dtype is not self.dtype or x.dim() != 2:
            raise ValueError(f"x: [T, {self.K}] of {self.dtype} is wanted")
        T, a = x.shape[0], self._args
        a.ldx = _rows(x, T, self.K, "x")
        if y is None:
            y = _empty((T, self.N), self.dtype, x.device, stream)
            a.ldy = self.N
        elif y.dtype is not self.dtype:
            raise ValueError("y: x's type is wanted")
        else:
            a.ldy = _rows(y, T, self.N, "y")
        a.T, a.x, a.y = T, x.data_ptr(), y.data_ptr()
        moe.moe_w4_linear(a, _handle(stream))
        return y


class DecodeBlock:
    """One pre-norm transformer block with a routed layer, for one new token of
    each sequence of a batch:

      h1 = N(x); q, k, v = Wqkv h1; rotate q, k and store k, v in the cache;
      r  = x + Wo attention(q);  h2 = N(r);  out = r + routed layer(h2)

    as the six launches norm, projection, append, attention, projection, norm,
    then the layer's own kernels and the residual addition (which takes the
    next block's norm with it when its weights are given)."""

    def __init__(self, layer: MoELayer, cache: PagedKVCache, qkv: W4Linear, out: W4Linear,
                 norm_in: torch.Tensor, norm_mid: torch.Tensor, cos=None, sin=None,
                 eps: float = 1e-5):
        self.layer, self.cache, self.qkv, self.out = layer, cache, qkv, out
        self.norm_in, self.norm_mid, self.cos, self.sin, self.eps = norm_in, norm_mid, cos, sin, eps
        self.Hq = qkv.N // cache.D - 2 * cache.Hkv
        if not (self.Hq > 0 and qkv.N == (self.Hq + 2 * cache.Hkv) * cache.D and
                out.K == self.Hq * cache.D and qkv.K == out.N == layer.H):
            raise ValueError("the projections, the cache and the layer do not fit each other")

    def forward(self, x, page_table, pos, seq_lens, h=None, norm_next=None, stream=None):
        """x [B, H] residual stream -> (r, h): the new stream and, with
        norm_next, the next block's input N(r; norm_next) (else None).  h: this
        block's input as the previous block returned it (None: N(x; norm_in)).
        pos [B]: the new tokens' positions; seq_lens [B] counts them too."""
        B, c = x.shape[0], self.cache
        if h is None:
            _, h = block_norm(x, w_pre=self.norm_in, need_r=False, eps=self.eps, stream=stream)
        p = self.qkv.forward(h, stream=stream).view(B, self.Hq + 2 * c.Hkv, c.D)
        q, k, v = p[:, :self.Hq], p[:, self.Hq:self.Hq + c.Hkv], p[:, self.Hq + c.Hkv:]
        q = c.append(k, v, page_table, pos, q=q, cos=self.cos, sin=self.sin, q_out=q, stream=stream)
        o = c.attend(q, page_table, seq_lens, stream=stream)
        a = self.out.forward(o.view(B, self.Hq * c.D), stream=stream)
        r, h = block_norm(x, a, w_pre=self.norm_mid, eps=self.eps, stream=stream)
        y = self.layer.forward(h, _empty(h.shape, h.dtype, h.device, stream), stream)
        return block_norm(r, y, w_pre=norm_next, need_h=norm_next is not None, r=r, eps=self.eps,
                          stream=stream)
