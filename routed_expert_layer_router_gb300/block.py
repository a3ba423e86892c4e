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


def _dt(t: torch.Tensor) -> int:
    code = _DT.get(t.dtype)
    if code is None:
        raise ValueError(f"no support for {t.dtype}")
    return code


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """An output that belongs to the stream that will write it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(s):
        return torch.empty(shape, dtype=dtype, device=device)


def _rows(t: torch.Tensor, T: int, H: int, name: str) -> None:
    _need(t.is_cuda and t.shape == (T, H) and (H == 1 or t.stride(1) == 1),
          f"{name}: [{T}, {H}] on the GPU with contiguous rows is wanted")


def _vector(t: torch.Tensor | None, n: int, dtypes, name: str) -> None:
    if t is not None:
        _need(t.is_cuda and t.shape == (n,) and t.is_contiguous() and t.dtype in dtypes,
              f"{name}: a contiguous [{n}] of {dtypes} on the GPU is wanted")


def _ints(t: torch.Tensor, dims: int, name: str) -> None:
    _need(t.is_cuda and t.dtype == torch.int32 and t.dim() == dims and
          (t.numel() == 0 or t.shape[-1] == 1 or t.stride(-1) == 1),
          f"{name}: int32 with {dims} dimensions on the GPU is wanted")


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
    _need(x.dim() == 2, "x: [T, H] is wanted")
    T, H = x.shape
    _rows(x, T, H, "x")
    if y is not None:
        _rows(y, T, H, "y")
    if r is not None:
        _rows(r, T, H, "r")
        _need(r.dtype == x.dtype, "r: x's type is wanted")
    elif need_r:
        r = _empty((T, H), x.dtype, x.device, stream)
    branch = y.dtype if y is not None else h.dtype if h is not None else h_dtype or x.dtype
    if h is not None:
        _rows(h, T, H, "h")
        _need(h.dtype == branch, "h: y's type is wanted")
    elif need_h:
        h = _empty((T, H), branch, x.device, stream)
    weight = next((w.dtype for w in (w_pre, w_post, b_pre, b_post) if w is not None), torch.float32)
    for w, name in ((w_pre, "w_pre"), (w_post, "w_post"), (b_pre, "b_pre"), (b_post, "b_post")):
        _vector(w, H, (weight,), name)
    if post_norm is None:
        post_norm = w_post is not None or b_post is not None
    row = col = 0
    if gate is not None:
        _need(gate.is_cuda and gate.dtype == branch and gate.shape in ((H,), (T, 1), (T, H)),
              f"gate: [{H}], [{T}, 1] or [{T}, {H}] of {branch} on the GPU is wanted")
        col = 1 if gate.shape[-1] == H and (H > 1 or gate.dim() == 1) else 0
        row = gate.stride(0) if gate.dim() == 2 else 0
        _need(not col or H == 1 or gate.stride(-1) == 1, "gate: contiguous rows are wanted")
    _need(kind in _KINDS, f"kind: one of {sorted(_KINDS)} is wanted")
    a = moe.moe_block_norm_args(
        T, H, _KINDS[kind], _dt(x), _DT.get(branch, -1), _DT.get(weight, -1),
        x.data_ptr(), x.stride(0), _ptr(y), y.stride(0) if y is not None else 0,
        _ptr(gate), row, col, moe.MOE_GATE_SIGMOID if gate_sigmoid else moe.MOE_GATE_NONE,
        1 if post_norm else 0, _ptr(w_post), _ptr(b_post), _ptr(w_pre), _ptr(b_pre),
        res_scale, branch_scale, eps, w_offset,
        _ptr(r), r.stride(0) if r is not None else 0, _ptr(h), h.stride(0) if h is not None else 0)
    moe.moe_block_norm(a, _stream(stream))
    return r, h


class PagedKVCache:
    """Keys and values of many sequences in two pools of pages, each
    [n_pages, Hkv, page_size, D] (any strides with contiguous D values): the
    16-bit type of the queries, or torch.float8_e4m3fn with k_scale / v_scale
    [Hkv] fp32.  Holds the pools, the attention's workspace and a sticky status
    word; calls on one handle must not overlap on the GPU."""

    def __init__(self, k_pages, v_pages, k_scale=None, v_scale=None):
        _need(k_pages.dim() == 4 and k_pages.shape == v_pages.shape and k_pages.is_cuda and
              v_pages.is_cuda and k_pages.dtype == v_pages.dtype and
              k_pages.stride() == v_pages.stride() and k_pages.stride(3) == 1,
              "pools: two alike [n_pages, Hkv, page_size, D] on the GPU are wanted")
        self.k_pages, self.v_pages, self.k_scale, self.v_scale = k_pages, v_pages, k_scale, v_scale
        n_pages, self.Hkv, self.page_size, self.D = k_pages.shape
        e4m3 = k_pages.dtype == torch.float8_e4m3fn
        _need(e4m3 or (k_scale is None and v_scale is None), "scales: only for 8-bit pools")
        _vector(k_scale, self.Hkv, (torch.float32,), "k_scale")
        _vector(v_scale, self.Hkv, (torch.float32,), "v_scale")
        self.view = moe.kvcache_view(
            k_pages.data_ptr(), v_pages.data_ptr(), k_pages.stride(0), k_pages.stride(1),
            k_pages.stride(2), n_pages, self.page_size, self.Hkv, self.D, _dt(k_pages),
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
        _need(t.is_cuda and t.dim() == 3 and t.shape[0] == N and t.shape[2] == self.D and
              t.stride(2) == 1, f"{name}: [{N}, heads, {self.D}] on the GPU is wanted")

    def append(self, k, v, page_table, pos, seq=None, q=None, cos=None, sin=None,
               interleaved=False, q_out=None, stream=None):
        """Stores k, v [N, Hkv, D] of N new tokens at positions pos [N] of
        sequences seq [N] (None: token n of sequence n), rotating k and q
        [N, Hq, D] by cos / sin [max_pos, rot / 2] when given
        (kvcache_append).  Returns the rotated q (None without q)."""
        N = pos.shape[0]
        self._heads(k, N, "k")
        self._heads(v, N, "v")
        _need(k.shape[1] == self.Hkv and v.shape[1] == self.Hkv and k.dtype == v.dtype,
              f"k, v: {self.Hkv} heads of one type are wanted")
        _ints(pos, 1, "pos")
        _ints(page_table, 2, "page_table")
        a = self._append
        a.N, a.dtype = N, _dt(k)
        a.k, a.k_row, a.k_head = k.data_ptr(), k.stride(0), k.stride(1)
        a.v, a.v_row, a.v_head = v.data_ptr(), v.stride(0), v.stride(1)
        if q is not None:
            self._heads(q, N, "q")
            _need(q.dtype == k.dtype, "q: the type of k is wanted")
            if q_out is None:
                q_out = _empty(q.shape, q.dtype, q.device, stream)
            else:
                self._heads(q_out, N, "q_out")
                _need(q_out.shape == q.shape and q_out.dtype == q.dtype, "q_out: q's shape and type")
            a.Hq, a.q, a.q_row, a.q_head = q.shape[1], q.data_ptr(), q.stride(0), q.stride(1)
            a.q_out, a.q_out_row, a.q_out_head = q_out.data_ptr(), q_out.stride(0), q_out.stride(1)
        else:
            _need(q_out is None, "q_out without q")
            a.Hq, a.q, a.q_out = 0, None, None
        if seq is not None:
            _ints(seq, 1, "seq")
            _need(seq.shape[0] == N, f"seq: [{N}] is wanted")
            a.seq = seq.data_ptr()
        else:
            a.seq = None
        a.pos = pos.data_ptr()
        a.page_table, a.table_ld = page_table.data_ptr(), page_table.stride(0)
        a.n_seqs, a.max_pages = page_table.shape
        _need((cos is None) == (sin is None), "cos and sin: both or none")
        if cos is not None:
            _need(cos.is_cuda and sin.is_cuda and cos.dim() == 2 and cos.shape == sin.shape and
                  cos.dtype == sin.dtype == torch.float32 and cos.is_contiguous() and
                  sin.is_contiguous(), "cos, sin: contiguous fp32 [max_pos, rot / 2] are wanted")
            a.cos, a.sin, a.rot, a.max_pos = (cos.data_ptr(), sin.data_ptr(), 2 * cos.shape[1],
                                              cos.shape[0])
        else:
            a.cos, a.sin, a.rot, a.max_pos = None, None, 0, 0
        a.interleaved = 1 if interleaved else 0
        moe.kvcache_append(a, _stream(stream))
        return q_out

    def attend(self, q, page_table, seq_lens, scale=None, window=0, softcap=0.0, out=None,
               lse=None, return_lse=False, stream=None):
        """Attention of one new token per sequence: q [B, Hq, D] over the first
        seq_lens [B] cached tokens (kvcache_attend).  scale defaults to
        D ** -0.5; window > 0 reads the last `window` positions only.  Returns
        out, or (out, lse [B, Hq] fp32) with return_lse or lse given."""
        B = q.shape[0]
        self._heads(q, B, "q")
        _ints(page_table, 2, "page_table")
        _ints(seq_lens, 1, "seq_lens")
        _need(page_table.shape[0] == B and seq_lens.shape[0] == B,
              f"page_table, seq_lens: {B} rows are wanted")
        if out is None:
            out = _empty(q.shape, q.dtype, q.device, stream)
        else:
            self._heads(out, B, "out")
            _need(out.shape == q.shape and out.dtype == q.dtype, "out: q's shape and type")
        if lse is not None:
            _need(lse.is_cuda and lse.dtype == torch.float32 and lse.shape == q.shape[:2] and
                  lse.is_contiguous(), "lse: contiguous fp32 [B, Hq] on the GPU is wanted")
        elif return_lse:
            lse = _empty(q.shape[:2], torch.float32, q.device, stream)
        a = self._attend
        a.B, a.Hq, a.dtype = B, q.shape[1], _dt(q)
        a.q, a.q_row, a.q_head = q.data_ptr(), q.stride(0), q.stride(1)
        a.out, a.out_row, a.out_head = out.data_ptr(), out.stride(0), out.stride(1)
        a.lse = _ptr(lse) or None
        a.page_table, a.table_ld = page_table.data_ptr(), page_table.stride(0)
        a.max_pages, a.seq_lens = page_table.shape[1], seq_lens.data_ptr()
        a.scale = self.D ** -0.5 if scale is None else scale
        a.softcap, a.window = softcap, window
        moe.kvcache_attend(a, _stream(stream))
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
        _need(fmt in _FORMATS, f"fmt: one of {sorted(_FORMATS)} is wanted")
        _need(codes.is_cuda and codes.dtype == torch.uint8 and codes.dim() == 2 and
              codes.is_contiguous(), "codes: contiguous uint8 [N, K / 2] on the GPU are wanted")
        self.N, self.K = codes.shape[0], 2 * codes.shape[1]
        _need(group > 0 and self.K % group == 0, f"group: a divisor of {self.K} is wanted")
        G = self.K // group
        _need(scales.is_cuda and scales.shape == (self.N, G) and scales.is_contiguous(),
              f"scales: contiguous [{self.N}, {G}] on the GPU are wanted")
        if zeros is not None:
            _need(zeros.is_cuda and zeros.dtype == torch.uint8 and
                  zeros.shape == (self.N, (G + 1) // 2) and zeros.is_contiguous(),
                  f"zeros: contiguous uint8 [{self.N}, {(G + 1) // 2}] on the GPU are wanted")
        _vector(bias, self.N, (scales.dtype,), "bias")
        self.codes, self.scales, self.zeros, self.bias = codes, scales, zeros, bias
        self.dtype = scales.dtype
        self._args = moe.moe_w4_linear_args(0, self.N, self.K, group, _dt(scales), _FORMATS[fmt],
                                            None, 0, codes.data_ptr(), scales.data_ptr(),
                                            _ptr(zeros), _ptr(bias), None, 0)

    def forward(self, x, y=None, stream=None) -> torch.Tensor:
        """x [T, K] -> y [T, N]."""
        _need(x.dim() == 2 and x.dtype == self.dtype, f"x: [T, {self.K}] of {self.dtype} is wanted")
        T = x.shape[0]
        _rows(x, T, self.K, "x")
        if y is None:
            y = _empty((T, self.N), x.dtype, x.device, stream)
        else:
            _rows(y, T, self.N, "y")
            _need(y.dtype == x.dtype, "y: x's type is wanted")
        a = self._args
        a.T, a.x, a.ldx, a.y, a.ldy = T, x.data_ptr(), x.stride(0), y.data_ptr(), y.stride(0)
        moe.moe_w4_linear(a, _stream(stream))
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
        _need(self.Hq > 0 and qkv.N == (self.Hq + 2 * cache.Hkv) * cache.D and
              out.K == self.Hq * cache.D and qkv.K == out.N == layer.H,
              "the projections, the cache and the layer do not fit each other")

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
