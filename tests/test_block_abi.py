"""The decode-block calls of include/moe.h refuse what they do not take, on the
host, before anything is enqueued (no GPU needed), and the binding's structures
have the header's layout."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 4096  # stands for any aligned device address


@pytest.fixture(scope="module")
def moe():
    from routed_expert_layer_router_gb300 import build, moe as m
    if not os.path.exists(m.LIB_PATH):
        build()
    m.lib()
    return m


def test_structure_layouts(moe, tmp_path):
    names = ["moe_block_norm_args", "kvcache_view", "kvcache_append_args", "kvcache_attend_args",
             "moe_w4_linear_args"]
    lines = []
    for n in names:
        lines.append(f'printf("{n} %zu\\n", sizeof({n}));')
        for f, _ in getattr(moe, n)._fields_:
            lines.append(f'printf("{n}.{f} %zu\\n", offsetof({n}, {f}));')
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "moe.h"\nint main(void) {\n' + "\n".join(lines) +
                   "\nreturn 0;\n}\n")
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-I" + os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    for line in out.splitlines():
        name, value = line.split()
        cls, _, field = name.partition(".")
        st = getattr(moe, cls)
        assert int(value) == (getattr(st, field).offset if field else ctypes.sizeof(st)), name


def norm_args(moe, **kw):
    a = moe.moe_block_norm_args(2, 64, 0, 0, 0, 1)
    a.x, a.ldx, a.y, a.ldy, a.r, a.ldr, a.h, a.ldh = P, 64, P, 64, P, 64, P, 64
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,st", [
    (dict(H=0), 1), (dict(T=-1), 1), (dict(kind=2), 1), (dict(gate_act=2), 1), (dict(x=None), 1),
    (dict(r=None, h=None), 1), (dict(y=None, post_norm=1), 1), (dict(y=None, gate=P), 1),
    (dict(gate=P, gate_col=2), 1), (dict(gate=P, gate_row=-1), 1), (dict(ldx=63), 1),
    (dict(ldy=63), 1), (dict(ldr=63), 1), (dict(ldh=63), 1), (dict(stream_type=2), 2),
    (dict(branch_type=3), 2), (dict(weight_type=2), 2), (dict(H=32769, ldx=40000), 2),
    (dict(stream_type=0, branch_type=1), 2), (dict(T=0), 0), (dict(T=0, x=None), 0)])
def test_block_norm(moe, kw, st):
    assert moe.lib().moe_block_norm(ctypes.byref(norm_args(moe, **kw)), None) == st


def view(moe, **kw):
    c = moe.kvcache_view(P, P, 2 * 16 * 64, 16 * 64, 64, 4, 16, 2, 64, 0, None, None)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


VIEWS = [(dict(Hkv=0), 1), (dict(D=0), 1), (dict(page_size=0), 1), (dict(n_pages=-1), 1),
         (dict(k_pages=None), 1), (dict(page_stride=-8), 1), (dict(D=24), 2), (dict(D=272), 2),
         (dict(kv_type=2), 2), (dict(kv_type=1), 2), (dict(token_stride=68), 2),
         (dict(v_pages=P + 8), 2), (dict(kv_type=3, head_stride=24), 2)]


def append_args(moe, c=None, **kw):
    a = moe.kvcache_append_args(c=view(moe, **(c or {})))
    a.N, a.Hq, a.dtype, a.n_seqs, a.max_pages, a.table_ld = 3, 4, 0, 1, 2, 2
    a.k, a.v, a.q, a.q_out, a.pos, a.page_table, a.cos, a.sin = P, P, P, P, P, P, P, P
    a.rot, a.max_pos = 32, 10
    for n in ("k", "v", "q", "q_out"):
        setattr(a, n + "_row", 256)
        setattr(a, n + "_head", 64)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("c,kw,st", [(c, {}, st) for c, st in VIEWS] + [({}, kw, st) for kw, st in [
    (dict(N=-1), 1), (dict(Hq=-1), 1), (dict(Hq=0), 1), (dict(k=None), 1), (dict(pos=None), 1),
    (dict(page_table=None), 1), (dict(q_out=None), 1), (dict(cos=None), 1), (dict(rot=0), 1),
    (dict(rot=80), 1), (dict(max_pos=-1), 1), (dict(n_seqs=-1), 1), (dict(dtype=1), 2),
    (dict(rot=24), 2), (dict(k_row=100), 2), (dict(q_head=4), 2), (dict(v=P + 2), 2),
    (dict(cos=P + 4), 2), (dict(N=0), 0)]])
def test_append(moe, c, kw, st):
    assert moe.lib().kvcache_append(ctypes.byref(append_args(moe, c, **kw)), None) == st


def attend_args(moe, c=None, **kw):
    a = moe.kvcache_attend_args(c=view(moe, **(c or {})))
    a.B, a.Hq, a.dtype, a.max_pages, a.table_ld = 3, 4, 0, 2, 2
    a.q, a.out, a.page_table, a.seq_lens, a.workspace = P, P, P, P, P
    a.q_row, a.q_head, a.out_row, a.out_head = 256, 64, 256, 64
    a.scale, a.workspace_bytes = 1.0, 1 << 30
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("c,kw,st", [(c, {}, st) for c, st in VIEWS] + [({}, kw, st) for kw, st in [
    (dict(B=-1), 1), (dict(Hq=0), 1), (dict(q=None), 1), (dict(out=None), 1),
    (dict(seq_lens=None), 1), (dict(page_table=None), 1), (dict(workspace=None), 1),
    (dict(workspace_bytes=4096), 1), (dict(window=-1), 1), (dict(softcap=-1.0), 1),
    (dict(softcap=float("nan")), 1), (dict(max_pages=-1), 1), (dict(Hq=5), 2), (dict(dtype=3), 2),
    (dict(q_row=100), 2), (dict(out_head=4), 2), (dict(out=P + 2), 2), (dict(workspace=P + 8), 2),
    (dict(B=0), 0)]])
def test_attend(moe, c, kw, st):
    assert moe.lib().kvcache_attend(ctypes.byref(attend_args(moe, c, **kw)), None) == st


def w4_args(moe, **kw):
    a = moe.moe_w4_linear_args(3, 40, 256, 64, 0, 0, P, 256, P, P, None, None, P, 40)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,st", [
    (dict(T=-1), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(group=0), 1), (dict(format=2), 1),
    (dict(format=1, zeros=P), 1), (dict(x=None), 1), (dict(codes=None), 1), (dict(scales=None), 1),
    (dict(y=None), 1), (dict(ldx=255), 1), (dict(ldy=39), 1), (dict(dtype=1), 2),
    (dict(group=16), 2), (dict(group=96), 2), (dict(x=P + 2), 2), (dict(codes=P + 1), 2),
    (dict(ldx=260), 2), (dict(T=9), 1), (dict(T=9, workspace=P, workspace_bytes=9 * 576 - 1), 1),
    (dict(T=9, workspace=P + 8, workspace_bytes=9 * 576), 2), (dict(T=0), 0)])
def test_w4(moe, kw, st):
    assert moe.lib().moe_w4_linear(ctypes.byref(w4_args(moe, **kw)), None) == st


def test_null_arguments_and_sizes(moe):
    L = moe.lib()
    for f in (L.moe_block_norm, L.kvcache_append, L.kvcache_attend, L.moe_w4_linear):
        assert f(None, None) == 1
    assert L.kvcache_attend_workspace_bytes(4, 3, 64) == 0
    assert L.kvcache_attend_workspace_bytes(4, 0, 64) == 0
    assert L.kvcache_attend_workspace_bytes(4, 2, 257) == 0
    assert L.kvcache_attend_workspace_bytes(4, 2, 64) > 4096
    # 256 values of a token with their sums: 576 bytes; none up to 8 tokens, nor for
    # f16 with E2M1 codes
    assert L.moe_w4_linear_workspace_bytes(8, 6144, 0, 0) == 0
    assert L.moe_w4_linear_workspace_bytes(9, 6144, 0, 0) == 9 * 24 * 576
    assert L.moe_w4_linear_workspace_bytes(9, 6160, 0, 1) == 9 * 25 * 576
    assert L.moe_w4_linear_workspace_bytes(9, 6144, 2, 0) == 9 * 24 * 576
    assert L.moe_w4_linear_workspace_bytes(9, 6144, 2, 1) == 0
