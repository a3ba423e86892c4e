"""The decode-block operators against plain fp64 torch: the block norm, the
paged cache's append and attention, the 4-bit linear product, and the block
that runs them with the routed layer.

Tolerances, per element, from the arithmetic: the output's rounding (half a
unit in the last place: U of its type, relative) plus the fp32 error of the
sums, a multiple of E = 2^-23 times the sum of the terms' magnitudes."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F16, F32, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
U = {BF: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}  # 8, 11, 24 significant bits
TINY = {BF: 2.0 ** -134, F16: 2.0 ** -25, F32: 2.0 ** -150}  # half the smallest subnormal
E = 2.0 ** -23
INF = math.inf


@pytest.fixture(scope="module")
def block():
    from routed_expert_layer_router_gb300 import block as b
    b.moe.lib()
    return b


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rn(g, *shape, dtype=F32, s=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * s).to(dtype)


def close(got, ref, slack, what=""):
    """|got - ref| <= U |ref| + slack, with the same infinities and NaNs."""
    got64 = got.double()
    assert torch.equal(torch.isnan(got64), torch.isnan(ref)), what
    inf = torch.isinf(ref)
    assert torch.equal(got64[inf], ref[inf]), what
    fine = torch.isfinite(ref)
    over = (got64 - ref).abs() - (U[got.dtype] * 1.001 * ref.abs() + TINY[got.dtype] + slack)
    worst = over[fine].max().item() if fine.any() else -1.0
    assert worst <= 0, f"{what}: {worst:.3e} over the bound"


# ----------------------------------------------------------------------- norm
def norm64(v, kind, w, b, eps, off):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    if w is not None:
        v = v * (w.double() + off)
    return v if b is None else v + b.double()


def norm_ref(x, y, kind, w_pre, w_post, b_pre, b_post, post, gate, sig, rs, bs, eps, off):
    r = x.double() * rs
    if y is not None:
        b = y.double()
        if post:
            b = norm64(b, kind, w_post, b_post, eps, off)
        if gate is not None:
            g = gate.double()
            b = b * (torch.sigmoid(g) if sig else g)
        r = r + bs * b
    return r, norm64(r, kind, w_pre, b_pre, eps, off)


def check_norm(block, x, y=None, kind="rms", w_pre=None, w_post=None, b_pre=None, b_post=None,
               post=None, gate=None, sig=False, rs=1.0, bs=1.0, eps=1e-5, off=0.0, **kw):
    post = (w_post is not None or b_post is not None) if post is None else post
    r0, h0 = norm_ref(x, y, kind, w_pre, w_post, b_pre, b_post, post, gate, sig, rs, bs, eps, off)
    r, h = block.block_norm(x, y, w_pre=w_pre, w_post=w_post, b_pre=b_pre, b_post=b_post,
                            post_norm=post, gate=gate, gate_sigmoid=sig, res_scale=rs,
                            branch_scale=bs, eps=eps, kind=kind, w_offset=off, **kw)
    # sums of H values: at most 32 in a row, then two trees of 5 levels; the
    # statistics enter twice: 64 units, at the size of the row's largest value
    bound = 64 * E
    rows = lambda t: t.abs().amax(-1, keepdim=True)  # noqa: E731
    if r is not None:
        close(r, r0, bound * rows(r0), "r")
    if h is not None:
        close(h, h0, bound * rows(h0), "h")
    return r, h


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("stream,branch", [(BF, BF), (F16, F16), (F32, F32), (F32, BF), (F32, F16)])
@pytest.mark.parametrize("T,H", [(1, 6144), (3, 2049), (5, 1), (2, 7), (7, 256), (4, 8192),
                                 (2, 16392), (1, 32768), (2, 5001), (700, 264)])
def test_norm_types_and_sizes(block, kind, stream, branch, T, H):
    g = gen(T * 7 + H)
    x, y = rn(g, T, H, dtype=stream, s=3.0), rn(g, T, H, dtype=branch)
    w = rn(g, H, s=0.2) + 1
    if H == 1 and kind == "layer":
        kw = {"eps": 1.0}  # a single value's deviation is 0
    else:
        kw = {}
    check_norm(block, x, y, kind, w_pre=w, rs=0.5, bs=-1.5, **kw)
    check_norm(block, x, y, kind, w_pre=w.to(branch), w_post=rn(g, H, dtype=branch),
               b_pre=rn(g, H, dtype=branch), b_post=rn(g, H, dtype=branch), off=1.0,
               gate=rn(g, H, dtype=branch), **kw)


@pytest.mark.parametrize("H", [512, 513])
@pytest.mark.parametrize("form", ["channel", "token", "full", "strided"])
@pytest.mark.parametrize("sig", [False, True])
def test_norm_gates(block, H, form, sig):
    g, T = gen(H), 9
    gate = {"channel": (H,), "token": (T, 1), "full": (T, H), "strided": (T, H + 24)}[form]
    gate = rn(g, *gate, dtype=BF, s=2.0)
    gate = gate[:, 8:8 + H] if form == "strided" else gate
    check_norm(block, rn(g, T, H), rn(g, T, H, dtype=BF), gate=gate, sig=sig, post=True)


def test_norm_without_a_branch_or_an_output(block):
    g = gen(1)
    x, y, w = rn(g, 4, 1024, dtype=BF), rn(g, 4, 1024, dtype=BF), rn(g, 1024)
    r, h = check_norm(block, x, w_pre=w, rs=2.0)
    r, h = check_norm(block, x, w_pre=w, need_r=False)
    assert r is None
    r, h = check_norm(block, x, y, need_h=False)
    assert h is None
    _, h = check_norm(block, rn(g, 4, 1024), w_pre=w, h_dtype=F16)
    assert h.dtype == F16
    r, h = block.block_norm(x[:0], y[:0], w_pre=w)
    assert r.shape == h.shape == (0, 1024)


def test_norm_strides_and_in_place(block):
    g = gen(2)
    for H, pad in ((640, 16), (640, 3), (77, 5)):  # aligned rows, odd strides, odd rows
        big = [rn(g, 6, H + pad, dtype=BF) for _ in range(4)]
        x, y, r, h = (t[:, :H] for t in big)
        edge = [t[:, H:].clone() for t in big]
        r0, h0 = check_norm(block, x, y, w_pre=None, post=True, r=r, h=h)
        assert r0.data_ptr() == r.data_ptr() and h0.data_ptr() == h.data_ptr()
        for t, e in zip(big, edge):
            assert torch.equal(t[:, H:], e)
        want = [r.clone(), h.clone()]
        block.block_norm(x, y, post_norm=True, r=x, h=y)
        assert torch.equal(x, want[0]) and torch.equal(y, want[1])
    t = rn(g, 3 * 641 + 1, dtype=BF)[1:].view(3, 641)[:, :640]  # base not 16-byte aligned
    check_norm(block, t, t, post=True)


@pytest.mark.parametrize("stream,branch", [(BF, BF), (F16, F16), (F32, F32), (F32, BF), (F32, F16)])
@pytest.mark.parametrize("T,H", [(320, 8192), (333, 5000), (401, 6001), (310, 8185), (305, 2049),
                                 (1000, 515), (306, 802), (500, 333)])
def test_norm_many_rows(block, stream, branch, T, H):
    """More rows than the GPU has CTAs for, aligned or beginning anywhere."""
    g = gen(T + H)
    x, y = rn(g, T, H, dtype=stream, s=3.0), rn(g, T, H, dtype=branch)
    w = rn(g, H, s=0.2) + 1
    check_norm(block, x, y, "rms", w_pre=w, w_post=w, gate=rn(g, T, H, dtype=branch), sig=True, rs=0.5)
    check_norm(block, x, y, "layer", w_pre=w.to(branch), b_pre=rn(g, H, dtype=branch),
               b_post=rn(g, H, dtype=branch), gate=rn(g, H, dtype=branch), bs=-1.5, off=1.0)
    check_norm(block, x, None, "layer", need_r=False, h_dtype=branch)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("stream,branch", [(BF, BF), (F32, F16), (F32, F32)])
def test_norm_many_odd_rows_stay_apart(block, kind, stream, branch):
    """Rows that share aligned accesses with their neighbours: what lies beside a row
    neither changes it nor is written, in place or not."""
    g, T, H = gen(11), 331, 1001
    big = [rn(g, T, H + 8, dtype=d) for d in (stream, branch, stream, branch)]
    x, y, r, h = (t[:, :H] for t in big)
    edge = [t[:, H:].clone() for t in big]
    gate = rn(g, T, 1, dtype=branch)
    kw = dict(kind=kind, post_norm=True, gate=gate, w_pre=rn(g, H))
    check_norm(block, x, y, kind, post=True, gate=gate, w_pre=kw["w_pre"], r=r, h=h)
    for t, e in zip(big, edge):
        assert torch.equal(t[:, H:], e)
    xd, yd = x.contiguous(), y.contiguous()
    want = [t.clone() for t in (r, h)]
    r1, h1 = block.block_norm(xd, yd, **kw)
    assert torch.equal(r1, want[0]) and torch.equal(h1, want[1])
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    for i, v in ((0, INF), (7, math.nan), (100, -INF), (330, math.nan)):
        (xd if i % 2 else yd)[i, (i * 37) % H] = v
        bad[i] = True
    gate[200] = INF
    bad[200] = True
    r2, h2 = block.block_norm(xd, yd, **kw)
    assert torch.equal(r2[~bad], want[0][~bad]) and torch.equal(h2[~bad], want[1][~bad])
    assert not r2[bad].isfinite().all(-1).any()
    gate[200] = 1.0
    block.block_norm(x, y, r=x, h=y, **kw)
    ok = torch.arange(T, device="cuda") != 200
    assert torch.equal(x[ok], want[0][ok]) and torch.equal(y[ok], want[1][ok])


def test_norm_extreme_rows(block):
    g, H = gen(3), 768
    x = rn(g, 6, H)
    x[0] = 0.0
    x[1] = 1e-20
    x[2] *= 1e15
    x[3, 5] = INF
    x[4, 7] = float("nan")
    x[5] = 4096.0 + x[5] * 1e-2  # a large mean: the variance is taken around it
    check_norm(block, x[:3], kind="rms")
    for kind in ("rms", "layer"):
        r, h = block.block_norm(x, kind=kind)
        assert torch.equal(r.isnan(), x.isnan()) and torch.equal(r.isinf(), x.isinf())
        assert h[4].isnan().all() and not h[[0, 1, 2, 5]].isnan().any()
        assert h[3].isnan()[5] and (kind == "layer" or (h[3, :5] == 0).all())
    _, h = block.block_norm(x[5:], kind="layer", eps=0.0)
    ref = norm64(x[5:].double(), "layer", None, None, 0.0, 0.0)
    # the mean's fp32 rounding, 2^-24 of 4096 and 45 additions, against a deviation of 1e-2
    assert (h.double() - ref).abs().max() <= 64 * E * 4096 / 1e-2


# ---------------------------------------------------------------------- cache
def pools(g, n_pages, Hkv, page, D, dtype, order="hnd"):
    shape = (n_pages, Hkv, page, D) if order == "hnd" else (n_pages, page, Hkv, D)
    out = []
    for _ in range(2):
        t = torch.randn(shape, generator=g, device="cuda")
        t = (t * 40).to(F8) if dtype == F8 else t.to(dtype)
        out.append(t if order == "hnd" else t.transpose(1, 2))
    return out


def table_for(g, lens, page, n_pages):
    cols = max(1, max(-(-max(n, 0) // page) for n in lens))
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    t = torch.full((len(lens), cols), -7, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        p = -(-max(n, 0) // page)
        t[b, :p] = perm[at:at + p]
        at += p
    assert at <= n_pages
    return t


def attend_ref(q, k_pages, v_pages, table, lens, ks, vs, scale, window, softcap, n_pages=None):
    """fp64 result, lse, and a bound of the error of each output value."""
    B, Hq, D = q.shape
    Hkv, page = k_pages.shape[1], k_pages.shape[2]
    n_pages = k_pages.shape[0] if n_pages is None else n_pages
    G = Hq // Hkv
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -INF, dtype=torch.float64, device="cuda")
    slack, lslack = torch.zeros_like(out), torch.zeros_like(lse)
    for b, n in enumerate(lens):
        n = max(0, min(n, table.shape[1] * page))
        at = torch.arange(max(0, n - window) if window else 0, n, device="cuda")
        ids = table[b].long()[at // page]
        ok = (ids >= 0) & (ids < n_pages)
        at, ids = at[ok], ids[ok]
        if not len(at):
            continue
        for h in range(Hkv):
            k, v = k_pages[ids, h, at % page].double(), v_pages[ids, h, at % page].double()
            if ks is not None:
                k, v = k * ks[h].double(), v * vs[h].double()
            qq = q[b, h * G:(h + 1) * G].double()
            s = qq @ k.T * scale
            size = (qq.abs() @ k.abs().T * abs(scale)).amax(-1)
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            p = torch.softmax(s, -1)
            sl = slice(h * G, (h + 1) * G)
            out[b, sl], lse[b, sl] = p @ v, torch.logsumexp(s, -1)
            # a score's error: D fp32 additions, the scale and the softmax's own
            # subtraction at its size; a weight: that, exp2's 2^-22 and the
            # 2^-16 of its two 16-bit parts; numerator and sum: len/16 + 64 additions
            es = (D + 8) * E * (size + 1)
            ep = 2 * es + 2.0 ** -16 + (len(at) / 16 + 64) * E
            slack[b, sl] = ep[:, None] * (p @ v.abs())
            lslack[b, sl] = es + (len(at) / 16 + 64) * E + 4 * E * lse[b, sl].abs()
    return out, lse, slack, lslack


def check_attend(block, q, k, v, table, lens, ks=None, vs=None, scale=None, window=0, softcap=0.0):
    cache = block.PagedKVCache(k, v, ks, vs)
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = cache.attend(q, table, seq, scale=scale, window=window, softcap=softcap,
                            return_lse=True)
    ro, rl, so, sl = attend_ref(q, k, v, table, lens, ks, vs,
                                q.shape[2] ** -0.5 if scale is None else scale, window, softcap)
    close(out, ro, so, "out")
    close(lse, rl, sl, "lse")
    again, lse2 = cache.attend(q, table, seq, scale=scale, window=window, softcap=softcap,
                               return_lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert not cache._ws[:4096].any()  # every call leaves the counters at zero
    return cache, out, lse


def scales_for(g, dtype, Hkv):
    if dtype != F8:
        return None, None
    return tuple(torch.rand(Hkv, generator=g, device="cuda") * 0.01 + 0.02 for _ in range(2))


@pytest.mark.parametrize("dtype,kv", [(BF, BF), (F16, F16), (BF, F8), (F16, F8)])
@pytest.mark.parametrize("G", [1, 3, 8, 9, 16, 20])
@pytest.mark.parametrize("D", [16, 64, 80, 128, 192, 256])
def test_attend_heads_and_types(block, dtype, kv, G, D):
    g, Hkv, page = gen(G * 1000 + D), 2, 16
    lens = [1, 77, 300, 0, 16]
    k, v = pools(g, 40, Hkv, page, D, kv)
    table = table_for(g, lens, page, 40)
    q = rn(g, len(lens), Hkv * G, D, dtype=dtype, s=2.0)
    check_attend(block, q, k, v, table, lens, *scales_for(g, kv, Hkv))


@pytest.mark.parametrize("page", [1, 5, 16, 24, 64, 100, 256])
@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("order", ["hnd", "nhd"])
def test_attend_pages_and_layouts(block, page, kv, order):
    g, Hkv, D, G = gen(page), 3, 64, 4
    lens = [0, 63, 64, 65, 1, 999, 2, 512, 128, 0, 31]
    n = sum(-(-x // page) for x in lens) + 2
    k, v = pools(g, n, Hkv, page, D, kv, order)
    check_attend(block, rn(g, len(lens), Hkv * G, D, dtype=BF), k, v,
                 table_for(g, lens, page, n), lens, *scales_for(g, kv, Hkv))


@pytest.mark.parametrize("window,softcap,scale", [(1, 0.0, None), (64, 0.0, None), (100, 30.0, None),
                                                  (4096, 2.0, 0.5), (0, 50.0, 1.0), (0, 0.0, 0.0),
                                                  (7, 0.0, -0.3)])
def test_attend_windows_caps_and_scales(block, window, softcap, scale):
    g, Hkv, D, page = gen(window), 2, 128, 16
    lens = [1, 100, 65, 700, 0, 4100]
    n = sum(-(-x // page) for x in lens)
    k, v = pools(g, n, Hkv, page, D, F16)
    check_attend(block, rn(g, len(lens), 12, D, dtype=F16, s=2.0), k, v,
                 table_for(g, lens, page, n), lens, scale=scale, window=window, softcap=softcap)


@pytest.mark.parametrize("B,Hkv,length", [(1, 1, 40000), (1, 8, 20011), (200, 2, 130), (65, 1, 1),
                                          (3, 4, 9000)])
def test_attend_split_and_joined(block, B, Hkv, length):
    """One long sequence cut over all CTAs, many short ones, and between."""
    g, D, page = gen(B), 128, 32
    lens = [max(0, length - 17 * b) if b % 7 else length for b in range(B)]
    n = sum(-(-x // page) for x in lens)
    k, v = pools(g, n, Hkv, page, D, BF)
    check_attend(block, rn(g, B, Hkv * 4, D, dtype=BF), k, v, table_for(g, lens, page, n), lens)


@pytest.mark.parametrize("dtype,kv", [(F16, F16), (BF, F8)])
@pytest.mark.parametrize("G,D", [(16, 224), (4, 128), (16, 128), (12, 64), (1, 64)])
def test_attend_same_bits_every_time(block, dtype, kv, G, D):
    """Rows cut between CTAs, whichever of them finishes last."""
    g, Hkv, page = gen(G + D), 2, 64
    lens = [926, 1, 0, 500, 926, 70, 301, 926, 640, 2, 926, 33, 800, 129]
    n = sum(-(-x // page) for x in lens)
    k, v = pools(g, n, Hkv, page, D, kv)
    cache = block.PagedKVCache(k, v, *scales_for(g, kv, Hkv))
    table, seq = table_for(g, lens, page, n), torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = rn(g, len(lens), Hkv * G, D, dtype=dtype)
    first = cache.attend(q, table, seq, return_lse=True)
    for _ in range(60):
        again = cache.attend(q, table, seq, return_lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_attend_empty_batches(block):
    g = gen(5)
    k, v = pools(g, 4, 2, 16, 64, BF)
    table = torch.zeros((3, 4), dtype=torch.int32, device="cuda")
    q = rn(g, 3, 4, 64, dtype=BF)
    cache, out, lse = check_attend(block, q, k, v, table, [0, 0, 0])
    assert not out.any() and (lse == -INF).all() and cache.read_status() == 0
    assert cache.attend(q[:0], table[:0], table[:0, 0].contiguous()).shape == (0, 4, 64)


@pytest.mark.parametrize("kv", [BF, F8])
def test_attend_ignores_what_lies_outside(block, kv):
    """NaN and infinities behind a sequence's end, before its window, in other
    sequences' pages and behind D never touch a row."""
    g, Hkv, D, page = gen(6), 2, 80, 24
    lens = [30, 100, 1, 0]
    n = 10
    clean = pools(g, n, Hkv, page, D + 16, kv)
    table = table_for(g, lens, page, n)
    ks, vs = scales_for(g, kv, Hkv)
    window = 40
    used = torch.zeros((n, page), dtype=torch.bool, device="cuda")
    for b, x in enumerate(lens):
        for p in range(max(0, x - window), x):
            used[table[b, p // page].item(), p % page] = True
    k, v = (t.float() for t in clean)
    for t in (k, v):
        t[..., D:] = float("nan")
        t.transpose(1, 2)[~used] = float("nan")
    if kv == BF:
        v.transpose(1, 2)[~used] = INF
    k, v = (t.to(kv)[..., :D] for t in (k, v))
    q = rn(g, 4, 6, D, dtype=BF)
    cache, out, lse = check_attend(block, q, k, v, table, lens, ks, vs, window=window)
    assert not out.isnan().any() and cache.read_status() == 0


def test_attend_values_that_are_read_do_show(block):
    g = gen(7)
    k, v = pools(g, 8, 1, 16, 64, BF)
    table = table_for(g, [100, 100], 16, 14) % 7
    k[table[0, 2].long(), 0, 3, 5] = float("nan")
    table[1] = 7
    q = rn(g, 2, 2, 64, dtype=BF)
    cache = block.PagedKVCache(k, v)
    out, lse = cache.attend(q, table, torch.tensor([100, 100], dtype=torch.int32, device="cuda"),
                            return_lse=True)
    assert out[0].isnan().all() and lse[0].isnan().all() and not out[1].isnan().any()


def test_attend_large_scores(block):
    """Scores of thousands, all equal or far apart; queries at the ends of bf16's range."""
    g, D = gen(8), 128
    for kv in (BF, F8):
        k, v = pools(g, 20, 1, 16, D, kv)
        table = table_for(g, [300], 16, 20)
        for s in (1e4, 1e-30, 0.0):
            q = rn(g, 1, 8, D, dtype=BF, s=s)
            check_attend(block, q, k, v, table, [300])
        q = rn(g, 1, 8, D, dtype=BF)
        q[0, :, 0] = 1e30  # one huge value: the other digits are below its reach
        out = block.PagedKVCache(k, v).attend(q, table, table.new_tensor([300]), scale=1e-30)
        assert torch.isfinite(out).all()


@pytest.mark.parametrize("dtype,kv", [(F16, F16), (BF, F8), (BF, BF)])
def test_attend_many_small_weights(block, dtype, kv):
    """A token whose weight is 2^26 times every other's: the others' values still
    count, for there are 100000 of them (each below f16's smallest number)."""
    n, page, D = 100000, 50, 16
    k = torch.zeros(n // page, 1, page, D, device="cuda")
    v = torch.ones_like(k)
    k[0, 0, 7, 0], v[0, 0, 7] = 1.0, 0.0
    q = torch.zeros(1, 2, D, device="cuda")
    q[..., 0] = 18.0
    table = torch.arange(n // page, dtype=torch.int32, device="cuda")[None]
    check_attend(block, q.to(dtype), k.to(kv), v.to(kv), table, [n],
                 *([torch.ones(1, device="cuda")] * 2 if kv == F8 else []), scale=1.0)


def test_attend_bad_pages_and_lengths(block):
    g, Hkv, D, page = gen(9), 2, 64, 16
    lens = [100, 50, 33]
    k, v = pools(g, 20, Hkv, page, D, BF)
    table = table_for(g, lens, page, 20)
    q = rn(g, 3, 4, D, dtype=BF)
    table[0, 2], table[1, :] = 20, -1
    cache, out, lse = check_attend(block, q, k, v, table, lens)
    assert cache.read_status() == 6 and cache.read_status() == 0  # MOE_ERR_DEVICE, then cleared
    assert not out[1].any() and (lse[1] == -INF).all()
    table = table_for(g, [112, 112, 112], page, 21)[:, :7] % 20
    cache, out, _ = check_attend(block, q, k, v, table, [5000, -3, 112])
    assert cache.read_status() == 6 and not out[1].any()


def test_attend_strided_rows_and_streams(block):
    g, Hkv, D = gen(10), 2, 64
    lens = [100, 50, 33]
    k, v = pools(g, 20, Hkv, 16, D, BF)
    table = torch.full((3, 19), -1, dtype=torch.int32, device="cuda")
    table[:, :7] = table_for(g, lens, 16, 20)
    qkv = rn(g, 3, 12, D, dtype=BF)
    q = qkv[:, 2:6]
    cache, out, lse = check_attend(block, q, k, v, table[:, :7], lens)
    wide = torch.zeros(3, 8, D, dtype=BF, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    got = cache.attend(q, table[:, :7], seq, out=wide[:, 1:5], stream=s)
    s.synchronize()
    assert torch.equal(got, out) and not wide[:, 0].any() and not wide[:, 5:].any()
    other = cache.attend(q, table[:, :7], seq, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(other, out)


def test_attend_in_a_graph(block):
    g = gen(11)
    lens = [5000, 50, 333]
    k, v = pools(g, 400, 2, 16, 128, BF)
    table = table_for(g, lens, 16, 400)
    q = rn(g, 3, 12, 128, dtype=BF)
    cache, out, _ = check_attend(block, q, k, v, table, lens)
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    buf = torch.zeros_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attend(q, table, seq, out=buf)
    for _ in range(3):
        buf.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf, out)
    seq.copy_(torch.tensor([77, 0, 1]))  # the lengths are read on the device
    graph.replay()
    assert torch.equal(buf, cache.attend(q, table, seq))


def test_attend_offsets_beyond_32_bits(block):
    """A pool of more than 2^32 bytes and 2^31 elements a tensor."""
    g, Hkv, page, D = gen(12), 2, 64, 128
    n = (1 << 31) // (Hkv * page * D) + 40
    k, v = (torch.zeros((n, Hkv, page, D), dtype=BF, device="cuda") for _ in range(2))
    for t in (k, v):
        t[-20:] = rn(g, 20, Hkv, page, D, dtype=BF)
        t[:20] = float("nan")
    table = (n - 1 - torch.randperm(20, device="cuda")).to(torch.int32).view(1, 20)
    q = rn(g, 1, 12, D, dtype=BF)
    check_attend(block, q, k, v, table, [1250])
    cache = block.PagedKVCache(k, v)
    new = rn(g, 3, Hkv, D, dtype=BF)
    pos = torch.tensor([0, 700, 1279], dtype=torch.int32, device="cuda")
    cache.append(new, new, table, pos, seq=torch.zeros_like(pos))
    for i, p in enumerate((0, 700, 1279)):
        assert torch.equal(k[table[0, p // page].long(), :, p % page], new[i])


# --------------------------------------------------------------------- append
def rotate64(t, cos, sin, interleaved):
    half = cos.shape[1]
    t, out = t.double(), t.double().clone()
    i = torch.arange(half, device="cuda")
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, s = cos.double()[:, None], sin.double()[:, None]
    out[..., a] = t[..., a] * c - t[..., b] * s
    out[..., b] = t[..., a] * s + t[..., b] * c
    return out


@pytest.mark.parametrize("dtype,kv", [(BF, BF), (F16, F16), (BF, F8), (F16, F8)])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (16, 16), (96, 96), (256, 32), (80, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(block, dtype, kv, D, rot, interleaved):
    g, Hq, Hkv, page, N = gen(D + rot), 6, 3, 5, 11
    lens = [7, 1, 20]
    table = table_for(g, lens, page, 12)
    k_pages, v_pages = pools(g, 12, Hkv, page, D, kv, "nhd")
    before = [t.clone() for t in (k_pages, v_pages)]
    places = [(0, 0), (2, 19), (1, 0), (2, 4), (2, 5), (0, 6), (2, 0), (0, 3), (2, 11), (2, -1), (2, 12)]
    seq = torch.tensor([s for s, _ in places], dtype=torch.int32, device="cuda")
    pos = torch.tensor([p for _, p in places], dtype=torch.int32, device="cuda")
    qkv = rn(g, N, Hq + 2 * Hkv, D, dtype=dtype, s=3.0)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    cos = sin = None
    if rot:
        angle = torch.rand(20, rot // 2, generator=g, device="cuda") * 6.3
        cos, sin = angle.cos(), angle.sin()
    ks, vs = scales_for(g, kv, Hkv)
    cache = block.PagedKVCache(k_pages, v_pages, ks, vs)
    qo = cache.append(k, v, table, pos, seq=seq, q=q, cos=cos, sin=sin, interleaved=interleaved)
    at = pos.clamp(min=0).long()
    rq, rk, rv = q.double(), k.double(), v.double()
    if rot:
        rq, rk = (rotate64(t, cos[at], sin[at], interleaved) for t in (q, k))
    rq[9] = 0  # position -1: skipped
    close(qo, rq, 4 * E * q.double().abs().amax(-1, keepdim=True), "q")
    written = torch.zeros(k_pages.shape, dtype=torch.bool, device="cuda")
    for n, (s, p) in enumerate(places):
        if p < 0:
            continue
        pg, slot = table[s, p // page].long(), p % page
        written[pg, :, slot] = True
        for pool, ref, src, sc in ((k_pages, rk, k, ks), (v_pages, rv, v, vs)):
            got = pool[pg, :, slot].double()
            if kv != F8:
                close(pool[pg, :, slot], ref[n], 4 * E * src[n].double().abs().amax(), "pool")
                continue
            want = (ref[n] / sc[:, None].double()).clamp(-448, 448)
            # half a step of 3 mantissa bits, or of the subnormals' 2^-9
            over = (got - want).abs() - (2.0 ** -4 * 1.001 * want.abs()).clamp(min=2.0 ** -10 * 1.001)
            assert over.max() <= 0
            if pool is v_pages or not rot:
                exact = (src[n].float() / sc[:, None]).clamp(-448, 448).to(F8)
                assert torch.equal(got, exact.double())
    for pool, old in zip((k_pages, v_pages), before):  # nothing else has changed
        assert torch.equal(pool.float()[~written], old.float()[~written])
    assert cache.read_status() == 0
    # queries in place, and none
    q2 = q.clone()
    assert cache.append(k, v, table, pos, seq=seq, q=q2, cos=cos, sin=sin, interleaved=interleaved,
                        q_out=q2) is q2
    assert torch.equal(q2, qo)
    assert cache.append(k, v, table, pos, seq=seq, cos=cos, sin=sin, interleaved=interleaved) is None


@pytest.mark.parametrize("N,Hq,Hkv,D", [(1, 48, 8, 128), (300, 2, 1, 64), (1, 200, 4, 256), (0, 4, 2, 64)])
def test_append_token_counts(block, N, Hq, Hkv, D):
    g, page = gen(N), 16
    n = -(-max(N, 1) // page)
    cache = block.PagedKVCache.create(n, page, Hkv, D)
    table = torch.arange(n, dtype=torch.int32, device="cuda").view(1, n)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    k, v, q = (rn(g, N, h, D, dtype=BF) for h in (Hkv, Hkv, Hq))
    out = cache.append(k, v, table, pos, seq=torch.zeros_like(pos), q=q)
    assert torch.equal(out, q)
    for pool, src in ((cache.k_pages, k), (cache.v_pages, v)):
        assert torch.equal(pool.transpose(1, 2).reshape(-1, Hkv, D)[:N], src)


def test_append_saturates_and_keeps_nan(block):
    cache = block.PagedKVCache.create(1, 16, 1, 16, dtype=F8)
    x = torch.zeros(1, 1, 16, dtype=BF, device="cuda")
    x[0, 0, :6] = torch.tensor([1e9, -1e9, INF, -INF, float("nan"), 0.1])
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache.append(x, x, zero.view(1, 1), zero)
    got = cache.k_pages[0, 0, 0].float()
    assert got[:4].tolist() == [448.0, -448.0, 448.0, -448.0] and got[4].isnan()


def test_append_out_of_range(block):
    g = gen(13)
    cache = block.PagedKVCache.create(4, 16, 1, 64)
    table = torch.tensor([[0, 1], [2, 9]], dtype=torch.int32, device="cuda")
    x = rn(g, 1, 1, 64, dtype=BF)
    angle = torch.zeros(20, 32, device="cuda")
    for s, p in ((0, 32), (2, 0), (-1, 0), (1, 16), (0, 20)):
        seq, pos = (torch.tensor([t], dtype=torch.int32, device="cuda") for t in (s, p))
        out = cache.append(x, x, table, pos, seq=seq, q=x, cos=angle, sin=angle)
        assert cache.read_status() == 6, (s, p)
        assert not out.any()
    assert not cache.k_pages.any() and not cache.v_pages.any()


# ------------------------------------------------------------------------- w4
def nibbles(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def dense64(codes, scales, zeros, group, fmt):
    c = nibbles(codes).long()
    N, K = c.shape
    if fmt == "e2m1":
        v = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6],
                         dtype=torch.float64, device="cuda")[c]
    else:
        z = 8 if zeros is None else nibbles(zeros)[:, :K // group].double().repeat_interleave(group, 1)
        v = c.double() - z
    return v * scales.double().repeat_interleave(group, 1)


def make_w4(g, N, K, group, dtype, fmt, zeros, bias):
    G = K // group
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.randn(N, G, generator=g, device="cuda") * 0.02).to(dtype)
    z = None
    if zeros:
        z = torch.randint(0, 256, (N, (G + 1) // 2), generator=g, device="cuda", dtype=torch.uint8)
    return codes, scales, z, rn(g, N, dtype=dtype) if bias else None


def check_w4(block, x, codes, scales, zeros, bias, group, fmt, **kw):
    w = dense64(codes, scales, zeros, group, fmt)
    ref = x.double() @ w.T
    K = x.shape[1]
    # fp32 sums: 16-deep products, the group's, the row's share of a warp and 8 warps
    slack = (K / 128 + 32) * E * (x.double().abs() @ w.abs().T)
    if bias is not None:
        ref = ref + bias.double()
        slack = slack + E * bias.double().abs()
    y = block.W4Linear(codes, scales, group, zeros=zeros, bias=bias, fmt=fmt).forward(x, **kw)
    close(y, ref, slack, "y")
    return y


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("fmt,zeros", [("u4", False), ("u4", True), ("e2m1", False)])
@pytest.mark.parametrize("K,group", [(32, 32), (256, 32), (480, 96), (1024, 64), (2176, 128),
                                     (1280, 640), (6144, 6144), (320, 160)])
@pytest.mark.parametrize("T,N", [(1, 64), (3, 17), (8, 1), (9, 33), (16, 100), (17, 40)])
def test_w4(block, dtype, fmt, zeros, K, group, T, N):
    g = gen(K + T)
    codes, scales, z, bias = make_w4(g, N, K, group, dtype, fmt, zeros, T % 2 == 1)
    check_w4(block, rn(g, T, K, dtype=dtype), codes, scales, z, bias, group, fmt)


@pytest.mark.parametrize("fmt,zeros", [("u4", True), ("e2m1", False)])
@pytest.mark.parametrize("T,N,K,group", [(1, 6144, 6144, 128), (13, 2000, 6144, 64),
                                         (40, 513, 2048, 32), (1, 31, 32768, 32)])
def test_w4_large(block, fmt, zeros, T, N, K, group):
    g = gen(N)
    codes, scales, z, bias = make_w4(g, N, K, group, BF, fmt, zeros, True)
    check_w4(block, rn(g, T, K, dtype=BF), codes, scales, z, bias, group, fmt)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("fmt,zeros", [("u4", True), ("e2m1", False)])
@pytest.mark.parametrize("T,N,K,group", [(40, 2000, 6144, 64), (17, 4000, 4096, 32), (33, 300, 8192, 128),
                                         (4, 512, 8192, 64), (2, 6144, 1024, 32), (13, 512, 8160, 96),
                                         (100, 4096, 2048, 128), (16, 8192, 4096, 256)])
def test_w4_splits(block, dtype, fmt, zeros, T, N, K, group):
    """Rows and K dealt to warps, CTAs and clusters in every way; x prepared before."""
    g = gen(T + N)
    codes, scales, z, bias = make_w4(g, N, K, group, dtype, fmt, zeros, True)
    x = rn(g, T, K, dtype=dtype)
    y = check_w4(block, x, codes, scales, z, bias, group, fmt)
    lin = block.W4Linear(codes, scales, group, zeros=z, bias=bias, fmt=fmt)
    assert torch.equal(y, lin.forward(x))


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("fmt", ["u4", "e2m1"])
def test_w4_each_code_at_each_place(block, dtype, fmt):
    """x a unit vector: y is one column of W, exactly (scale 1)."""
    g, N, K = gen(20), 48, 64
    codes, _, z, _ = make_w4(g, N, K, 32, dtype, fmt, fmt == "u4", False)
    scales = torch.ones(N, 2, dtype=dtype, device="cuda")
    w = dense64(codes, scales, z, 32, fmt)
    y = block.W4Linear(codes, scales, 32, zeros=z, fmt=fmt).forward(
        torch.eye(K, dtype=dtype, device="cuda"))
    assert torch.equal(y.double(), w.T)


def test_w4_infinities_stay_in_their_row(block):
    g, K = gen(21), 288
    codes, scales, z, _ = make_w4(g, 40, K, 32, BF, "u4", True, False)
    scales[3, 8], scales[20, 0] = INF, float("nan")
    x = rn(g, 2, K, dtype=BF)
    x[1, 5] = float("nan")
    y = block.W4Linear(codes, scales, 32, zeros=z).forward(x)
    assert y[1].isnan().all() and y[0, 20].isnan()
    rest = [i for i in range(40) if i not in (3, 20)]
    assert y[0, rest].isfinite().all() and y[0, 3].isinf()


def test_w4_strides_and_streams(block):
    g, N, K = gen(22), 100, 512
    codes, scales, z, b = make_w4(g, N, K, 128, F16, "u4", False, True)
    wide = rn(g, 5, K + 8, dtype=F16)
    y = check_w4(block, wide[:, 8:], codes, scales, z, b, 128, "u4")
    out = torch.zeros(5, N + 3, dtype=F16, device="cuda")
    lin = block.W4Linear(codes, scales, 128, bias=b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lin.forward(wide[:, 8:], y=out[:, 1:1 + N], stream=s)
    s.synchronize()
    assert torch.equal(out[:, 1:1 + N], y) and not out[:, 0].any() and not out[:, N + 1:].any()
    assert lin.forward(wide[:0, 8:]).shape == (0, N)


# ------------------------------------------------------------------- refusals
def test_wrong_arguments_are_refused(block):
    g = gen(30)
    x = rn(g, 2, 64, dtype=BF)
    for bad in (dict(y=x[:1]), dict(y=x.T), dict(w_pre=rn(g, 63)), dict(gate=x.float(), y=x),
                dict(kind="max"), dict(r=rn(g, 2, 64)), dict(w_pre=rn(g, 64), b_pre=rn(g, 64, dtype=BF))):
        with pytest.raises(ValueError):
            block.block_norm(x, **bad)
    with pytest.raises(block.moe.MoeError):  # f16 stream with a bf16 branch
        block.block_norm(x.half(), x)
    with pytest.raises(block.moe.MoeError):  # a gate without a branch
        block.block_norm(x, gate=x)
    k, v = pools(g, 4, 2, 16, 64, BF)
    cache = block.PagedKVCache(k, v)
    table = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    q = rn(g, 2, 4, 64, dtype=BF)
    for args in ((q[:, :, :32], table, lens), (q, table.long(), lens), (q, table, lens[:1]),
                 (q[0], table, lens)):
        with pytest.raises(ValueError):
            cache.attend(*args)
    for bad in (q.half(), q[:, :3]):  # another type than the pool's, heads that do not divide
        with pytest.raises(block.moe.MoeError):
            cache.attend(bad, table, lens)
    with pytest.raises(block.moe.MoeError):
        cache.attend(q, table, lens, window=-1)
    with pytest.raises(block.moe.MoeError):  # rows that are not 16-byte aligned
        cache.attend(rn(g, 2, 4, 65, dtype=BF)[:, :, 1:], table, lens)
    with pytest.raises(ValueError):
        block.PagedKVCache(k, v[:3])
    with pytest.raises(ValueError):
        block.PagedKVCache(k, v, k_scale=torch.ones(2, device="cuda"))
    kk = rn(g, 2, 2, 64, dtype=BF)
    with pytest.raises(ValueError):
        cache.append(kk, kk, table, lens, cos=torch.zeros(4, 32, device="cuda"))
    with pytest.raises(block.moe.MoeError):  # rotation of more values than a head has
        t = torch.zeros(4, 64, device="cuda")
        cache.append(kk, kk, table, lens, cos=t, sin=t)
    codes, scales, z, b = make_w4(g, 8, 64, 32, BF, "u4", True, True)
    for bad in (dict(group=48), dict(group=32, fmt="int4"), dict(group=32, zeros=z[:, :0])):
        with pytest.raises(ValueError):
            block.W4Linear(codes, scales, **bad)
    with pytest.raises(block.moe.MoeError):  # E2M1 has no zero points
        block.W4Linear(codes, scales, 32, zeros=z, fmt="e2m1").forward(x)
    with pytest.raises(ValueError):
        block.W4Linear(codes, scales, 32).forward(x.half())
    assert cache.read_status() == 0


# ------------------------------------------------------------------ the block
def test_decode_block_with_the_routed_layer(block):
    """Three steps of a two-sequence batch through norm, projections, cache,
    attention and the routed layer, against fp64 on the same intermediate
    values (each operator's own output feeds the next)."""
    import gen as inputs
    import gen.device as gd
    wl = inputs.WORKLOADS["tiny"]
    dw = gd.build(wl, T_max=wl.T)
    try:
        g, H, Hq, Hkv, D, group = gen(40), wl.H, 4, 2, 32, 64
        qkv = block.W4Linear(*make_w4(g, (Hq + 2 * Hkv) * D, H, group, BF, "u4", False, False)[:2], group)
        out = block.W4Linear(*make_w4(g, H, Hq * D, group, BF, "e2m1", False, False)[:2], group, fmt="e2m1")
        cache = block.PagedKVCache.create(6, 2, Hkv, D)
        angle = torch.rand(8, D // 2, generator=g, device="cuda") * 6
        n1, n2, n3 = (rn(g, H, s=0.1) + 1 for _ in range(3))
        blk = block.DecodeBlock(dw.moe_layers[0], cache, qkv, out, n1, n2, angle.cos(), angle.sin())
        table = torch.tensor([[4, 0, 2], [1, 5, 3]], dtype=torch.int32, device="cuda")
        keys = [[], []]
        for step in range(3):
            x = rn(g, 2, H, dtype=BF)
            pos = torch.tensor([step, step], dtype=torch.int32, device="cuda")
            r, h = blk.forward(x, table, pos, pos + 1, norm_next=n3)
            # the same, operator by operator, from the fp64 formulas
            _, h1 = block.block_norm(x, w_pre=n1, need_r=False)
            close(h1, norm64(x.double(), "rms", n1, None, 1e-5, 0), 64 * E * 4, "h1")
            p = qkv.forward(h1).view(2, Hq + 2 * Hkv, D)
            rot = [rotate64(t, angle.cos()[step:step + 1], angle.sin()[step:step + 1], False)
                   for t in (p[:, :Hq], p[:, Hq:Hq + Hkv])]
            for b in range(2):
                keys[b].append((rot[1][b].to(BF), p[b, Hq + Hkv:]))
            o = torch.empty(2, Hq, D, dtype=torch.float64, device="cuda")
            for b in range(2):
                k, v = (torch.stack([t[i] for t in keys[b]]).double() for i in range(2))
                for hd in range(Hq):
                    kv = hd // (Hq // Hkv)
                    w = torch.softmax(rot[0].to(BF)[b, hd].double() @ k[:, kv].T * D ** -0.5, -1)
                    o[b, hd] = w @ v[:, kv]
            a = o.view(2, Hq * D) @ dense64(out.codes, out.scales, None, group, "e2m1").T
            r1 = x.double() + a
            h2 = norm64(r1, "rms", n2, None, 1e-5, 0).to(BF)
            y = dw.moe_layers[0].forward(h2).double()
            ref = r1 + y
            # bf16 at the attention's and both projections' outputs, at h2 and y
            # (whose layer's own bound is 2e-2 of its size): within 4e-2 of the stream
            assert (r.double() - ref).abs().max() <= 4e-2 * ref.abs().max()
            close(h, norm64(r.double(), "rms", n3, None, 1e-5, 0), 2.0 ** -8 * 8, "h")
        assert cache.read_status() == 0 and dw.moe_layers[0].read_status() == 0
        same, none = blk.forward(x, table, pos, pos + 1, h=h1)
        assert none is None and torch.equal(same, r)
    finally:
        dw.close()
