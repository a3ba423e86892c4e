"""The decode-block operators as they are measured: the fused block norm, the
paged key-value cache's append and attention, and the 4-bit linear product.

Each case is one call of one operator.  ``run`` computes it in plain torch
(fp32 throughout, rounded once at the end) or, with ``own`` set, through the
library's public calls (routed_expert_layer_router_gb300.block).  ``exact``
computes the same outputs in fp64 from the definitions.
"""
from __future__ import annotations

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
      "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- the cases
def _norm(name, T, H, stream, branch, kind="rms", post=False, gate="none", res_scale=1.0):
    return {"name": name, "op": "norm", "T": T, "H": H, "stream": stream, "branch": branch,
            "kind": kind, "post": post, "gate": gate, "res_scale": res_scale}


def _append(name, N, Hq, Hkv, D, dtype, kv, page, rot, interleaved=False):
    return {"name": name, "op": "append", "N": N, "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": dtype,
            "kv": kv, "page": page, "rot": rot, "interleaved": interleaved}


def _attend(name, B, Lmax, Hq, Hkv, D, dtype, kv, page, window=0, softcap=0.0):
    return {"name": name, "op": "attend", "B": B, "Lmax": Lmax, "Hq": Hq, "Hkv": Hkv, "D": D,
            "dtype": dtype, "kv": kv, "page": page, "window": window, "softcap": softcap}


def _w4(name, T, N, K, group, dtype, fmt="u4", zeros=False, bias=False):
    return {"name": name, "op": "w4", "T": T, "N": N, "K": K, "group": group, "dtype": dtype,
            "fmt": fmt, "zeros": zeros, "bias": bias}


def listed():
    return [
        # the routed layer's one-token step: residual add and the next block's norm
        _norm("norm 1 token", 1, 6144, "bf16", "bf16"),
        # a decode batch with an odd hidden size: layer norm, one gate logit a token
        _norm("norm 64 odd", 64, 2049, "f16", "f16", kind="layer", gate="token"),
        # the 4096-token prefill chunk: fp32 residual stream, norms on both sides, channel gate
        _norm("norm 4096 sandwich", 4096, 6144, "f32", "bf16", post=True, gate="channel",
              res_scale=0.5),
        # one decode token: rotation of q and k, k and v stored
        _append("append 1 token", 1, 48, 8, 128, "bf16", "bf16", 64, 128),
        # the prefill chunk's keys and values, kept in 8 bits, half of each head rotated
        _append("append 4096 e4m3", 4096, 48, 8, 128, "bf16", "e4m3", 16, 64, True),
        # a short single conversation: the call's latency
        _attend("attend 1x777", 1, 777, 16, 2, 128, "bf16", "bf16", 16),
        # a ragged decode batch over an 8-bit cache, some slots of the batch idle
        _attend("attend 32 ragged e4m3", 32, 16384, 48, 8, 128, "bf16", "e4m3", 64),
        # one long document, odd length
        _attend("attend 1x131075", 1, 131075, 48, 8, 128, "bf16", "bf16", 64),
        # sliding window with capped scores, every head its own keys, pages that end inside tiles
        _attend("attend 33 window", 33, 5000, 16, 16, 64, "f16", "f16", 24, window=1024,
                softcap=30.0),
        # the smallest projection: latency
        _w4("w4 1 small", 1, 256, 256, 32, "f16", fmt="e2m1"),
        # one token through an attention block's square projection
        _w4("w4 1x6144", 1, 6144, 6144, 128, "bf16", zeros=True),
        # a decode batch through the fused query/key/value projection
        _w4("w4 13 fused qkv", 13, 8192, 6144, 64, "bf16", bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "append", "attend", "w4"])
    if op == "norm":
        H = _log(rng, 256, 8192)
        H = H if rng.random() < 0.4 else -(-H // 8) * 8
        T = _log(rng, 1, min(4096, 4096 * 6144 // H))
        branch = rng.choice(["bf16", "f16", "f32"])
        post = rng.random() < 0.5
        c = _norm("", T, H, rng.choice([branch, "f32"]), branch, rng.choice(["rms", "layer"]), post,
                  rng.choice(["none", "channel", "token", "full"]), rng.choice([1.0, 0.5, 1.25]))
    elif op == "append":
        Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 96, 128, 256])
        Hq = Hkv * rng.choice([1, 2, 3, 5, 6, 8])
        N = _log(rng, 1, min(4096, 4096 * 64 * 128 // ((Hq + 2 * Hkv) * D)))
        dtype = rng.choice(["bf16", "f16"])
        c = _append("", N, Hq, Hkv, D, dtype, rng.choice([dtype, "e4m3"]),
                    rng.choice([1, 5, 16, 64]), rng.choice([0, 32, 64, D]), rng.random() < 0.5)
    elif op == "attend":
        Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 96, 128, 256])
        B = _log(rng, 1, 64)
        Lmax = _log(rng, 1, min(131072, (1 << 27) // (B * Hkv * D)))
        dtype = rng.choice(["bf16", "f16"])
        c = _attend("", B, Lmax, Hkv * rng.choice([1, 4, 6, 8, 12, 16]), Hkv, D, dtype,
                    rng.choice([dtype, "e4m3"]), rng.choice([1, 5, 16, 24, 64, 128]),
                    rng.choice([0, 0, 1, 100, 4096]), rng.choice([0.0, 0.0, 30.0]))
    else:
        group = rng.choice([32, 64, 128])
        K = max(1, _log(rng, 256, 16384) // group) * group
        N = _log(rng, 16, min(16384, 8192 * 6144 // K))
        fmt = rng.choice(["u4", "e2m1"])
        c = _w4("", _log(rng, 1, 16), N, K, group, rng.choice(["bf16", "f16"]), fmt,
                fmt == "u4" and rng.random() < 0.5, rng.random() < 0.3)
    del c["name"]
    return c


# ------------------------------------------------------------------ the inputs
def _lens(c):
    """Lengths of a batch: spread evenly over 1..Lmax, the first Lmax; the last of
    every 16 slots idle."""
    out = []
    for b in range(c["B"]):
        f = 1.0 if b == 0 else (b * 0.6180339887498949) % 1.0
        out.append(0 if b % 16 == 15 else max(1, int(round(f * c["Lmax"]))))
    return out


def _pages(lens, page, gen):
    """A page table [B][columns] over a shuffled pool, and the pool's size."""
    cols = max(1, max(-(-n // page) for n in lens))
    used = sum(-(-n // page) for n in lens)
    pool = torch.randperm(used + 3, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((len(lens), cols), dtype=torch.int32)
    index = torch.zeros((len(lens), cols), dtype=torch.int64)
    at = 0
    for b, n in enumerate(lens):
        p = -(-n // page)
        index[b, :p] = torch.arange(at, at + p)
        table[b, :p] = 1
        at += p
    keep = table.cuda()
    return torch.where(keep == 1, pool[index.cuda()], torch.zeros_like(keep)), used + 3


def _inputs(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def rn(*shape, dtype="f32", s=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * s).to(DT[dtype])

    def ru(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        gate = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[c["gate"]]
        return {"x": rn(T, H, dtype=c["stream"], s=2.0), "y": rn(T, H, dtype=c["branch"]),
                "w_pre": rn(H, s=0.1) + 1, "w_post": rn(H, s=0.1) + 1 if c["post"] else None,
                "b_pre": rn(H, s=0.1) if c["kind"] == "layer" else None,
                "gate": None if gate is None else rn(*gate, dtype=c["branch"])}
    if c["op"] == "append":
        N, Hq, Hkv, D, page = (c[n] for n in ("N", "Hq", "Hkv", "D", "page"))
        start = 37  # the sequence already holds this many tokens
        table, n_pages = _pages([start + N], page, g)
        qkv = rn(N, Hq + 2 * Hkv, D, dtype=c["dtype"])  # as the fused projection writes it
        half = c["rot"] // 2
        angle = torch.arange(start + N, device="cuda", dtype=torch.float32)[:, None] * (
            10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float32) / max(half, 1)))
        kv8 = c["kv"] == "e4m3"
        pool = [torch.zeros((n_pages, Hkv, page, D), dtype=DT[c["kv"]], device="cuda")
                for _ in range(2)]
        return {"q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hkv], "v": qkv[:, Hq + Hkv:],
                "k_pages": pool[0], "v_pages": pool[1], "table": table,
                "pos": torch.arange(start, start + N, device="cuda", dtype=torch.int32),
                "seq": torch.zeros(N, device="cuda", dtype=torch.int32),
                "cos": angle.cos() if half else None, "sin": angle.sin() if half else None,
                "k_scale": ru(Hkv, lo=0.005, hi=0.02) if kv8 else None,
                "v_scale": ru(Hkv, lo=0.005, hi=0.02) if kv8 else None}
    if c["op"] == "attend":
        lens = _lens(c)
        table, n_pages = _pages(lens, c["page"], g)
        kv8 = c["kv"] == "e4m3"
        shape = (n_pages, c["Hkv"], c["page"], c["D"])
        s = 40.0 if kv8 else 1.0
        k, v = (torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, s, generator=g)
                .to(DT[c["kv"]]) for _ in range(2))
        return {"q": rn(c["B"], c["Hq"], c["D"], dtype=c["dtype"], s=1.5), "k_pages": k,
                "v_pages": v, "table": table,
                "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
                "k_scale": ru(c["Hkv"], lo=0.02, hi=0.03) if kv8 else None,
                "v_scale": ru(c["Hkv"], lo=0.02, hi=0.03) if kv8 else None}
    T, N, K, group = (c[n] for n in ("T", "N", "K", "group"))
    G = K // group
    return {"x": rn(T, K, dtype=c["dtype"]),
            "codes": torch.randint(0, 256, (N, K // 2), generator=g, device="cuda",
                                   dtype=torch.uint8),
            "scales": ru(N, G, lo=0.002, hi=0.006).to(DT[c["dtype"]]),
            "zeros": torch.randint(0, 256, (N, (G + 1) // 2), generator=g, device="cuda",
                                   dtype=torch.uint8) if c["zeros"] else None,
            "bias": rn(N, dtype=c["dtype"]) if c["bias"] else None}


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:  # the handles that a program keeps beside its weights and its cache
        from routed_expert_layer_router_gb300 import block
        if "k_pages" in s:
            s["cache"] = block.PagedKVCache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
        elif "codes" in s:
            s["linear"] = block.W4Linear(s["codes"], s["scales"], case["group"], zeros=s["zeros"],
                                         bias=s["bias"], fmt=case["fmt"])
    return s


# ------------------------------------------------------------- one call of each
EPS = 1e-5


def run(state):
    c = state["case"]
    f = globals()[("_own_" if own else "_plain_") + c["op"]]
    return f(c, state)


def _own_norm(c, s):
    from routed_expert_layer_router_gb300 import block
    r, h = block.block_norm(s["x"], s["y"], w_pre=s["w_pre"], w_post=s["w_post"],
                            b_pre=s["b_pre"], gate=s["gate"], gate_sigmoid=c["gate"] == "token",
                            res_scale=c["res_scale"], eps=EPS, kind=c["kind"])
    return {"r": r, "h": h}


def _own_append(c, s):
    q = s["cache"].append(s["k"], s["v"], s["table"], s["pos"], seq=s["seq"], q=s["q"],
                          cos=s["cos"], sin=s["sin"], interleaved=c["interleaved"])
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _own_attend(c, s):
    out, lse = s["cache"].attend(s["q"], s["table"], s["lens"], window=c["window"],
                                 softcap=c["softcap"], return_lse=True)
    return {"out": out, "lse": lse}


def _own_w4(c, s):
    return s["linear"].forward(s["x"])


def _normalize(v, kind, w, b):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    v = v * w
    return v if b is None else v + b


def _plain_norm(c, s):
    b = s["y"].float()
    if s["w_post"] is not None:
        b = _normalize(b, c["kind"], s["w_post"], None)
    if s["gate"] is not None:
        gate = s["gate"].float()
        b = b * (torch.sigmoid(gate) if c["gate"] == "token" else gate)
    r = s["x"].float() * c["res_scale"] + b
    h = _normalize(r, c["kind"], s["w_pre"], s["b_pre"])
    return {"r": r.to(s["x"].dtype), "h": h.to(s["y"].dtype)}


def _rotate(v, cos, sin, interleaved):
    """v [N][heads][D]; the first 2 * cos.shape[1] values of a head turn in pairs."""
    half = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = v[..., 0:2 * half:2], v[..., 1:2 * half:2]
    else:
        a, b = v[..., :half], v[..., half:2 * half]
    ra, rb = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((ra, rb), -1).flatten(-2) if interleaved else torch.cat((ra, rb), -1)
    return torch.cat((turned, v[..., 2 * half:]), -1)


def _plain_append(c, s):
    q, k, v, pos = s["q"].float(), s["k"].float(), s["v"].float(), s["pos"].long()
    if s["cos"] is not None:
        cos, sin = s["cos"][pos], s["sin"][pos]
        q, k = (_rotate(t, cos, sin, c["interleaved"]) for t in (q, k))
    page = s["table"][s["seq"].long(), pos // c["page"]].long()
    at = pos % c["page"]
    if c["kv"] == "e4m3":
        k = (k / s["k_scale"][:, None]).clamp(-448, 448)
        v = (v / s["v_scale"][:, None]).clamp(-448, 448)
        s["k_pages"].view(torch.uint8)[page, :, at] = k.to(DT["e4m3"]).view(torch.uint8)
        s["v_pages"].view(torch.uint8)[page, :, at] = v.to(DT["e4m3"]).view(torch.uint8)
    else:
        s["k_pages"][page, :, at] = k.to(DT[c["kv"]])
        s["v_pages"][page, :, at] = v.to(DT[c["kv"]])
    return {"q": q.to(s["q"].dtype), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_attend(c, s):
    B, Hq, Hkv, D, page = (c[n] for n in ("B", "Hq", "Hkv", "D", "page"))
    table, lens = s["table"].long(), s["lens"]
    L = table.shape[1] * page

    def rows(pool, scale):  # [B][Hkv][L][D]
        if c["kv"] == "e4m3":
            t = pool.view(torch.uint8)[table].view(DT["e4m3"]).float() * scale[:, None, None]
        else:
            t = pool[table].float()
        return t.transpose(1, 2).reshape(B, Hkv, L, D)

    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    score = q @ rows(s["k_pages"], s["k_scale"]).transpose(-1, -2) * D ** -0.5
    if c["softcap"]:
        score = c["softcap"] * torch.tanh(score / c["softcap"])
    at = torch.arange(L, device="cuda")
    seen = at < lens[:, None]
    if c["window"]:
        seen = seen & (at >= lens[:, None] - c["window"])
    seen = seen[:, None, None]
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = p @ rows(s["v_pages"], s["v_scale"]) / torch.where(total > 0, total, 1)
    lse = top + torch.log(total)
    return {"out": out.view(B, Hq, D).to(s["q"].dtype), "lse": lse.view(B, Hq)}


def _nibbles(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _plain_w4(c, s):
    N, K, group = c["N"], c["K"], c["group"]
    codes = _nibbles(s["codes"])
    if c["fmt"] == "e2m1":
        w = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")[codes.long()]
    else:
        w = codes.float()
    w = w.view(N, K // group, group)
    if c["fmt"] == "u4":
        w = w - (8.0 if s["zeros"] is None else
                 _nibbles(s["zeros"])[:, :K // group, None].float())
    w = (w * s["scales"].float()[..., None]).view(N, K)
    y = s["x"].float() @ w.t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["x"].dtype)


# ------------------------------------------- the bytes and operations of one pass
def work(c):
    if c["op"] == "norm":
        T, H, sb, bb = c["T"], c["H"], BYTES[c["stream"]], BYTES[c["branch"]]
        gate = {"none": 0, "channel": H, "token": T, "full": T * H}[c["gate"]]
        weights = H * 4 * (1 + c["post"] + (c["kind"] == "layer"))
        return {"bytes": 2 * T * H * (sb + bb) + gate * bb + weights,
                "flops": T * H * (12 if c["post"] else 8)}
    if c["op"] == "append":
        N, D, e = c["N"], c["D"], BYTES[c["dtype"]]
        return {"bytes": N * D * (2 * c["Hq"] * e + 2 * c["Hkv"] * (e + BYTES[c["kv"]]))
                + N * (c["rot"] * 4 + 8),
                "flops": N * c["rot"] * 3 * (c["Hq"] + c["Hkv"])}
    if c["op"] == "attend":
        seen = sum(min(n, c["window"]) if c["window"] else n for n in _lens(c))
        row = c["Hkv"] * c["D"]
        return {"bytes": 2 * seen * row * BYTES[c["kv"]] + seen * 4 // c["page"]
                + c["B"] * c["Hq"] * (2 * c["D"] * BYTES[c["dtype"]] + 4),
                "flops": 4 * seen * c["Hq"] * c["D"]}
    T, N, K, G = c["T"], c["N"], c["K"], c["K"] // c["group"]
    return {"bytes": N * K // 2 + N * G * 2 + (N * G // 2 if c["zeros"] else 0)
            + (N * 2 if c["bias"] else 0) + T * (N + K) * 2,
            "flops": 2 * T * N * K}


# ----------------------------------------------------- the definitions in 64 bits
def exact(c, seed):
    s = {k: (v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v)
         for k, v in _inputs(c, seed).items()}
    return globals()["_exact_" + c["op"]](c, s)


def _exact_norm(c, s):
    def norm(v, w, b):
        if c["kind"] == "layer":
            var, mean = torch.var_mean(v, -1, correction=0, keepdim=True)
            v = (v - mean) / torch.sqrt(var + EPS)
        else:
            v = v / torch.sqrt(v.pow(2).sum(-1, keepdim=True) / c["H"] + EPS)
        return torch.addcmul(torch.zeros_like(v) if b is None else b.expand_as(v), v, w)

    y = s["y"] if s["w_post"] is None else norm(s["y"], s["w_post"], None)
    if c["gate"] == "token":
        y = y / (1 + torch.exp(-s["gate"]))
    elif s["gate"] is not None:
        y = y * s["gate"]
    r = torch.add(y, s["x"], alpha=c["res_scale"])
    return {"r": r, "h": norm(r, s["w_pre"], s["b_pre"])}


def _exact_append(c, s):
    start, page, half = 37, c["page"], c["rot"] // 2
    out = {}
    for n in "qk":
        t = s[n].clone()
        if half:
            i = torch.arange(half, device="cuda")
            a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
            turn = torch.complex(s["cos"], s["sin"])[start:, None]
            z = torch.complex(s[n][..., a], s[n][..., b]) * turn
            t[..., a], t[..., b] = z.real, z.imag
        out[n] = t
    pools = {}
    for n, rows in (("k", out["k"]), ("v", s["v"])):
        pool = torch.zeros_like(s[n + "_pages"], dtype=torch.float64)
        if c["kv"] == "e4m3":
            rows = (rows / s[n + "_scale"].view(1, -1, 1)).clamp(-448, 448)
        flat = pool.transpose(1, 2).reshape(-1, c["Hkv"], c["D"])  # [page * token]
        p = torch.arange(start, start + c["N"], device="cuda")
        flat[s["table"][0].long()[p // page] * page + p % page] = rows
        pools[n + "_pages"] = flat.view(-1, page, c["Hkv"], c["D"]).transpose(1, 2)
    return {"q": out["q"], **pools}


def _exact_attend(c, s):
    B, Hq, D, page = c["B"], c["Hq"], c["D"], c["page"]
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    each = Hq // c["Hkv"]
    for b, n in enumerate(_lens(c)):
        lo = max(0, n - c["window"]) if c["window"] else 0
        if n <= lo:
            continue
        at = torch.arange(lo, n, device="cuda")
        page_of, slot = s["table"][b].long()[at // page], at % page
        for h in range(c["Hkv"]):
            k, v = s["k_pages"][page_of, h, slot], s["v_pages"][page_of, h, slot]
            if c["kv"] == "e4m3":
                k, v = k * s["k_scale"][h], v * s["v_scale"][h]
            mine = slice(h * each, (h + 1) * each)
            z = torch.einsum("gd,nd->gn", s["q"][b, mine], k) / math.sqrt(D)
            if c["softcap"]:
                z = c["softcap"] * torch.tanh(z / c["softcap"])
            lse[b, mine] = torch.logsumexp(z, -1)
            out[b, mine] = torch.softmax(z, -1) @ v
    return {"out": out, "lse": lse}


def _exact_w4(c, s):
    N, K, group = c["N"], c["K"], c["group"]
    w = torch.empty((N, K), dtype=torch.float64, device="cuda")
    for half in range(2):
        code = (s["codes"].int() >> (4 * half)) & 15
        if c["fmt"] == "e2m1":
            m, e = code & 1, (code >> 1) & 3
            mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e.double() - 1))
            w[:, half::2] = torch.where(code >= 8, -mag, mag)
        else:
            w[:, half::2] = code.double()
    for j in range(K // group):
        cols = slice(j * group, (j + 1) * group)
        if c["fmt"] == "u4":
            zero = 8 if s["zeros"] is None else ((s["zeros"][:, j // 2].int() >> (4 * (j % 2))) & 15)
            w[:, cols] -= zero if s["zeros"] is None else zero[:, None].double()
        w[:, cols] *= s["scales"][:, j, None]
    y = torch.einsum("tk,nk->tn", s["x"], w)
    return y if s["bias"] is None else y + s["bias"]
