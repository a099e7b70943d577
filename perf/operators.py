"""The fp8 operators of a block around the routed-MoE layer, as they are measured.

Four operators, in the order a transformer block on an e4m3 checkpoint calls them:

``rmsnorm``   residual addition + root-mean-square norm, written in the input's type (for the router) and as e4m3
              rows with a float32 scale per 128 columns (for the products);
``quantize``  the same e4m3 rows of an activation that needs no norm (an attention output before its projection);
``gemm``      out = A W^T on e4m3 operands: A with a scale per row and 128 columns, W with a scale per 128 x 128 block;
``ffn``       the gated FFN of a list of experts on e4m3 weights, for permuted (token, expert) pairs, followed by the
              gate-weighted combine.

With ``own`` false ``run`` computes them in plain torch operations in float32; with ``own`` true it calls the library.
"""
import math

import torch

own = False

BLOCK = 128        # columns (and weight rows) that share a scale
TOP = 448.0        # the largest e4m3 value
TINY = 2.0 ** -126   # the smallest scale: a block of zeros keeps a finite inverse
EPS = 1e-6
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _up(n, m):
    return (n + m - 1) // m * m


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decoded token of a 4096-wide model: the smallest call, launch latency
        dict(name="rmsnorm-token", op="rmsnorm", T=1, H=4096, dtype="bf16", wide=False),
        # a prefill chunk of 8192 tokens of the same model, read out of a fused projection's wider rows
        dict(name="rmsnorm-prefill", op="rmsnorm", T=8192, H=4096, dtype="bf16", wide=True),
        # a float32 stream of odd width (a partial last block, no 16-byte rows)
        dict(name="rmsnorm-odd-f32", op="rmsnorm", T=1021, H=2051, dtype="f32", wide=False),
        # attention outputs of a decode batch and of a prefill chunk, before the output projection
        dict(name="quantize-batch", op="quantize", T=32, H=7168, dtype="bf16", wide=False),
        dict(name="quantize-prefill", op="quantize", T=8192, H=7168, dtype="bf16", wide=False),
        # projection of one token: the weight's bytes
        dict(name="gemm-token", op="gemm", M=1, N=4096, K=4096, dtype="bf16"),
        # projection of a decode batch of 32 into a 7168-wide stream, kept in float32
        dict(name="gemm-batch-f32", op="gemm", M=32, N=7168, K=2048, dtype="f32"),
        # odd everything: rows, columns and a reduction that end inside a tile and a scale block
        dict(name="gemm-odd", op="gemm", M=611, N=2001, K=1133, dtype="bf16"),
        # projection of a prefill chunk: the tensor cores
        dict(name="gemm-prefill", op="gemm", M=8192, N=7168, K=4096, dtype="bf16"),
        # the routed and shared experts of one token (6 of 256, 4096 x 2048)
        dict(name="ffn-token", op="ffn", T=1, H=4096, I=2048, E=256, k=6, shared=True, skew=0.5),
        # a decode batch of 32 tokens over 8 of 128 small experts (2048 x 768)
        dict(name="ffn-batch", op="ffn", T=32, H=2048, I=768, E=128, k=8, shared=False, skew=0.5),
        # a prefill chunk of 4096 tokens over 6 of 64 experts plus the shared one: tensor cores and every weight
        dict(name="ffn-prefill", op="ffn", T=4096, H=4096, I=2048, E=64, k=6, shared=True, skew=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rmsnorm", "quantize", "gemm", "ffn"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("rmsnorm", "quantize"):
        H = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            H = _up(H, 64)
        T = min(_log(rng, 1, 16384), 8192 * 4096 // H)
        return dict(op=op, T=T, H=H, dtype=dtype, wide=rng.random() < 0.3)
    if op == "gemm":
        N, K = _log(rng, 32, 8192), _log(rng, 32, 8192)
        if rng.random() < 0.5:
            N, K = _up(N, 128), _up(K, 128)
        M = min(_log(rng, 1, 8192), 8192 * 7168 * 4096 // (N * K))
        return dict(op=op, M=M, N=N, K=K, dtype=dtype)
    unit = rng.choice([16, 128])
    H, I = _up(_log(rng, 256, 4096), unit), _up(_log(rng, 128, 2048), unit)
    E = _log(rng, 4, 64)
    k = rng.randint(1, min(8, E))
    return dict(op=op, T=min(_log(rng, 1, 4096), 4096 * 6 // k), H=H, I=I, E=E, k=k, shared=rng.random() < 0.5,
                skew=rng.choice([0.0, 0.5, 1.0, 2.0]))


def work(case):
    if case["op"] in ("rmsnorm", "quantize"):
        T, H, b = case["T"], case["H"], 4 if case["dtype"] == "f32" else 2
        scales = 4 * ((H + BLOCK - 1) // BLOCK)
        if case["op"] == "quantize":
            return {"bytes": T * (H * (b + 1) + scales), "flops": 3 * T * H}
        return {"bytes": T * (H * (4 * b + 1) + scales) + H * b, "flops": 8 * T * H}
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        kb, b = (K + BLOCK - 1) // BLOCK, 4 if case["dtype"] == "f32" else 2
        return {"bytes": M * K + N * K + M * N * b + 4 * kb * (M + (N + BLOCK - 1) // BLOCK), "flops": 2 * M * N * K}
    T, H, I, k, sh = case["T"], case["H"], case["I"], case["k"], int(case["shared"])
    # experts that get a token, where the router asks for all of them equally often
    active = case["E"] * (1.0 - (1.0 - k / case["E"]) ** T) + sh
    return {"bytes": int(active * _blob(H, I)[-1]) + T * (H + 2 * H), "flops": 6 * T * (k + sh) * H * I}


# ----------------------------------------------------------------- inputs --

def _randn(shape, gen):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)


def _codes(v):
    """float32 within +-448 (a little above rounds to it) -> e4m3."""
    return v.clamp(-TOP, TOP).to(torch.float8_e4m3fn)


def _quantize_rows(y):
    """Rows in float32 -> e4m3 codes and a scale per row and 128 columns."""
    T, H = y.shape
    g = torch.nn.functional.pad(y, (0, _up(H, BLOCK) - H)).view(T, -1, BLOCK)
    scales = (g.abs().amax(-1) / TOP).clamp_min(TINY)
    return _codes(g * (1.0 / scales)[..., None]).view(T, -1)[:, :H], scales


def _weight(n, k, gen):
    """An e4m3 weight [n][k], N(0, 0.02) before rounding, and its scale per 128 x 128 block."""
    w = torch.zeros((_up(n, BLOCK), _up(k, BLOCK)), device=DEV)
    w[:n, :k] = _randn((n, k), gen) * 0.02
    b = w.view(-1, BLOCK, w.shape[1] // BLOCK, BLOCK)
    scales = (b.abs().amax((1, 3)) / TOP).clamp_min(TINY)
    q = _codes(b / scales[:, None, :, None]).view(w.shape)
    return q[:n, :k], scales


def _blob(H, I):
    """Byte offsets in an expert's blob: gate, up, down, their scales, and the blob's size."""
    n, hb, ib = H * I, (H + BLOCK - 1) // BLOCK, (I + BLOCK - 1) // BLOCK
    s = 3 * n
    return (0, n, 2 * n, s, s + 4 * hb * ib, s + 8 * hb * ib, _up(s + 12 * hb * ib, 16))


def _blob_views(blob, H, I):
    """(codes, scales) of gate, up and down inside one expert's bytes."""
    o, hb, ib = _blob(H, I), (H + BLOCK - 1) // BLOCK, (I + BLOCK - 1) // BLOCK
    out = []
    for i, (n, k, nb, kb) in enumerate([(I, H, ib, hb), (I, H, ib, hb), (H, I, hb, ib)]):
        out.append((blob[o[i]:o[i] + n * k].view(torch.float8_e4m3fn).view(n, k),
                    blob[o[3 + i]:o[3 + i] + 4 * nb * kb].view(torch.float32).view(nb, kb)))
    return out


def _padded(q, ld):
    """Codes in rows of ld bytes (16-byte rows for the products), the padding holding other bytes."""
    buf = torch.full((q.shape[0], ld), 3.0, device=DEV).to(torch.float8_e4m3fn)
    buf.view(torch.uint8)[:, :q.shape[1]] = q.view(torch.uint8)
    return buf


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = dict(case)
    if case["op"] in ("rmsnorm", "quantize"):
        T, H, dt = case["T"], case["H"], TYPES[case["dtype"]]
        ld = H + 64 if case["wide"] else H
        x = _randn((T, ld), gen)
        x[:, ::97] *= 20.0   # the outlier channels of a residual stream
        st["x"], st["ldx"] = x.to(dt), ld
        if case["op"] == "rmsnorm":
            st["residual"] = (_randn((T, H), gen) * 3.0).to(dt)
            st["weight"] = (1.0 + 0.1 * _randn((H,), gen)).to(dt)
            st["residual_out"] = torch.empty((T, H), dtype=dt, device=DEV)
            st["y"] = torch.empty((T, H), dtype=dt, device=DEV)
        st["q"] = torch.zeros((T, _up(H, 16)), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
        st["scales"] = torch.empty((T, (H + BLOCK - 1) // BLOCK), device=DEV)
        return st
    st["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        a, st["a_scales"] = _quantize_rows(_randn((M, K), gen))
        w, st["w_scales"] = _weight(N, K, gen)
        st["ld"] = _up(K, 16)
        st["a"], st["w"] = _padded(a, st["ld"]), _padded(w, st["ld"])
        st["out"] = torch.empty((M, N), dtype=TYPES[case["dtype"]], device=DEV)
        return st
    T, H, I, E, k, sh = (case[n] for n in ("T", "H", "I", "E", "k", "shared"))
    x, st["x_scales"] = _quantize_rows(_randn((T, H), gen))
    st["x"] = x.contiguous()
    z = _randn((T, E), gen) + case["skew"] * _randn((1, E), gen)   # some experts are asked for more often
    top, ids = torch.topk(z, k, dim=1)
    st["gates"] = torch.softmax(top, 1)
    flat = ids.reshape(-1)
    perm = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0)
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k, device=DEV)
    st["offsets"], st["perm"], st["inv"] = (v.to(torch.int32) for v in (offsets, perm, inv))
    st["bounds"] = offsets.tolist()   # the host's copy, as the routing leaves it
    st["experts"] = [e for e in range(E) if st["bounds"][e + 1] > st["bounds"][e]] + ([-1] if sh else [])
    # every expert has a slot; a slot is not the expert's own number
    st["n_slots"] = E + sh
    st["slots"] = [E if e < 0 else E - 1 - e for e in st["experts"]]
    st["weights"] = torch.zeros((E + sh, _blob(H, I)[-1]), dtype=torch.uint8, device=DEV)
    for s in st["slots"]:
        for (q, sc), n, m in zip(_blob_views(st["weights"][s], H, I), (I, I, H), (H, H, I)):
            w, ws = _weight(n, m, gen)
            q.view(torch.uint8).copy_(w.view(torch.uint8))
            sc.copy_(ws)
    rows = T * k + T
    st["h"] = torch.empty((rows, I), dtype=torch.uint8, device=DEV)
    st["h_scales"] = torch.empty((rows, (I + BLOCK - 1) // BLOCK), device=DEV)
    st["y"] = torch.empty((rows, H), device=DEV)
    st["out"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    return st


# -------------------------------------------------------------------- run --

def _run_own(st):
    import moe_expert_offload_top_b200 as ft
    stream = torch.cuda.current_stream()
    if st["op"] == "rmsnorm":
        ft.ft_rmsnorm_fp8(st["x"], st["ldx"], st["residual"], st["H"], st["weight"], st["dtype"] == "bf16", st["T"],
                          st["H"], EPS, st["residual_out"], st["y"], st["q"], st["q"].shape[1], st["scales"], stream)
        return {"residual": st["residual_out"], "y": st["y"], "q": st["q"][:, :st["H"]], "scales": st["scales"]}
    if st["op"] == "quantize":
        ft.ft_quantize_fp8(st["x"], st["ldx"], st["dtype"] == "bf16", st["T"], st["H"], st["q"], st["q"].shape[1],
                           st["scales"], stream)
        return {"q": st["q"][:, :st["H"]], "scales": st["scales"]}
    if st["op"] == "gemm":
        ft.ft_gemm_fp8(st["a"], st["ld"], st["a_scales"], st["w"], st["ld"], st["w_scales"], st["M"], st["N"], st["K"],
                       st["dtype"] == "bf16", st["out"], st["N"], st["err"], stream)
        return st["out"]
    ft.ft_expert_ffn_fp8(st["x"], st["H"], st["x_scales"], st["T"], st["H"], st["I"], st["k"], st["weights"],
                         st["n_slots"], st["experts"], st["slots"], st["offsets"], st["perm"], st["h"],
                         st["h_scales"], st["y"], st["err"], stream)
    ft.ft_combine(st["y"], st["gates"], st["inv"], st["T"], st["H"], st["k"], st["shared"], True, st["out"], stream)
    return st["out"]


def _spread_rows(q, scales):
    """e4m3 rows -> float32."""
    return q.float() * scales.repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _spread_blocks(q, scales):
    """An e4m3 weight with block scales -> float32."""
    s = scales.repeat_interleave(BLOCK, 0)[:q.shape[0]].repeat_interleave(BLOCK, 1)[:, :q.shape[1]]
    return q.float() * s


def run(state):
    if own:
        return _run_own(state)
    st = state
    if st["op"] in ("rmsnorm", "quantize"):
        H = st["H"]
        v = st["x"][:, :H].float()
        if st["op"] == "quantize":
            q, scales = _quantize_rows(v)
            return {"q": q, "scales": scales}
        dt = TYPES[st["dtype"]]
        r = (v + st["residual"].float()).to(dt)
        v = r.float()
        y = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * st["weight"].float()
        q, scales = _quantize_rows(y)
        return {"residual": r, "y": y.to(dt), "q": q, "scales": scales}
    if st["op"] == "gemm":
        K = st["K"]
        a = _spread_rows(st["a"][:, :K], st["a_scales"])
        w = _spread_blocks(st["w"][:, :K], st["w_scales"])
        return (a @ w.t()).to(TYPES[st["dtype"]])
    T, H, I, k = st["T"], st["H"], st["I"], st["k"]
    x = _spread_rows(st["x"], st["x_scales"])
    y = torch.zeros((T * k + T, H), device=DEV)
    for e, s in zip(st["experts"], st["slots"]):
        gate, up, down = (_spread_blocks(*m) for m in _blob_views(st["weights"][s], H, I))
        lo, hi = (T * k, T * k + T) if e < 0 else (st["bounds"][e], st["bounds"][e + 1])
        xe = x if e < 0 else x[st["perm"][lo:hi].long() // k]
        a = xe @ gate.t()
        h = a / (1.0 + torch.exp(-a)) * (xe @ up.t())
        y[lo:hi] = _spread_rows(*_quantize_rows(h)) @ down.t()
    out = (y[st["inv"].long()].view(T, k, H) * st["gates"][..., None]).sum(1)
    if st["shared"]:
        out += y[T * k:]
    return out.to(torch.bfloat16)


# ------------------------------------------------------------------ exact --

def _scale64(v, axes):
    """Block scales of float64 blocks, as the float32 numbers that are stored."""
    return (v.abs().amax(axes, keepdim=True) / TOP).clamp_min(TINY).float().double()


def _rows64(y):
    """(codes, scales) of float64 rows, block by block."""
    qs, ss = [], []
    for c in range(0, y.shape[1], BLOCK):
        b = y[:, c:c + BLOCK]
        s = _scale64(b, (1,))
        qs.append((b / s).clamp(-TOP, TOP).to(torch.float8_e4m3fn))
        ss.append(s)
    return torch.cat(qs, 1), torch.cat(ss, 1)


def _product64(a, sa, w, sw):
    """sum over 128-blocks of (a block . w block) times the row's and the block's scale, in float64."""
    sw = sw.double().repeat_interleave(BLOCK, 0)[:w.shape[0]]
    out = torch.zeros((a.shape[0], w.shape[0]), dtype=torch.float64, device=a.device)
    for kb in range((a.shape[1] + BLOCK - 1) // BLOCK):
        c = slice(kb * BLOCK, min((kb + 1) * BLOCK, a.shape[1]))
        left = a[:, c].double() * sa[:, kb].double()[:, None]
        out.addmm_(left, (w[:, c].double() * sw[:, kb][:, None]).t())
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quantize":
        q, scales = _rows64(st["x"][:, :case["H"]].double())
        return {"q": q, "scales": scales}
    if case["op"] == "rmsnorm":
        dt = TYPES[case["dtype"]]
        r = (st["x"][:, :case["H"]].double() + st["residual"].double()).to(dt)   # the stream as it is stored
        v = r.double()
        y = v / torch.sqrt((v ** 2).sum(1, keepdim=True) / case["H"] + EPS) * st["weight"].double()
        q, scales = _rows64(y)
        return {"residual": r.double(), "y": y, "q": q, "scales": scales}
    if case["op"] == "gemm":
        K = case["K"]
        return _product64(st["a"][:, :K], st["a_scales"], st["w"][:, :K], st["w_scales"])
    T, k = case["T"], case["k"]
    out = torch.zeros((T, case["H"]), dtype=torch.float64, device=DEV)
    for e, s in zip(st["experts"], st["slots"]):
        (g, sg), (u, su), (d, sd) = _blob_views(st["weights"][s], case["H"], case["I"])
        if e < 0:
            tok, weight = torch.arange(T, device=DEV), torch.ones(T, dtype=torch.float64, device=DEV)
        else:
            pairs = st["perm"][st["bounds"][e]:st["bounds"][e + 1]].long()
            tok, weight = pairs // k, st["gates"].reshape(-1)[pairs].double()
        a = _product64(st["x"][tok], st["x_scales"][tok], g, sg)
        h = a * torch.sigmoid(a) * _product64(st["x"][tok], st["x_scales"][tok], u, su)
        out.index_add_(0, tok, _product64(*_rows64(h), d, sd) * weight[:, None])
    return out
