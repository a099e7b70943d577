"""GPU parity of the fp8 operators against the float64 oracle (oracle/fp8.py), at the sizes and
inputs where they can go wrong: one row, rows and widths that end inside a tile or a scale
block, odd widths and strides, blocks of zeros, NaN and infinities, experts without tokens,
memory around the outputs, other streams and captured graphs.

Tolerances.  e4m3 codes: equal wherever the exact quotient is further from a tie than the f32
error of the value it rounds; scales and f32 values: the roundings counted beside each bound."""
import numpy as np
import pytest
import torch

import moe_expert_offload_top_b200 as ft
from oracle import fp8, moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
U32 = 2.0 ** -24     # half an f32 step of 1
UBF = 2.0 ** -8      # half a bf16 step of 1
EPS = 1e-5


def _dt(bf16):
    return torch.bfloat16 if bf16 else torch.float32


def _err():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _np(t):
    return t.detach().double().cpu().numpy()


def _bytes(t):
    return t.cpu().numpy()


def check_codes(codes, scales, y, rel, absolute=0.0):
    """codes / scales hold the quantised rows of the float64 y, whose own f32 error is at most
    rel * |y| + absolute.  The scale adds a division and the inverse another, and the product a
    rounding: 4 more roundings."""
    s = fp8.row_scales(y)
    d = fp8.spread(absolute, y.shape[1]) if np.ndim(absolute) else absolute
    tol_s = (rel + 4 * U32) * s + np.max(absolute, initial=0.0) / fp8.TOP
    assert (np.abs(scales - s) <= tol_s).all()
    ss = fp8.spread(s, y.shape[1])
    q = y / ss
    want = fp8.round_e4m3(q)
    got = fp8.decode(codes)
    # the value that was rounded differs from q by at most:
    slack = (2 * rel + 8 * U32) * np.abs(q) + 2 * d / ss
    off = got != want
    near_tie = fp8.tie_distance(q) * np.abs(q) <= slack + 1e-300
    beyond_top = np.abs(q) >= fp8.TOP * (1 - 1e-3)
    assert (~off | near_tie | beyond_top).all(), "codes differ away from a tie"
    assert (np.abs(got - q) <= 0.5 * fp8.step(q) * (1 + 1e-6) + slack).all()


# ------------------------------------------------------------- norm, rows --

NORM_SHAPES = [  # T, H
    (1, 1), (1, 127), (3, 128), (2, 129), (5, 200), (7, 256), (64, 1000), (297, 264), (300, 2048), (1, 4096), (33, 7168),
    (300, 2051), (2, 9000), (301, 9000), (1, 32768), (2, 32767)]


def _norm_bound(H):
    """Relative f32 error of a normed value: the sum of squares is a chain of at most 32 per thread
    (8 elements x 4 chunks), 5 steps in a warp and 32 warps, each rounding 2^-24 of a sum of
    positive terms, halved by the square root; then mean, eps, square root, inverse and two products."""
    return (69 / 2 + 8) * U32


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,H", NORM_SHAPES)
def test_rmsnorm(T, H, bf16):
    g = torch.Generator().manual_seed(T * 40000 + H)
    ldx, ldr, ldq = (H, H, H) if (T + H) % 2 else (H + 8, H + 16, H + 8)
    x = (torch.randn((T, ldx), generator=g) * 2).to(_dt(bf16)).to(DEV)
    res = (torch.randn((T, ldr), generator=g) * 5).to(_dt(bf16)).to(DEV)
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(_dt(bf16)).to(DEV)
    res_out = torch.full((T + 1, ldr), 77.0, dtype=_dt(bf16), device=DEV)
    y = torch.full((T + 1, H), 77.0, dtype=_dt(bf16), device=DEV)
    q = torch.full((T + 1, ldq), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((T + 1, fp8.blocks(H)), -1.0, device=DEV)
    ft.ft_rmsnorm_fp8(x, ldx, res, ldr, w, bf16, T, H, EPS, res_out, y, q, ldq, s)
    r32 = (x[:, :H].float() + res[:, :H].float()).to(_dt(bf16))
    assert torch.equal(res_out[:T, :H], r32)                       # one f32 addition, one rounding: exact
    assert (res_out[T] == 77).all() and (res_out[:, H:] == 77).all() and (y[T] == 77).all()
    assert (q[T] == 0x55).all() and (q[:, H:] == 0x55).all() and (s[T] == -1).all()
    ref = fp8.rmsnorm(_np(r32), _np(w), EPS)
    rel = _norm_bound(H)
    tol = rel + (UBF if bf16 else 0.0)
    assert (np.abs(_np(y[:T]) - ref) <= tol * np.abs(ref) * (1 + UBF) + 1e-38).all()
    check_codes(_bytes(q[:T, :H]), _np(s[:T]), ref, rel)


@pytest.mark.parametrize("bf16", [True, False])
def test_rmsnorm_in_place_and_optional_outputs(bf16):
    T, H = 19, 640
    x = torch.randn((T, H), device=DEV).to(_dt(bf16))
    w = torch.randn(H, device=DEV).to(_dt(bf16))
    res = torch.randn((T, H), device=DEV).to(_dt(bf16))
    outs = []
    for res_out in (None, res.clone(), x.clone()):
        y, q = torch.zeros_like(x), torch.zeros((T, H), dtype=torch.uint8, device=DEV)
        s = torch.zeros((T, 5), device=DEV)
        xi, ri = x, res
        if res_out is not None and torch.equal(res_out, res):
            ri = res_out       # the stream in place
        elif res_out is not None:
            xi = res_out       # over x
        ft.ft_rmsnorm_fp8(xi, H, ri, H, w, bf16, T, H, EPS, res_out, y, q, H, s)
        outs.append((y, q, s))
        if res_out is not None:
            assert torch.equal(res_out, (x.float() + res.float()).to(_dt(bf16)))
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))
    y2, q2, s2 = torch.zeros_like(outs[0][0]), torch.zeros_like(outs[0][1]), torch.zeros_like(outs[0][2])
    ft.ft_rmsnorm_fp8(x, H, res, H, w, bf16, T, H, EPS, None, y2, None, H, None)
    ft.ft_rmsnorm_fp8(x, H, res, H, w, bf16, T, H, EPS, None, None, q2, H, s2)
    assert torch.equal(y2, outs[0][0]) and torch.equal(q2, outs[0][1]) and torch.equal(s2, outs[0][2])
    # no residual: the norm of x
    ft.ft_rmsnorm_fp8(x, H, None, 0, w, bf16, T, H, EPS, None, y2, None, H, None)
    ref = fp8.rmsnorm(_np(x), _np(w), EPS)
    assert (np.abs(_np(y2) - ref) <= (_norm_bound(H) + (UBF if bf16 else 0)) * np.abs(ref) * (1 + UBF)).all()


def test_unaligned_rows_give_the_same_codes():
    """An address that rules out wide accesses changes the kernel, not what it computes (up to the
    order of the sum of squares)."""
    T, H = 40, 512
    flat = torch.randn(T * H + 1, device=DEV)
    x = flat[1:].view(T, H)
    w = torch.ones(H, device=DEV)
    q, s, y = torch.zeros((T, H), dtype=torch.uint8, device=DEV), torch.zeros((T, 4), device=DEV), torch.zeros_like(x)
    ft.ft_rmsnorm_fp8(x, H, None, 0, w, False, T, H, EPS, None, y, q, H, s)
    check_codes(_bytes(q), _np(s), fp8.rmsnorm(_np(x), np.ones(H), EPS), _norm_bound(H))
    a, b = (torch.zeros((T, H), dtype=torch.uint8, device=DEV) for _ in range(2))
    sa, sb = torch.zeros((T, 4), device=DEV), torch.zeros((T, 4), device=DEV)
    ft.ft_quantize_fp8(x, H, False, T, H, a, H, sa)
    ft.ft_quantize_fp8(x.clone(), H, False, T, H, b, H, sb)
    assert torch.equal(a, b) and torch.equal(sa, sb)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,H", NORM_SHAPES)
def test_quantize(T, H, bf16):
    g = torch.Generator().manual_seed(H * 7 + T)
    x = torch.randn((T, H + 24), generator=g) * torch.exp2(torch.randint(-30, 30, (T, 1), generator=g).float())
    x[:, :: max(1, H // 3)] = 0
    x = x.to(_dt(bf16)).to(DEV)
    q = torch.full((T, H + 8), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.zeros((T, fp8.blocks(H)), device=DEV)
    ft.ft_quantize_fp8(x, H + 24, bf16, T, H, q, H + 8, s)
    assert (q[:, H:] == 0x55).all()
    check_codes(_bytes(q[:, :H]), _np(s), _np(x[:, :H]), 0.0)


@pytest.mark.parametrize("H", [512, 511])
def test_zero_tiny_nan_and_infinite_blocks(H):
    x = torch.randn((6, H), device=DEV)
    x[0] = 0
    x[1, :128] = 0
    x[1, 128:256] = 1e-41           # a block of subnormals: the smallest scale, codes below its step
    x[2, 130] = float("nan")
    x[3, 5] = float("inf")
    x[4, 300] = -float("inf")
    q, s = torch.zeros((6, H), dtype=torch.uint8, device=DEV), torch.zeros((6, 4), device=DEV)
    ft.ft_quantize_fp8(x, H, False, 6, H, q, H, s)
    v, sc = fp8.decode(_bytes(q)), _np(s)
    assert (v[0] == 0).all() and (sc[0] == fp8.TINY).all() and (v[1, :256] == 0).all() and sc[1, 1] == fp8.TINY
    with np.errstate(invalid="ignore"):
        full = v * fp8.spread(sc, H)
    assert np.isnan(full[2, 128:256]).all() and np.isnan(full[3, :128]).all() and np.isnan(full[4, 256:384]).all()
    for row, bad in ((2, 1), (3, 0), (4, 2)):   # the other blocks are those of a row without the bad value
        clean = x[row].clone()
        clean[128 * bad:128 * bad + 128] = 1.0
        q2, s2 = torch.zeros((1, H), dtype=torch.uint8, device=DEV), torch.zeros((1, 4), device=DEV)
        ft.ft_quantize_fp8(clean, H, False, 1, H, q2, H, s2)
        keep = [b for b in range(4) if b != bad]
        assert torch.equal(s[row, keep], s2[0, keep])
        for b in keep:
            assert torch.equal(q[row, 128 * b:128 * b + 128], q2[0, 128 * b:128 * b + 128])


def test_norm_keeps_a_bad_row_to_itself():
    T, H = 5, 384
    x = torch.randn((T, H), device=DEV)
    w = torch.ones(H, device=DEV)
    good = [0, 1, 3, 4]
    y0, y1 = torch.zeros_like(x), torch.zeros_like(x)
    q, s = torch.zeros((T, H), dtype=torch.uint8, device=DEV), torch.zeros((T, 3), device=DEV)
    ft.ft_rmsnorm_fp8(x, H, None, 0, w, False, T, H, EPS, None, y0, q, H, s)
    x[2, 7] = float("nan")
    ft.ft_rmsnorm_fp8(x, H, None, 0, w, False, T, H, EPS, None, y1, q, H, s)
    assert torch.equal(y0[good], y1[good]) and torch.isnan(y1[2]).all() and torch.isnan(s[2]).all()


# ---------------------------------------------------------------- product --

def _operand(rows, K, ld, gen, codes=None):
    """Random e4m3 bytes of every magnitude (no NaN), rows ld apart, the padding full of NaN codes."""
    c = torch.randint(0, 127, (rows, K), generator=gen) | (torch.randint(0, 2, (rows, K), generator=gen) << 7)
    buf = torch.full((rows, ld), 0x7F, dtype=torch.uint8)
    buf[:, :K] = c.to(torch.uint8) if codes is None else codes
    return buf.to(DEV)


def _scales(shape, gen):
    return torch.exp2(torch.rand(shape, generator=gen) * 12 - 10).to(DEV)


GEMM_SHAPES = [  # M, N, K
    (1, 1, 1), (1, 16, 16), (1, 129, 128), (2, 300, 127), (3, 64, 129), (1, 4096, 1024), (16, 512, 640), (17, 128, 256),
    (31, 2001, 1133), (33, 256, 4096), (64, 768, 2048), (65, 130, 384), (127, 384, 257), (128, 256, 512),
    (129, 257, 1000), (16, 16384, 2048), (32, 16384, 4096),
    (200, 1000, 200), (300, 520, 136), (513, 1300, 900), (1024, 2048, 512)]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("M,N,K", GEMM_SHAPES)
def test_gemm(M, N, K, bf16):
    gen = torch.Generator().manual_seed(M * 131 + N * 17 + K)
    ld = -(-K // 16) * 16 + (16 if (M + N) % 2 else 0)
    a, w = _operand(M, K, ld, gen), _operand(N, K, ld, gen)
    sa, sw = _scales((M, fp8.blocks(K)), gen), _scales((fp8.blocks(N), fp8.blocks(K)), gen)
    ldo = N if M % 2 else N + 5
    out = torch.full((M + 1, ldo), 77.0, dtype=_dt(bf16), device=DEV)
    err = _err()
    ft.ft_gemm_fp8(a, ld, sa, w, ld, sw, M, N, K, bf16, out, ldo, err)
    assert err.item() == 0
    ref, l1 = fp8.product(fp8.decode(_bytes(a)[:, :K]), _np(sa), fp8.decode(_bytes(w)[:, :K]), _np(sw))
    tol = fp8.product_bound(l1, K) + (UBF * np.abs(ref) * (1 + UBF) if bf16 else 0.0)
    assert (np.abs(_np(out[:M, :N]) - ref) <= tol).all(), np.max(np.abs(_np(out[:M, :N]) - ref) / tol)
    assert (out[M] == 77).all() and (out[:, N:] == 77).all()


def test_gemm_nan_codes_and_zero_rows():
    M, N, K = 140, 300, 384
    gen = torch.Generator().manual_seed(1)
    a, w = _operand(M, K, K, gen), _operand(N, K, K, gen)
    a[5] = 0
    a[130, 17] = 0x7F
    w[299, 380] = 0xFF
    sa, sw = _scales((M, 3), gen), _scales((3, 3), gen)
    sa[6] = 0.0
    for rows in (M, 20):     # both kernels' tile shapes
        out, err = torch.zeros((rows, N), device=DEV), _err()
        ft.ft_gemm_fp8(a, K, sa, w, K, sw, rows, N, K, False, out, N, err)
        bad = torch.isnan(out)
        want = torch.zeros_like(bad)
        want[:, 299] = True
        if rows > 130:
            want[130] = True
        assert torch.equal(bad, want)
        assert (out[5, :299] == 0).all() and (out[6, :299] == 0).all()


def test_gemm_streams_and_repeats_are_equal():
    """The same call on other streams at once, and again, gives the same bits."""
    gen = torch.Generator().manual_seed(2)
    for M, N, K in ((4, 1024, 4096), (260, 700, 1024)):
        a, w = _operand(M, K, K, gen), _operand(N, K, K, gen)
        sa, sw = _scales((M, K // 128), gen), _scales((fp8.blocks(N), K // 128), gen)
        first, err = torch.zeros((M, N), device=DEV), _err()
        ft.ft_gemm_fp8(a, K, sa, w, K, sw, M, N, K, False, first, N, err)
        torch.cuda.synchronize()
        outs = [torch.zeros((M, N), device=DEV) for _ in range(8)]
        streams = [torch.cuda.Stream() for _ in range(4)]
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            ft.ft_gemm_fp8(a, K, sa, w, K, sw, M, N, K, False, o, N, err, streams[i % 4])
        torch.cuda.synchronize()
        assert err.item() == 0 and all(torch.equal(o, first) for o in outs)


# ------------------------------------------------------------- expert FFN --

class Ffn:
    """One set of experts and routed tokens, with the oracle's view of both."""

    def __init__(self, T, H, I, E, k, shared, seed, empty=(), skew=0.0, pad=0):
        rng = np.random.default_rng(seed)
        self.T, self.H, self.I, self.E, self.k, self.shared = T, H, I, E, k, shared
        self.n_slots = E + 2
        order = rng.permutation(self.n_slots)
        self.blob = ft.ft_fp8_blob_bytes(H, I)
        arena = rng.integers(0, 255, (self.n_slots, self.blob), dtype=np.uint8)   # unused slots: any bytes
        allowed = [e for e in range(E) if e not in empty]
        z = rng.standard_normal((T, E)) + skew * rng.standard_normal((1, E))
        z[:, list(empty)] = -1e9
        self.ids = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
        assert len(allowed) >= k
        self.experts, self.slots, self.parts = [], [], {}
        for e in list(range(E)) + ([-1] if shared else []):
            self.experts.append(e)                      # experts without tokens stay in the list
            self.slots.append(int(order[e if e >= 0 else E]))
            m = [rng.standard_normal(s) * 0.05 for s in ((I, H), (I, H), (H, I))]
            arena[self.slots[-1]] = fp8.blob(*m)
            self.parts[e] = fp8.blob_parts(arena[self.slots[-1]], H, I)
        self.weights = torch.from_numpy(arena).to(DEV)
        xv, self.xs_np = fp8.quantize_rows(rng.standard_normal((T, H)))
        self.x_np = xv
        ldx = H + pad
        buf = np.full((T, ldx), 0x7F, dtype=np.uint8)
        buf[:, :H] = fp8.encode(xv)
        self.x, self.ldx = torch.from_numpy(buf).to(DEV), ldx
        self.xs = torch.from_numpy(self.xs_np.astype(np.float32)).to(DEV)
        ids = torch.from_numpy(self.ids).to(DEV)
        self.counts, self.offsets = (torch.zeros(n, dtype=torch.int32, device=DEV) for n in (E, E + 1))
        self.perm, self.inv = (torch.zeros(T * k, dtype=torch.int32, device=DEV) for _ in range(2))
        ft.ft_permute(ids, T, k, E, self.counts, self.offsets, self.perm, self.inv)
        self.buffers()

    def buffers(self):
        rows = self.T * self.k + self.T
        self.h = torch.full((rows, self.I), 0x55, dtype=torch.uint8, device=DEV)
        self.hs = torch.full((rows, fp8.blocks(self.I)), -1.0, device=DEV)
        self.y = torch.full((rows, self.H), 77.0, device=DEV)
        self.err = _err()

    def run(self, stream=None, experts=None, slots=None):
        ft.ft_expert_ffn_fp8(self.x, self.ldx, self.xs, self.T, self.H, self.I, self.k, self.weights, self.n_slots,
                             self.experts if experts is None else experts, self.slots if slots is None else slots,
                             self.offsets, self.perm, self.h, self.hs, self.y, self.err, stream)

    def check(self, skip=()):
        assert self.err.item() == 0
        off, perm = _bytes(self.offsets), _bytes(self.perm)
        h, hs, y = _bytes(self.h), _np(self.hs), _np(self.y)
        owned = np.zeros(len(y), dtype=bool)
        for e in self.experts:
            if e in skip:
                continue
            lo, hi = (self.T * self.k, self.T * self.k + self.T) if e < 0 else (off[e], off[e + 1])
            if lo == hi:
                continue
            owned[lo:hi] = True
            tok = np.arange(self.T) if e < 0 else perm[lo:hi] // self.k
            (g, sg), (u, su), (d, sd) = self.parts[e]
            a, la = fp8.product(self.x_np[tok], self.xs_np[tok], g, sg)
            b, lb = fp8.product(self.x_np[tok], self.xs_np[tok], u, su)
            ref = fp8.silu(a) * b
            # |silu'| <= 1.1; expf (2 ulp), sum, division and product: 8 roundings
            bound = (1.1 * fp8.product_bound(la, self.H) * (np.abs(b) + fp8.product_bound(lb, self.H)) +
                     np.abs(fp8.silu(a)) * fp8.product_bound(lb, self.H) + 8 * U32 * np.abs(ref))
            worst = np.array([[bound[r, 128 * c:128 * c + 128].max() for c in range(fp8.blocks(self.I))]
                              for r in range(len(tok))])
            check_codes(h[lo:hi], hs[lo:hi], ref, 0.0, worst)
            # y from the rows that were stored: their codes are checked above
            yr, ly = fp8.product(fp8.decode(h[lo:hi]), hs[lo:hi], d, sd)
            tol = fp8.product_bound(ly, self.I)
            assert (np.abs(y[lo:hi] - yr) <= tol).all(), np.max(np.abs(y[lo:hi] - yr) / tol)
        assert (y[~owned] == 77).all() and (h[~owned] == 0x55).all() and (hs[~owned] == -1).all()


FFN_SHAPES = [  # T, H, I, E, k, shared, empty, skew
    (1, 256, 128, 4, 2, False, (), 0.0), (1, 128, 128, 1, 1, True, (), 0.0), (1, 16, 16, 3, 3, True, (), 0.0),
    (5, 144, 80, 6, 2, True, (0, 3), 0.0), (16, 512, 384, 8, 4, False, (), 1.0), (17, 256, 128, 2, 1, True, (), 0.0),
    (33, 400, 144, 5, 2, False, (4,), 2.0), (64, 256, 256, 4, 2, True, (), 0.0), (130, 384, 272, 3, 2, True, (1,), 0.0),
    (300, 256, 128, 16, 4, True, (2, 15), 2.0), (700, 512, 256, 4, 2, False, (), 0.5), (129, 128, 640, 2, 2, True, (), 0.0),
    # the shared expert launched apart from experts with few tokens
    (40, 256, 256, 16, 2, True, (), 0.0), (100, 512, 272, 32, 2, True, (3,), 1.0)]


@pytest.mark.parametrize("T,H,I,E,k,shared,empty,skew", FFN_SHAPES)
def test_expert_ffn(T, H, I, E, k, shared, empty, skew):
    f = Ffn(T, H, I, E, k, shared, seed=T + H + I, empty=empty, skew=skew, pad=16 * (T % 2))
    f.run()
    f.check()


@pytest.mark.parametrize("T", [3, 90])
def test_expert_ffn_leaves_rows_of_unlisted_experts(T):
    f = Ffn(T, 256, 192, 6, 3, True, seed=5)
    drop = {1, 4, -1}
    keep = [(e, s) for e, s in zip(f.experts, f.slots) if e not in drop]
    f.run(experts=[e for e, _ in keep], slots=[s for _, s in keep])
    f.check(skip=drop)


def test_expert_ffn_many_tiles_per_cta():
    """Several tiles for every CTA: buffers, barriers and ring stages wrap around across tiles."""
    f = Ffn(1500, 1024, 640, 32, 4, True, seed=9, skew=1.0)
    f.run()
    f.check()


def test_expert_ffn_one_expert_owns_every_pair():
    f = Ffn(150, 256, 128, 3, 1, False, seed=11, empty=(0, 2))
    f.run()
    f.check()


@pytest.mark.parametrize("T,H,I", [(60, 256, 128), (47, 1024, 144)])
def test_expert_ffn_crowded_expert_in_a_long_list(T, H, I):
    """One of 32 experts has every token, where the even share is two: its CTAs take its tokens in turn."""
    f = Ffn(T, H, I, 32, 1, False, seed=13, empty=tuple(e for e in range(32) if e != 7))
    f.run()
    f.check()


@pytest.mark.parametrize("T", [1, 24, 400])
def test_captured_and_replayed(T):
    """A captured call computes from what its inputs hold at the replay."""
    f = Ffn(T, 256, 256, 5, 2, True, seed=21)
    x = torch.randn((T, 256), device=DEV)
    w = torch.ones(256, device=DEV)
    out = torch.zeros((T, 256), device=DEV)
    gates = torch.full((T, 2), 0.5, device=DEV)

    def chain(stream):
        ft.ft_rmsnorm_fp8(x, 256, None, 0, w, False, T, 256, EPS, None, None, f.x, f.ldx, f.xs, stream)
        f.run(stream)
        ft.ft_combine(f.y, gates, f.inv, T, 256, 2, True, False, out, stream)

    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        chain(s)
    for seed in (1, 2):
        x.copy_(torch.randn((T, 256), generator=torch.Generator().manual_seed(seed)))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        chain(None)
        torch.cuda.synchronize()
        assert torch.equal(got, out)
    f.x_np, f.xs_np = fp8.decode(_bytes(f.x)[:, :256]), _np(f.xs)
    f.check()


def test_layer_on_fp8_rows():
    """The operators in a row, as a block uses them: norm -> routing -> experts -> combine -> quantise ->
    projection, each step against the oracle from the bytes the step before it left."""
    T, H, I, E, k, N = 24, 512, 256, 8, 2, 320
    rng = np.random.default_rng(3)
    f = Ffn(T, H, I, E, k, True, seed=33)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(DEV).bfloat16()
    stream = torch.from_numpy(rng.standard_normal((T, H))).to(DEV).bfloat16()
    w = torch.from_numpy(1 + 0.1 * rng.standard_normal(H)).to(DEV).bfloat16()
    y = torch.zeros_like(x)
    ft.ft_rmsnorm_fp8(x, H, stream, H, w, True, T, H, EPS, stream, y, f.x, f.ldx, f.xs)
    router = torch.from_numpy(rng.standard_normal((E, H)).astype(np.float32) * 0.02).to(DEV)
    logits, gates = torch.zeros((T, E), device=DEV), torch.zeros((T, k), device=DEV)
    ids = torch.zeros((T, k), dtype=torch.int32, device=DEV)
    ft.ft_route_decode(y, True, router, T, H, E, k, "sigmoid", logits, ids, gates, f.counts, f.offsets, f.perm, f.inv,
                       _err())
    f.run()
    mixed = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    ft.ft_combine(f.y, gates, f.inv, T, H, k, True, True, mixed)
    mq, ms = torch.zeros((T, H), dtype=torch.uint8, device=DEV), torch.zeros((T, H // 128), device=DEV)
    ft.ft_quantize_fp8(mixed, H, True, T, H, mq, H, ms)
    wq, ws = fp8.quantize_weight(rng.standard_normal((N, H)) * 0.02)
    wd, wsd = torch.from_numpy(wq).to(DEV), torch.from_numpy(ws).to(DEV)
    out = torch.zeros((T, N), device=DEV)
    ft.ft_gemm_fp8(mq, H, ms, wd, H, wsd, T, N, H, False, out, N, f.err)
    torch.cuda.synchronize()

    ref = fp8.rmsnorm(_np(stream), _np(w), EPS)
    check_codes(_bytes(f.x)[:, :H], _np(f.xs), ref, _norm_bound(H))
    f.x_np, f.xs_np = fp8.decode(_bytes(f.x)[:, :H]), _np(f.xs)
    f.check()
    yy, g, inv = _np(f.y), _np(gates), _bytes(f.inv).reshape(T, k)
    want = sum(g[:, j, None] * yy[inv[:, j]] for j in range(k)) + yy[T * k:]
    l1 = sum(g[:, j, None] * np.abs(yy[inv[:, j]]) for j in range(k)) + np.abs(yy[T * k:])
    assert (np.abs(_np(mixed) - want) <= UBF * np.abs(want) * (1 + UBF) + 8 * U32 * l1).all()
    check_codes(_bytes(mq), _np(ms), _np(mixed), 0.0)
    ref, l1 = fp8.product(fp8.decode(_bytes(mq)), _np(ms), fp8.decode(wq), ws)
    assert (np.abs(_np(out) - ref) <= fp8.product_bound(l1, H)).all()


def test_rows_and_products_past_2_to_31_elements():
    """Row offsets need 64 bits; the last rows are checked."""
    T, H = 70000, 32752
    x = torch.randn((1, H), device=DEV).bfloat16().repeat(T, 1)
    x[T - 2] *= 3
    q, s = torch.zeros((T, H), dtype=torch.uint8, device=DEV), torch.zeros((T, fp8.blocks(H)), device=DEV)
    ft.ft_quantize_fp8(x, H, True, T, H, q, H, s)
    check_codes(_bytes(q[T - 3:]), _np(s[T - 3:]), _np(x[T - 3:]), 0.0)
    del x, q, s
    gen = torch.Generator().manual_seed(8)
    M, N, K = 66000, 33000, 16
    a, w = _operand(1, K, K, gen).repeat(M, 1), _operand(N, K, K, gen)
    a[M - 2] = _operand(1, K, K, gen)
    sa, sw = _scales((M, 1), gen), _scales((fp8.blocks(N), 1), gen)
    out, err = torch.zeros((M, N), dtype=torch.bfloat16, device=DEV), _err()
    ft.ft_gemm_fp8(a, K, sa, w, K, sw, M, N, K, True, out, N, err)
    ref, l1 = fp8.product(fp8.decode(_bytes(a[M - 3:])), _np(sa[M - 3:]), fp8.decode(_bytes(w)), _np(sw))
    tol = fp8.product_bound(l1, K) + UBF * np.abs(ref) * (1 + UBF)
    assert err.item() == 0 and (np.abs(_np(out[M - 3:]) - ref) <= tol).all()


def test_ffn_past_2_to_31_elements():
    T, H, I, E = 40000, 7168, 128, 8      # every token takes every expert: 320000 rows of y and 40000 shared
    gen = torch.Generator().manual_seed(4)
    rng = np.random.default_rng(4)
    row = _operand(1, H, H, gen)
    x = row.repeat(T, 1)
    x[T - 1] = _operand(1, H, H, gen)
    xs = _scales((T, H // 128), gen)
    raw = [fp8.blob(*[rng.standard_normal(s) * 0.05 for s in ((I, H), (I, H), (H, I))]) for _ in range(E + 1)]
    weights = torch.from_numpy(np.stack(raw)).to(DEV)
    offsets = (torch.arange(E + 1, device=DEV) * T).int()
    perm = (torch.arange(T, device=DEV)[None, :] * E + torch.arange(E, device=DEV)[:, None]).reshape(-1).int()
    rows = T * E + T
    h, hs = torch.zeros((rows, I), dtype=torch.uint8, device=DEV), torch.zeros((rows, 1), device=DEV)
    y, err = torch.zeros((rows, H), device=DEV), _err()
    ft.ft_expert_ffn_fp8(x, H, xs, T, H, I, E, weights, E + 1, list(range(E)) + [-1], list(range(E + 1)), offsets, perm,
                         h, hs, y, err)
    assert err.item() == 0
    for e in (0, E - 1, E):          # E: the shared expert
        for t in (0, T - 2, T - 1):
            at = e * T + t
            (g, sg), (u, su), (d, sd) = fp8.blob_parts(raw[e], H, I)
            xv, sv = fp8.decode(_bytes(x[t:t + 1])), _np(xs[t:t + 1])
            a, la = fp8.product(xv, sv, g, sg)
            b, lb = fp8.product(xv, sv, u, su)
            ref = fp8.silu(a) * b
            bound = (1.1 * fp8.product_bound(la, H) * (np.abs(b) + fp8.product_bound(lb, H)) +
                     np.abs(fp8.silu(a)) * fp8.product_bound(lb, H) + 8 * U32 * np.abs(ref))
            check_codes(_bytes(h[at:at + 1]), _np(hs[at:at + 1]), ref, 0.0, bound.max(1, keepdims=True))
            yr, ly = fp8.product(fp8.decode(_bytes(h[at:at + 1])), _np(hs[at:at + 1]), d, sd)
            assert (np.abs(_np(y[at:at + 1]) - yr) <= fp8.product_bound(ly, I)).all()


def test_ffn_streams_at_once():
    """Calls on several streams, each with its own rows, give the bits of a call alone."""
    f = Ffn(20, 512, 256, 12, 3, True, seed=41)
    f.run()
    torch.cuda.synchronize()
    want = f.y.clone()
    f.check()
    outs, streams = [], [torch.cuda.Stream() for _ in range(4)]
    for i in range(8):
        f.buffers()
        outs.append((f.h, f.hs, f.y, f.err))
    torch.cuda.synchronize()
    for i, (f.h, f.hs, f.y, f.err) in enumerate(outs):
        f.run(streams[i % 4])
    torch.cuda.synchronize()
    assert all(torch.equal(o[2], want) and o[3].item() == 0 for o in outs)


def test_other_devices_and_host_outputs_are_refused():
    x = torch.randn((2, 128), device=DEV)
    q, s = torch.zeros((2, 128), dtype=torch.uint8), torch.zeros((2, 1), device=DEV)
    with pytest.raises(ft.FtError) as e:
        ft.ft_quantize_fp8(x, 128, False, 2, 128, q, 128, s)
    assert e.value.code == ft.FT_ERR_INVALID and "current device" in str(e.value)
