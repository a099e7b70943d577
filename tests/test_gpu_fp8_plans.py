"""Every form of the fp8 products against the float64 oracle, whatever the estimate of time would
pick: the 128 x 256 tiles and each streaming kernel (tokens per CTA x parts of K x CTAs per
expert), forced by the ft_debug_* entries, at odd sizes, partial blocks, NaN codes, lists with
empty and unlisted experts, on several streams and captured; and the public calls at sizes
whose plan is asserted.

Tolerances are those of fp8.product_bound: parts of K added over the cluster take the place of
as many steps of the chain over blocks, so the roundings counted there are not exceeded."""
import numpy as np
import pytest
import torch

import moe_expert_offload_top_b200 as ft
from oracle import fp8
from test_gpu_fp8 import DEV, EPS, UBF, Ffn, _bytes, _dt, _err, _norm_bound, _np, _operand, _scales, check_codes

pytestmark = pytest.mark.gpu

TILES = (0, 1, 1)
PRODUCT = [TILES] + [(nt, split, chunks) for nt in (16, 32, 128) for split, chunks in ((1, 3), (2, 1), (4, 2), (8, 1))]
GATE_UP = [TILES] + [(nt, split, chunks) for nt in (16, 32, 64) for split, chunks in ((1, 2), (2, 1), (4, 3), (8, 1))]


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _gemm_case(M, N, K, seed, pad=0):
    gen = torch.Generator().manual_seed(seed)
    ld = -(-K // 16) * 16 + pad
    a, w = _operand(M, K, ld, gen), _operand(N, K, ld, gen)
    sa, sw = _scales((M, fp8.blocks(K)), gen), _scales((fp8.blocks(N), fp8.blocks(K)), gen)
    return ld, a, w, sa, sw


def _check_product(out, a, sa, w, sw, K, bf16):
    ref, l1 = fp8.product(fp8.decode(_bytes(a)[:, :K]), _np(sa), fp8.decode(_bytes(w)[:, :K]), _np(sw))
    tol = fp8.product_bound(l1, K) + (UBF * np.abs(ref) * (1 + UBF) if bf16 else 0.0)
    off = np.abs(_np(out) - ref)
    assert (off <= tol).all(), np.max(off / tol)


# K = 1133: eight whole blocks of K and a ninth that ends inside; 1250: more than one chunk of factors
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("M,N,K,ldo", [
    (1, 130, 1133, 131),        # one row, rows of out that no wide store fits
    (150, 300, 1250, 304),      # 16-byte rows of out, a ragged last column
    (150, 300, 1250, 320),      # 32-byte rows
    (261, 515, 1024, 517),      # several tiles, odd rows
    (40, 264, 2000, 264)])
@pytest.mark.parametrize("plan", PRODUCT)
def test_gemm_by_plan(plan, M, N, K, ldo, bf16):
    ld, a, w, sa, sw = _gemm_case(M, N, K, M + N + K, pad=16)
    out, err = torch.full((M + 1, ldo), 77.0, dtype=_dt(bf16), device=DEV), _err()
    ft.ft_debug_gemm_fp8(a, ld, sa, w, ld, sw, M, N, K, bf16, out, ldo, err, plan)
    assert err.item() == 0
    _check_product(out[:M, :N], a, sa, w, sw, K, bf16)
    assert (out[M] == 77).all() and (out[:, N:] == 77).all()


@pytest.mark.parametrize("plan", [p for p in PRODUCT if p[1] <= 2])
@pytest.mark.parametrize("M,N,K", [(1, 1, 129), (3, 17, 200), (129, 257, 255)])
def test_gemm_by_plan_two_blocks(plan, M, N, K):
    """As few blocks of K as the plan allows: each part has one at most."""
    ld, a, w, sa, sw = _gemm_case(M, N, K, 3)
    out, err = torch.zeros((M, N), device=DEV), _err()
    ft.ft_debug_gemm_fp8(a, ld, sa, w, ld, sw, M, N, K, False, out, N, err, plan)
    assert err.item() == 0
    _check_product(out, a, sa, w, sw, K, False)


@pytest.mark.parametrize("plan", PRODUCT)
def test_gemm_by_plan_nan_codes_and_zero_rows(plan):
    """A NaN code reaches its row or column and nothing else; rows of zeros and zero scales give zeros."""
    M, N, K = 140, 300, 1100
    ld, a, w, sa, sw = _gemm_case(M, N, K, 1)
    a[5] = 0
    a[130, 17] = 0x7F
    w[299, 1080] = 0xFF
    sa[6] = 0.0
    out, err = torch.zeros((M, N), device=DEV), _err()
    ft.ft_debug_gemm_fp8(a, ld, sa, w, ld, sw, M, N, K, False, out, N, err, plan)
    assert err.item() == 0
    want = torch.zeros((M, N), dtype=torch.bool, device=DEV)
    want[:, 299] = True
    want[130] = True
    assert torch.equal(torch.isnan(out), want)
    assert (out[5, :299] == 0).all() and (out[6, :299] == 0).all()


@pytest.mark.parametrize("plan", [TILES, (16, 1, 2), (32, 4, 1), (128, 2, 1), (128, 8, 1)])
def test_gemm_by_plan_streams_repeats_and_graph(plan):
    """The same call on four streams at once, again, and captured gives the same bits."""
    M, N, K = 260, 1000, 2048
    ld, a, w, sa, sw = _gemm_case(M, N, K, 2)
    first, err = torch.zeros((M, N), device=DEV), _err()

    def call(out, stream=None):
        ft.ft_debug_gemm_fp8(a, ld, sa, w, ld, sw, M, N, K, False, out, N, err, plan, -1, stream)
    call(first)
    torch.cuda.synchronize()
    outs = [torch.zeros((M, N), device=DEV) for _ in range(8)]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        call(o, streams[i % 4])
    torch.cuda.synchronize()
    assert err.item() == 0 and all(torch.equal(o, first) for o in outs)
    graph, out = torch.cuda.CUDAGraph(), outs[0]
    with torch.cuda.graph(graph, stream=streams[0]):
        call(out, streams[0])
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    assert err.item() == 0


# ------------------------------------------------- expert FFN, by plan --

class PlannedFfn(Ffn):
    plans = (TILES, TILES)

    def run(self, stream=None, experts=None, slots=None):
        ft.ft_debug_expert_ffn_fp8(self.x, self.ldx, self.xs, self.T, self.H, self.I, self.k, self.weights, self.n_slots,
                                   self.experts if experts is None else experts, self.slots if slots is None else slots,
                                   self.offsets, self.perm, self.h, self.hs, self.y, self.err, *self.plans, -1, stream)


# every gate/up form, each with another form of the down product
PAIRS = [(g, PRODUCT[(5 * i + 1) % len(PRODUCT)]) for i, g in enumerate(GATE_UP)] + [(TILES, TILES), ((64, 2, 1), TILES)]


@pytest.mark.parametrize("gate_up,down", PAIRS)
@pytest.mark.parametrize("T,H,I,E,k,shared,empty,skew", [
    (1, 1040, 1040, 4, 2, True, (), 0.0),            # H and I end inside their last block; one token
    (75, 912, 928, 5, 2, True, (0, 4), 1.0),       # experts without tokens first and last in the list
    (140, 1024, 1024, 3, 1, False, (), 2.0)])
def test_expert_ffn_by_plan(gate_up, down, T, H, I, E, k, shared, empty, skew):
    f = PlannedFfn(T, H, I, E, k, shared, seed=T + H, empty=empty, skew=skew, pad=16 * (T % 2))
    f.plans = gate_up, down
    f.run()
    f.check()


@pytest.mark.parametrize("plan", [TILES, (16, 2, 1), (32, 1, 1), (64, 1, 2)])
def test_expert_ffn_by_plan_unlisted_experts(plan):
    f = PlannedFfn(90, 272, 400, 6, 3, True, seed=5)
    f.plans = plan, (128 if plan[0] == 64 else plan[0], *plan[1:])
    drop = {1, 4, -1}
    keep = [(e, s) for e, s in zip(f.experts, f.slots) if e not in drop]
    f.run(experts=[e for e, _ in keep], slots=[s for _, s in keep])
    f.check(skip=drop)


@pytest.mark.parametrize("plan", [TILES, (64, 1, 1), (32, 2, 2)])
def test_expert_ffn_by_plan_streams_and_graph(plan):
    f = PlannedFfn(130, 400, 272, 5, 2, True, seed=41)
    f.plans = plan, (128 if plan[0] == 64 else plan[0], *plan[1:])
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
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        f.run(streams[0])
    f.y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(f.y, want) and f.err.item() == 0


# ---------------------------------------------- public calls, plan asserted --

@pytest.mark.parametrize("M,N,K,bf16,nt,split", [
    (700, 8200, 1133, True, 0, 1),      # tiles, a ragged K
    (1030, 8101, 1250, False, 0, 1),     # tiles, odd rows of out
    (200, 768, 2048, True, 32, 2), (160, 520, 1100, False, 32, 4), (300, 2048, 2048, True, 128, 2),
    (300, 1030, 4000, False, 128, 4), (300, 512, 7100, True, 128, 8), (2, 7168, 2000, False, 16, 2)])
def test_gemm_at_sizes_of_each_plan(M, N, K, bf16, nt, split):
    aligned = N * (2 if bf16 else 4) % 16 == 0
    assert ft.ft_debug_fp8_plan(1, M, 1, N, K, _sms(), aligned)[:2] == (nt, split)
    ld, a, w, sa, sw = _gemm_case(M, N, K, N)
    out, err = torch.zeros((M, N), dtype=_dt(bf16), device=DEV), _err()
    ft.ft_gemm_fp8(a, ld, sa, w, ld, sw, M, N, K, bf16, out, N, err)
    assert err.item() == 0
    rows = [0, 1, M // 2, M - 2, M - 1]      # the whole is compared with the tiles' own check above
    _check_product(out[rows], a[rows], sa[rows], w, sw, K, bf16)
    forced = torch.zeros_like(out)
    ft.ft_debug_gemm_fp8(a, ld, sa, w, ld, sw, M, N, K, bf16, forced, N, err,
                         ft.ft_debug_fp8_plan(1, M, 1, N, K, _sms(), aligned))
    assert torch.equal(forced, out)


@pytest.mark.parametrize("T,H,I,E,k,nt", [(900, 528, 400, 3, 2, 0), (1000, 1040, 272, 4, 2, 0)])
def test_expert_ffn_at_sizes_of_the_tiles(T, H, I, E, k, nt):
    even = T * k / E
    rows = max(min(T, int(np.ceil(even + 3 * np.sqrt(even)))), T)
    assert ft.ft_debug_fp8_plan(0, rows, E + 1, I, H, _sms())[0] == nt
    f = Ffn(T, H, I, E, k, True, seed=T, empty=(1,), skew=0.5)
    f.run()
    f.check()


# -------------------------------------------------------------- norm, rows --

@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,H", [(297, 4112), (300, 7168), (400, 9008), (299, 16384)])
def test_rmsnorm_many_wide_aligned_rows(T, H, bf16):
    """Two chunks per thread: more than 296 aligned rows wider than 4096."""
    g = torch.Generator().manual_seed(H)
    x, res = ((torch.randn((T, H + 16), generator=g) * s).to(_dt(bf16)).to(DEV) for s in (2, 5))
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(_dt(bf16)).to(DEV)
    y = torch.full((T + 1, H), 77.0, dtype=_dt(bf16), device=DEV)
    r = torch.full((T + 1, H + 16), 77.0, dtype=_dt(bf16), device=DEV)
    q = torch.full((T + 1, H + 16), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((T + 1, fp8.blocks(H)), -1.0, device=DEV)
    ft.ft_rmsnorm_fp8(x, H + 16, res, H + 16, w, bf16, T, H, EPS, r, y, q, H + 16, s)
    want = (x[:, :H].float() + res[:, :H].float()).to(_dt(bf16))
    assert torch.equal(r[:T, :H], want) and (r[T] == 77).all() and (r[:, H:] == 77).all()
    assert (y[T] == 77).all() and (q[T] == 0x55).all() and (q[:, H:] == 0x55).all() and (s[T] == -1).all()
    ref = fp8.rmsnorm(_np(want), _np(w), EPS)
    rel = _norm_bound(H)
    assert (np.abs(_np(y[:T]) - ref) <= (rel + (UBF if bf16 else 0.0)) * np.abs(ref) * (1 + UBF) + 1e-38).all()
    check_codes(_bytes(q[:T, :H]), _np(s[:T]), ref, rel)


@pytest.mark.parametrize("H", [512, 515])
def test_norm_of_rows_whose_squares_leave_f32(H):
    """As the header says: zeros where the sum of squares overflows, infinities and NaN where it vanishes and
    eps is 0; the rows beside them are those of a call without such rows."""
    x = torch.randn((6, H), device=DEV)
    x[1], x[3], x[4] = 1e25, 1e-30, 0.0
    x[3, 5] = 0.0
    w = torch.full((H,), 0.5, device=DEV)
    n = fp8.blocks(H)
    y, q, s = torch.zeros_like(x), torch.zeros((6, H), dtype=torch.uint8, device=DEV), torch.zeros((6, n), device=DEV)
    ft.ft_rmsnorm_fp8(x, H, None, 0, w, False, 6, H, 0.0, None, y, q, H, s)
    assert (y[1] == 0).all() and (s[1] == fp8.TINY).all() and (q[1] == 0).all()
    zero = x[3] == 0
    assert torch.isnan(y[3][zero]).all() and torch.isinf(y[3][~zero]).all() and torch.isnan(y[4]).all()
    keep = [0, 2, 5]
    y2, q2, s2 = torch.zeros((3, H), device=DEV), torch.zeros((3, H), dtype=torch.uint8, device=DEV), torch.zeros((3, n), device=DEV)
    ft.ft_rmsnorm_fp8(x[keep].contiguous(), H, None, 0, w, False, 3, H, 0.0, None, y2, q2, H, s2)
    assert torch.equal(y[keep], y2) and torch.equal(q[keep], q2) and torch.equal(s[keep], s2)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,H", [(32, 7168), (300, 4096), (33, 2051), (5, 200)])
def test_quantised_rows_are_the_formula_bit_for_bit(T, H, bf16):
    """s = max(max |y| / 448, 2^-126) rounded once, q = e4m3(y * (1 / s)) with the inverse and the product
    rounded once each: three IEEE operations, so the bits are known."""
    g = torch.Generator().manual_seed(T + H)
    x = (torch.randn((T, H), generator=g) * torch.exp2(torch.randint(-20, 20, (T, 1), generator=g).float())).to(_dt(bf16))
    pad = torch.zeros((T, fp8.blocks(H) * 128))
    pad[:, :H] = x.float()
    b = pad.numpy().reshape(T, -1, 128)
    scale = np.maximum(np.abs(b).max(2) / np.float32(448), np.float32(2.0 ** -126))
    assert scale.dtype == np.float32
    v = (b * (np.float32(1) / scale)[..., None]).reshape(T, -1)[:, :H]
    assert v.dtype == np.float32
    q, s = torch.zeros((T, H), dtype=torch.uint8, device=DEV), torch.zeros((T, fp8.blocks(H)), device=DEV)
    ft.ft_quantize_fp8(x.to(DEV), H, bf16, T, H, q, H, s)
    assert np.array_equal(s.cpu().numpy(), scale)
    assert np.array_equal(fp8.decode(_bytes(q)), fp8.round_e4m3(v))


# ------------------------------------- a device wait that runs out (1 ms) --

@pytest.mark.parametrize("at", [0, 1, 2])
@pytest.mark.parametrize("nt,split", [(16, 1), (16, 8), (32, 4), (128, 2)])
def test_stream_product_gives_up(nt, split, at):
    """A wait of every CTA's chunk `at` gives up: the chunks before it are right, it and those behind it
    are left unwritten, the call returns, and the next call is right."""
    M, N, K = 5 * nt - 3, 300, 2048
    ld, a, w, sa, sw = _gemm_case(M, N, K, nt)
    want, err = torch.zeros((M, N), device=DEV), _err()
    ft.ft_debug_gemm_fp8(a, ld, sa, w, ld, sw, M, N, K, False, want, N, err, (nt, split, 1))
    assert err.item() == 0
    out = torch.full((M, N), 77.0, device=DEV)
    ft.ft_debug_gemm_fp8(a, ld, sa, w, ld, sw, M, N, K, False, out, N, err, (nt, split, 1), at)
    assert err.item() == 129
    assert torch.equal(out[:nt * at], want[:nt * at]) and (out[nt * at:] == 77).all()
    err.zero_()
    ft.ft_debug_gemm_fp8(a, ld, sa, w, ld, sw, M, N, K, False, out, N, err, (nt, split, 1))
    assert err.item() == 0 and torch.equal(out, want)


@pytest.mark.parametrize("at", [0, 1])
def test_tile_product_gives_up(at):
    """The same for the tiles: a CTA's first tiles are right, the one that gave up and later ones unwritten."""
    ctas, M, N, K = _sms(), 2560, 4096, 1280      # 320 tiles of 128 x 256, column by column of tiles
    ld, a, w, sa, sw = _gemm_case(M, N, K, 6)
    want, err = torch.zeros((M, N), device=DEV), _err()
    ft.ft_debug_gemm_fp8(a, ld, sa, w, ld, sw, M, N, K, False, want, N, err, TILES)
    assert err.item() == 0
    out = torch.full((M, N), 77.0, device=DEV)
    ft.ft_debug_gemm_fp8(a, ld, sa, w, ld, sw, M, N, K, False, out, N, err, TILES, at)
    assert err.item() == 121
    for t in range(M // 128 * (N // 256)):
        r, c = slice(t % 20 * 128, t % 20 * 128 + 128), slice(t // 20 * 256, t // 20 * 256 + 256)
        assert torch.equal(out[r, c], want[r, c]) if t < ctas * at else (out[r, c] == 77).all()
    err.zero_()
    ft.ft_debug_gemm_fp8(a, ld, sa, w, ld, sw, M, N, K, False, out, N, err, TILES)
    assert err.item() == 0 and torch.equal(out, want)


@pytest.mark.parametrize("gate_up,down", [((16, 2, 1), (16, 1, 1)), ((64, 1, 1), (128, 1, 1)), (TILES, TILES)])
def test_expert_ffn_gives_up(gate_up, down):
    f = PlannedFfn(150, 400, 272, 3, 2, True, seed=8)
    ft.ft_debug_expert_ffn_fp8(f.x, f.ldx, f.xs, f.T, f.H, f.I, f.k, f.weights, f.n_slots, f.experts, f.slots, f.offsets,
                               f.perm, f.h, f.hs, f.y, f.err, gate_up, down, 0)
    assert f.err.item() == (129 if gate_up[0] else 121)
    assert (f.h == 0x55).all() and (f.hs == -1).all()
    f.buffers()
    f.plans = gate_up, down
    f.run()
    f.check()


# ------------------------------------------------- SiLU, NaN and infinities --

FORMS = [TILES, (16, 1, 1), (32, 1, 2), (64, 1, 1)]


def _planned(T, H, I, E, k, shared, seed, form):
    f = PlannedFfn(T, H, I, E, k, shared, seed=seed)
    f.plans = form, (128 if form[0] == 64 else form[0], *form[1:])
    return f


@pytest.mark.parametrize("form", FORMS)
def test_silu_over_its_whole_range(form):
    """One column of x is 1, so that a = x_scale * gate code and u = x_scale * up code * its scale: from 1e-30 to
    1e18, where exp(-a) is inf, around the smallest quotients, and far positive.  a is rounded
    twice (the scales' product, the product with the code), u twice, silu by (9 + 2.4 |a|), the
    product once, in units of 2^-24; a's error reaches silu times 1 + |a|.  Below -87.3 silu may be 0."""
    H, I = 144, 144
    scales = np.float32([1e-30, 1e-3, 0.3, 1.0, 3.7, 9.1, 20.0, 43.0, 58.3, 64.0, 80.0, 86.9, 87.4, 88.0, 88.5, 88.8, 100.0,
                         1e4, 1e12, 1e18])
    T = len(scales)
    f = _planned(T, H, I, 1, 1, False, 3, form)
    rng = np.random.default_rng(5)
    x = np.zeros((T, H))
    x[:, 7] = 1.0
    gate, up = np.zeros((I, H)), np.zeros((I, H))
    gate[:, 7] = np.resize([1.0, -1.0, 0.5, -0.5, -0.9375, 0.0625, -2.0 ** -9, -1.125], I)
    gate[128:, 7] = -1.0     # a block whose scale is that of its negative a
    up[:, 7] = fp8.round_e4m3(rng.standard_normal(I))
    raw = np.frombuffer(b"".join(fp8.encode(m).tobytes() for m in (gate, up, np.zeros((H, I)))), dtype=np.uint8)
    sg, su = np.float32([[1.0, 1.0], [1.0, 1.0]]), np.float32([[0.3, 1.0], [7.0, 1.0]])
    raw = np.concatenate([raw, np.frombuffer(sg.tobytes() + su.tobytes() + sg.tobytes(), dtype=np.uint8)])
    f.weights[f.slots[0], :len(raw)] = torch.from_numpy(raw).to(DEV)
    f.x[:, :H] = torch.from_numpy(fp8.encode(x)).to(DEV)
    f.xs[:] = torch.from_numpy(scales[:, None]).to(DEV)
    f.run()
    assert f.err.item() == 0
    a = scales[:, None].astype(np.float64) * gate[None, :, 7]
    u = scales[:, None].astype(np.float64) * np.repeat(su[:, 0].astype(np.float64), 128)[:I] * up[None, :, 7]
    ref = fp8.silu(a) * u
    U = 2.0 ** -24
    bound = np.abs(ref) * U * (2 * (1 + np.abs(a)) + 2 + 9 + 2.4 * np.abs(a) + 1) + np.where(a < -87.3, 1.1e-36 * np.abs(u), 0)
    h, hs = _bytes(f.h), _np(f.hs)
    for t in range(T):      # a row by itself: the bounds differ by 60 orders of magnitude
        worst = np.array([[bound[t, :128].max(), bound[t, 128:].max()]])
        for b, c in ((0, slice(0, 128)), (1, slice(128, I))):
            check_codes(h[t:t + 1, c], hs[t:t + 1, b:b + 1], ref[t:t + 1, c], 0.0, worst[:, b:b + 1])


@pytest.mark.parametrize("form", FORMS)
def test_ffn_keeps_nan_and_infinities_to_their_rows(form):
    T, H, I, E, k = 70, 272, 272, 4, 2
    f = _planned(T, H, I, E, k, True, 17, form)
    f.run()
    torch.cuda.synchronize()
    h0, hs0, y0 = f.h.clone(), f.hs.clone(), f.y.clone()
    f.buffers()
    f.x[3, 200] = 0x7F                       # a NaN code
    f.xs[40, 1] = float("nan")               # a NaN scale
    f.xs[41, 0] = 3e38                       # sums that overflow
    off, perm = _bytes(f.offsets), _bytes(f.perm)
    lo, hi = off[2], off[3]
    n = 3 * H * I                            # expert 2: a NaN in S_up's block of h columns 128 .. 255
    blob = f.weights[f.slots[2]]
    sc = blob[n:n + 4 * 3 * 9].view(torch.float32).view(3, 3, 3)
    sc[1, 1, 0] = float("nan")
    f.run()
    torch.cuda.synchronize()
    assert f.err.item() == 0
    token = np.concatenate([perm // k, np.arange(T)])
    bad_rows = torch.from_numpy(np.isin(token, (3, 40, 41))).to(DEV)
    bad_expert = torch.zeros_like(bad_rows)
    bad_expert[lo:hi] = True
    clean = ~bad_rows & ~bad_expert
    assert torch.equal(f.h[clean], h0[clean]) and torch.equal(f.hs[clean], hs0[clean]) and torch.equal(f.y[clean], y0[clean])
    nan_rows = torch.from_numpy(np.isin(token, (3, 40))).to(DEV)
    assert torch.isnan(f.hs[nan_rows]).all() and torch.isnan(f.y[nan_rows]).all()
    assert (~torch.isfinite(f.hs[bad_rows])).all(dim=1).all() and (~torch.isfinite(f.y[bad_rows])).all()
    rest = bad_expert & ~bad_rows
    assert rest.any() and torch.isnan(f.hs[rest][:, 1]).all() and torch.isnan(f.y[rest]).all()
    assert torch.equal(f.hs[rest][:, [0, 2]], hs0[rest][:, [0, 2]])


# --------------------------- calls that the header allows, at odd addresses and lists --

@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("plan", [TILES, (16, 2, 1), (128, 1, 2)])
@pytest.mark.parametrize("off", [1, 2, 4, 8])
def test_gemm_into_rows_at_any_element(plan, bf16, off):
    """out begins `off` elements behind a wide boundary while its rows are 32 bytes apart in step."""
    M, N, K = 140, 272, 384
    ld, a, w, sa, sw = _gemm_case(M, N, K, off)
    flat, err = torch.full((M * N + 16,), 77.0, dtype=_dt(bf16), device=DEV), _err()
    out = flat[off:off + M * N].view(M, N)
    ft.ft_debug_gemm_fp8(a, ld, sa, w, ld, sw, M, N, K, bf16, out, N, err, plan)
    assert err.item() == 0
    _check_product(out, a, sa, w, sw, K, bf16)
    assert (flat[:off] == 77).all() and (flat[off + M * N:] == 77).all()


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("odd", ["x", "residual", "weight", "residual_out", "y", "q", "scales"])
def test_norm_with_one_buffer_at_an_odd_element(odd, bf16):
    T, H = 21, 640
    g = torch.Generator().manual_seed(4)

    def place(name, t):
        off = 1 if name == odd else 0
        flat = torch.zeros(t.numel() + 64, dtype=t.dtype, device=DEV)
        view = flat[off:off + t.numel()].view(t.shape)
        view.copy_(t)
        return view
    x, res = (place(n, torch.randn((T, H), generator=g).to(_dt(bf16))) for n in ("x", "residual"))
    w = place("weight", (1 + 0.3 * torch.randn(H, generator=g)).to(_dt(bf16)))
    r, y = (place(n, torch.zeros((T, H), dtype=_dt(bf16))) for n in ("residual_out", "y"))
    q, s = place("q", torch.zeros((T, H), dtype=torch.uint8)), place("scales", torch.zeros((T, 5)))
    ft.ft_rmsnorm_fp8(x, H, res, H, w, bf16, T, H, EPS, r, y, q, H, s)
    want = (x.float() + res.float()).to(_dt(bf16))
    assert torch.equal(r, want)
    ref = fp8.rmsnorm(_np(want), _np(w), EPS)
    rel = _norm_bound(H)
    assert (np.abs(_np(y) - ref) <= (rel + (UBF if bf16 else 0.0)) * np.abs(ref) * (1 + UBF) + 1e-38).all()
    check_codes(_bytes(q), _np(s), ref, rel)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_expert_ffn_of_the_shared_expert_alone(T):
    f = Ffn(T, 272, 400, 4, 2, True, seed=6)
    f.run(experts=[-1], slots=[f.slots[f.experts.index(-1)]])
    f.check(skip=range(4))


@pytest.mark.parametrize("T", [1, 60])
def test_expert_ffn_with_the_list_turned_round(T):
    """The list's order does not matter: the shared expert first, the others from the last."""
    f = Ffn(T, 256, 144, 16, 3, True, seed=7, empty=(2,))
    f.run(experts=f.experts[::-1], slots=f.slots[::-1])
    f.check()


@pytest.mark.parametrize("T,forced", [(1, None), (9, None), (70, None), (70, TILES)])
def test_expert_ffn_with_every_expert_listed(T, forced):
    """256 routed experts and the shared one, most of them without tokens: what a captured call lists."""
    f = PlannedFfn(T, 144, 80, 256, 6, True, seed=12) if forced else Ffn(T, 144, 80, 256, 6, True, seed=12)
    assert len(f.experts) == 257
    f.run()
    f.check()
