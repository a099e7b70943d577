"""CPU checks of the fp8 operators: the oracle's e4m3 against hand values and torch, the blob
size, and every refusal of the entry points (they come before anything touches a GPU)."""
import numpy as np
import pytest
import torch

import moe_expert_offload_top_b200 as ft
from oracle import fp8

P = 1 << 20        # a 16-byte aligned address that is never read: the calls below are refused


def test_e4m3_hand_values():
    assert [fp8.decode(c) for c in (0x00, 0x01, 0x07, 0x08, 0x38, 0x3C, 0x7E, 0xBC)] == [
        0.0, 2.0 ** -9, 7 * 2.0 ** -9, 2.0 ** -6, 1.0, 1.5, 448.0, -1.5]
    assert np.isnan(fp8.decode(0x7F)) and np.isnan(fp8.decode(0xFF))
    # ties to even, subnormals, saturation
    v = np.array([1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, 460.0, 1e9, -465.0])
    assert fp8.round_e4m3(v).tolist() == [1.0, 1.25, 0.0, 2.0 ** -8, 448.0, 448.0, -448.0]


def test_e4m3_rounding_and_codes_match_torch():
    rng = np.random.default_rng(0)
    v = (rng.standard_normal(20000) * np.exp2(rng.integers(-14, 8, 20000))).clip(-448, 448).astype(np.float32)
    ref = torch.from_numpy(v).to(torch.float8_e4m3fn)
    got = fp8.round_e4m3(v)
    assert np.array_equal(got, ref.double().numpy())
    assert np.array_equal(fp8.decode(fp8.encode(got)), got)


def test_scales_of_zero_and_partial_blocks():
    y = np.zeros((2, 200))
    y[1, 199] = -3.5
    q, s = fp8.quantize_rows(y)
    assert s.tolist() == [[fp8.TINY, fp8.TINY], [fp8.TINY, np.float32(3.5 / 448)]]
    assert q[1, 199] == -448 and np.count_nonzero(q) == 1


@pytest.mark.parametrize("H,I", [(16, 16), (128, 256), (144, 400), (4096, 2048)])
def test_blob_bytes(H, I):
    n = 3 * H * I + 12 * -(-H // 128) * -(-I // 128)
    assert ft.ft_fp8_blob_bytes(H, I) == (n + 15) // 16 * 16
    assert ft.ft_fp8_blob_bytes(H + 1, I) == 0 and ft.ft_fp8_blob_bytes(H, 0) == 0
    if H < 1000:
        z = np.zeros
        assert len(fp8.blob(z((I, H)), z((I, H)), z((H, I)))) == ft.ft_fp8_blob_bytes(H, I)


def _refused(fn, base, change, word):
    args = dict(base, **change)
    with pytest.raises(ft.FtError) as e:
        fn(*args.values())
    assert e.value.code == ft.FT_ERR_INVALID
    assert fn.__name__ in str(e.value) and word in str(e.value), str(e.value)


NORM = dict(x=P, ldx=256, residual=P, ldr=256, weight=P, x_is_bf16=1, T=4, H=256, eps=1e-6, residual_out=P, y=P, q=P,
            ldq=256, scales=P)


@pytest.mark.parametrize("change,word", [
    (dict(T=-1), "size"), (dict(H=0), "size"), (dict(H=32769, ldx=40000, ldr=40000, ldq=40000), "32768"),
    (dict(ldx=255), "stride"), (dict(ldr=255), "stride"), (dict(ldq=255), "stride"), (dict(x=None), "null"),
    (dict(weight=None), "null"), (dict(scales=None), "null"), (dict(q=None, y=None), "null"),
    (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(x=P + 1), "aligned"), (dict(y=P + 1), "aligned"),
    (dict(residual=P + 1), "aligned"), (dict(scales=P + 2), "aligned"),
])
def test_rmsnorm_refusals(change, word):
    _refused(ft.ft_rmsnorm_fp8, NORM, change, word)


QUANT = dict(x=P, ldx=256, x_is_bf16=0, T=4, H=256, q=P, ldq=256, scales=P)


@pytest.mark.parametrize("change,word", [
    (dict(T=-1), "size"), (dict(H=-3), "size"), (dict(ldx=255), "stride"), (dict(ldq=128), "stride"),
    (dict(x=None), "null"), (dict(q=None), "null"), (dict(scales=None), "null"), (dict(x=P + 2), "aligned"),
])
def test_quantize_refusals(change, word):
    _refused(ft.ft_quantize_fp8, QUANT, change, word)


GEMM = dict(a=P, lda=256, a_scales=P, w=P, ldw=256, w_scales=P, M=4, N=64, K=250, out_is_bf16=1, out=P, ldo=64, err=P)


@pytest.mark.parametrize("change,word", [
    (dict(M=-1), "size"), (dict(N=-1), "size"), (dict(K=0), "size"), (dict(lda=240), "stride"),
    (dict(ldw=240), "stride"), (dict(ldo=63), "stride"), (dict(lda=264), "16"), (dict(ldw=264), "16"),
    (dict(a=P + 8), "16-byte"), (dict(w=P + 8), "16-byte"), (dict(a=None), "null"), (dict(w=None), "null"),
    (dict(a_scales=None), "null"), (dict(w_scales=None), "null"), (dict(out=None), "null"), (dict(err=None), "null"),
    (dict(out=P + 1), "aligned"), (dict(a_scales=P + 1), "aligned"),
])
def test_gemm_refusals(change, word):
    _refused(ft.ft_gemm_fp8, GEMM, change, word)


FFN = dict(x=P, ldx=256, x_scales=P, T=4, H=256, I=128, top_k=2, weights=P, n_slots=3, experts=[0, 5, -1],
           slots=[2, 0, 1], offsets=P, perm=P, h=P, h_scales=P, y=P, err=P)


@pytest.mark.parametrize("change,word", [
    (dict(T=-1), "size"), (dict(top_k=0), "size"), (dict(top_k=17), "size"), (dict(n_slots=0), "size"),
    (dict(H=250), "multiples of 16"), (dict(I=8), "multiples of 16"), (dict(ldx=240), "ldx"), (dict(ldx=264), "ldx"),
    (dict(T=2 ** 30), "2^31"), (dict(experts=[0, 256, -1]), "entry"), (dict(experts=[0, -2, -1]), "entry"),
    (dict(slots=[0, 3, 1]), "entry"), (dict(slots=[0, -1, 1]), "entry"), (dict(experts=[5, 5, -1]), "twice"),
    (dict(experts=[-1, 5, -1]), "twice"), (dict(x=P + 8), "16-byte"), (dict(y=P + 8), "16-byte"),
    (dict(weights=P + 8), "16-byte"), (dict(h=None), "null"), (dict(err=None), "null"), (dict(perm=None), "null"),
    (dict(offsets=P + 2), "aligned"),
])
def test_ffn_refusals(change, word):
    _refused(ft.ft_expert_ffn_fp8, FFN, change, word)


def test_lists_of_different_lengths_are_refused():
    with pytest.raises(ValueError):
        ft.ft_expert_ffn_fp8(*dict(FFN, slots=[0, 1]).values())


def test_empty_calls_do_nothing():
    ft.ft_rmsnorm_fp8(*dict(NORM, T=0).values())
    ft.ft_quantize_fp8(*dict(QUANT, T=0).values())
    ft.ft_gemm_fp8(*dict(GEMM, M=0).values())
    ft.ft_gemm_fp8(*dict(GEMM, N=0).values())
    ft.ft_expert_ffn_fp8(*dict(FFN, T=0).values())
    ft.ft_expert_ffn_fp8(*dict(FFN, experts=[], slots=[]).values())
