"""How the fp8 products choose their form, and the refusals of forced plans (no GPU)."""
import pytest
import torch

import moe_expert_offload_top_b200 as ft
from test_fp8_cpu import FFN, GEMM, NORM, P, QUANT, _refused


@pytest.mark.parametrize("mode,rows,groups,N,K,want", [
    (1, 1, 1, 4096, 4096, (16, 4)), (1, 32, 1, 7168, 2048, (32, 2)), (1, 300, 1, 2048, 2048, (128, 2)),
    (1, 8192, 1, 7168, 4096, (0, 1)), (0, 1, 7, 2048, 4096, (16, 1)), (0, 4096, 1, 128, 1024, (64, 2)),
    (0, 4096, 64, 2048, 4096, (0, 1))])
def test_plan_of_ordinary_sizes(mode, rows, groups, N, K, want):
    nt, split, chunks = ft.ft_debug_fp8_plan(mode, rows, groups, N, K)
    assert (nt, split) == want
    assert chunks == (1 if nt == 0 else -(-rows // nt))


@pytest.mark.parametrize("mode", [0, 1])
def test_every_plan_is_one_that_the_kernels_take(mode):
    for rows in (1, 3, 16, 17, 33, 65, 129, 300, 1000, 5000, 70000):
        for N in (1, 16, 129, 500, 2048, 8192):
            for K in (1, 16, 129, 300, 1000, 4096):
                nt, split, chunks = ft.ft_debug_fp8_plan(mode, rows, 5, N, K)
                assert nt in ((0, 16, 32, 64) if mode == 0 else (0, 16, 32, 128))
                assert split in (1, 2, 4, 8) and split <= -(-K // 128) and 1 <= chunks <= 64
                assert nt == 0 or nt * chunks >= rows


@pytest.mark.parametrize("args", [(2, 1, 1, 1, 1), (0, -1, 1, 1, 1), (0, 1, 0, 1, 1), (0, 1, 1, 0, 1), (0, 1, 1, 1, 0),
                                  (0, 1, 1, 1, 1, 0), (1, 1, 1, 2 ** 31 - 1, 1)])
def test_plan_refusals(args):
    with pytest.raises(ft.FtError) as e:
        ft.ft_debug_fp8_plan(*args)
    assert "ft_debug_fp8_plan" in str(e.value)


@pytest.mark.parametrize("plan", [(64, 1, 1), (8, 1, 1), (-16, 1, 1), (16, 0, 1), (16, 3, 1), (16, 4, 1), (16, 16, 1),
                                  (16, 1, 0), (16, 1, 65)])
def test_forced_plans_are_checked(plan):
    _refused(ft.ft_debug_gemm_fp8, dict(GEMM, plan=plan), {}, "plan")        # K = 250: two blocks
    _refused(ft.ft_debug_expert_ffn_fp8, dict(FFN, gate_up=(0, 1, 1), down=plan), {}, "plan")
    gate_up = (128, *plan[1:]) if plan[0] == 64 else plan
    _refused(ft.ft_debug_expert_ffn_fp8, dict(FFN, gate_up=gate_up, down=(0, 1, 1)), {}, "plan")


@pytest.mark.parametrize("change,word", [(dict(lda=240), "stride"), (dict(a=None), "null"), (dict(out=7), "aligned")])
def test_forced_calls_check_their_arguments(change, word):
    _refused(ft.ft_debug_gemm_fp8, dict(GEMM, plan=(0, 1, 1)), change, word)


def test_forced_empty_calls_do_nothing():
    ft.ft_debug_gemm_fp8(*dict(GEMM, M=0, plan=(0, 1, 1)).values())
    ft.ft_debug_expert_ffn_fp8(*dict(FFN, T=0, gate_up=(0, 1, 1), down=(0, 1, 1)).values())


@pytest.mark.parametrize("fail_at", [-2, (1 << 20) + 1])
def test_failing_chunk_is_checked(fail_at):
    _refused(ft.ft_debug_gemm_fp8, dict(GEMM, plan=(0, 1, 1), fail_at=fail_at), {}, "plan")
    _refused(ft.ft_debug_expert_ffn_fp8, dict(FFN, gate_up=(0, 1, 1), down=(0, 1, 1), fail_at=fail_at), {}, "plan")


TOP = 2 ** 31 - 2 ** 16


@pytest.mark.parametrize("change", [dict(M=TOP + 1), dict(M=2 ** 31 - 1), dict(N=TOP + 1, ldo=2 ** 31),
                                    dict(N=2 ** 31 - 1, ldo=2 ** 31), dict(K=TOP + 1, lda=2 ** 31, ldw=2 ** 31),
                                    dict(K=2 ** 31 - 1, lda=2 ** 31, ldw=2 ** 31)])
def test_products_whose_tiles_would_pass_32_bits_are_refused(change):
    _refused(ft.ft_gemm_fp8, GEMM, change, "2^31 - 2^16")


def test_the_largest_product_sizes_are_not_refused_for_their_size():
    _refused(ft.ft_gemm_fp8, GEMM, dict(M=TOP, N=TOP, ldo=TOP, K=TOP, lda=2 ** 31, ldw=2 ** 31, a=None), "null")


@pytest.mark.parametrize("change", [
    dict(T=(2 ** 31 - 1) // 3), dict(T=(2 ** 31 - 2 ** 14) // 3), dict(T=TOP // 3 + 1), dict(T=TOP // 17 + 1, top_k=16),
    dict(H=2 ** 31 - 16, ldx=2 ** 31), dict(I=2 ** 31 - 16)])
def test_expert_lists_whose_rows_would_pass_32_bits_are_refused(change):
    """The copy of the pairs' rows steps past the last row by up to 8192: 32 bits have to hold that."""
    _refused(ft.ft_expert_ffn_fp8, FFN, change, "2^31 - 2^16")


def test_the_most_pairs_are_not_refused_for_their_number():
    _refused(ft.ft_expert_ffn_fp8, FFN, dict(T=TOP // 3, h=None), "null")


def test_norm_over_x_in_rows_of_another_stride_is_refused():
    base = dict(NORM, residual=P + (1 << 16))     # residual_out is x
    _refused(ft.ft_rmsnorm_fp8, base, dict(ldx=512), "stride")
    _refused(ft.ft_rmsnorm_fp8, base, dict(ldr=272, residual=None), "stride")
    _refused(ft.ft_rmsnorm_fp8, base, dict(ldx=512, T=1, scales=None), "null")     # one row: any strides
    _refused(ft.ft_rmsnorm_fp8, base, dict(scales=None), "null")


CALLS = [(ft.ft_rmsnorm_fp8, NORM, {}), (ft.ft_quantize_fp8, QUANT, {}), (ft.ft_gemm_fp8, GEMM, {}),
         (ft.ft_expert_ffn_fp8, FFN, {}), (ft.ft_debug_gemm_fp8, GEMM, dict(plan=(0, 1, 1))),
         (ft.ft_debug_expert_ffn_fp8, FFN, dict(gate_up=(0, 1, 1), down=(0, 1, 1)))]


@pytest.mark.parametrize("fn,base,more,name", [(f, b, m, k) for f, b, m in CALLS for k, v in b.items() if v is P])
def test_host_memory_is_refused(fn, base, more, name):
    """A kernel that read it would fault the GPU."""
    host = torch.zeros(1 << 12, dtype=torch.uint8)
    for value in (host, host.numpy()):
        _refused(fn, dict(base, **more), {name: value}, "current device")


class Elsewhere:
    """A tensor of some device, as the binding sees one."""

    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device

    def data_ptr(self):
        return P


def test_tensors_of_two_devices_are_refused():
    for name in ("a", "w_scales", "err"):
        tensors = {k: Elsewhere(1 if k == name else 0) for k, v in GEMM.items() if v is P}
        _refused(ft.ft_gemm_fp8, GEMM, tensors, "current device")
