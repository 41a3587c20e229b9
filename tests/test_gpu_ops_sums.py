"""How the operators of include/dg_ops.h add up: the order of a token's
experts, and sums held in 32 bits."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg
from tests import ops_ref as ref
from tests.gpu_util import to_dev
from tests.test_gpu_ops import MOE_ORDER, host, moe_case, run_moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["fp32", "e8m0"])
@pytest.mark.parametrize("T", [1, 3, 40])
def test_moe_one_expert_listed_several_times_is_added_in_the_order_of_the_list(T, kind):
    """2^30 o, -2^30 o and o, one after the other, leave o; in any other order
    most of o's bits are lost."""
    c = moe_case(41, T, 3, 5, 256, 256, kind)
    c["ids"][:] = 2
    one = dict(c, weights=np.tile(np.array([0, 0, 1], np.float32), (T, 1)))
    c["weights"] = np.tile(np.array([2.0 ** 30, -2.0 ** 30, 1], np.float32), (T, 1))
    want = host(run_moe(one, kind))
    assert np.abs(want).max() > 0.1
    d = [to_dev(c[n]) for n in MOE_ORDER]
    call = dg.dg_moe_mlp_fp8 if kind == "fp32" else dg.dg_moe_mlp_fp8_e8m0
    first = call(*d)
    assert (host(first) == want).all()
    for _ in range(8):
        assert torch.equal(call(*d), first)


@pytest.mark.parametrize("kind", ["fp32", "e8m0"])
@pytest.mark.parametrize("T", [1, 3, 12, 40])
def test_moe_bits_repeat_with_experts_repeated_in_a_row(T, kind):
    c = moe_case(42, T, 3, 3, 384, 256, kind)
    c["ids"] = np.tile(np.array([1, 0, 1], np.int32), (T, 1))
    d = [to_dev(c[n]) for n in MOE_ORDER]
    call = dg.dg_moe_mlp_fp8 if kind == "fp32" else dg.dg_moe_mlp_fp8_e8m0
    first = call(*d)
    for _ in range(8):
        assert torch.equal(call(*d), first)
    want, tol = ref.moe(*[c[n] for n in MOE_ORDER], kind)
    assert (np.abs(host(first) - want) <= tol + ref.BF16 * (np.abs(want) + tol) + 1e-37).all()


@pytest.mark.parametrize("kind", ["fp32", "e8m0"])
@pytest.mark.parametrize("T", [2, 20, 70, 200])
def test_moe_second_product_is_held_in_32_bits(T, kind):
    """Every hidden value is the same, so column n of the second product is its
    code times w2's row n: two products of 448 * 448 that cancel, and one
    2^-18 of their size, which fewer bits than fp32's would drop."""
    H, I = 256, 256
    c = moe_case(43, T, 1, 2, H, I, kind)
    c["w13"][:] = 0
    c["w13"][:, :, 0] = 0x38              # 1.0: gate and up are x's first value
    c["x"][:, 0] = 0x40                   # 2.0
    c["sx"][:] = 127 if kind == "e8m0" else 1.0
    for s in ("s13", "s2"):
        c[s][:] = 127 if kind == "e8m0" else 1.0
    c["w2"][:] = 0
    k = np.arange(H) % 120
    c["w2"][:, np.arange(H), k] = 0x7E                # 448
    c["w2"][:, np.arange(H), (k + 3) % 128] = 0xFE    # -448
    c["w2"][:, np.arange(H), (k + 5) % 128] = 0x01    # 2^-9
    c["weights"][:] = 1
    h = 2.0 / (1 + np.exp(-2.0)) * 2
    d = h / 448 if kind == "fp32" else 2.0 ** np.ceil(np.log2(h / 448))
    q = float(ref.e4m3_round(np.float64(h / d)))
    want = q * d * 2.0 ** -9
    # three products and the sums between them: at most 4 roundings of the largest
    tol = 4 * ref.FP32 * 2 * q * d * 448 + (ref.BF16 + 32 * ref.FP32) * want
    got = host(run_moe(c, kind))
    assert tol < 0.9 * want
    assert (np.abs(got - want) <= tol).all(), (got.min(), got.max(), want)
