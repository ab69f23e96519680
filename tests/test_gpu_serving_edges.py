"""Edges of the operators that serve many requests at once, and of the serving step that runs them.

Tolerances of the adapters, with u the unit roundoff of the outputs' type: an output is rounded once (u |out|); the
sum over x meets B as two or more terms of the operands' type, which lose at most 2^-16 of it for bfloat16 (8 + 8 bits)
and 2^-20 for float16 (11 + 11 bits, less what falls below the smallest); the two products are summed in float32,
(K + R) adds of at most 2^-23 of the sum of their terms' sizes; where the second product is summed onto the old value,
16 of them at most are of its size.
"""
import numpy as np
import pytest
import torch

import sharded_gemm_gb300 as tp
from sharded_gemm_gb300 import build as tpbuild
from sharded_gemm_gb300 import synth
from sharded_gemm_gb300.workloads import PagedServing, SharedServing
from test_gpu_serving import (BF16, F16, F32, U, call_lora, check_verify, dev, drafted, embeddings, i32, lora_data,
                              lora_ref, make_adapters, padded, settings_of, status, verify_ref)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    tpbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    tp.tp_set_policy(tp.TP_POLICY_AUTO)


# ------------------------------------------------------------------ the bits of h
@pytest.mark.parametrize("dt,out_dt", [(BF16, BF16), (F16, F16), (BF16, F16), (F16, BF16)])
@pytest.mark.parametrize("T,R", [(1, 16), (40, 16), (300, 64), (600, 128), (1100, 16), (1500, 64), (1030, 32)])
def test_adapters_keep_16_bits_of_the_sum_over_x(T, R, dt, out_dt):
    """Where an adapter's outputs cancel, what is left is as exact as the outputs' type holds it."""
    n, K, O = 3, 512, 256
    x, a, b, y, s = lora_data("column", T, 2, K, O, R, n, dt, out_dt, T + R)
    ids = np.random.default_rng(T).integers(0, n, T)
    plan = tp.tp_lora_plan(i32(ids), T, n)
    lost = (2.0 ** -16 if dt == BF16 else 2.0 ** -20) + (K + R) * 2.0 ** -23
    for start in ([torch.zeros_like(t) for t in y], y):
        got = call_lora("column", x, a, b, plan, start, scales=s, out=[torch.empty_like(t) for t in y])
        ref, big = lora_ref(x, a, b, dev(ids), s, start)
        for g, f, size, old in zip(got, ref, big, start):
            tol = U[out_dt] * f.abs() + lost * size + 2.0 ** -19 * old.double().abs() + 2.0 ** -24
            worst = ((g.double() - f).abs() / tol).max()
            assert worst <= 1, float(worst)
    assert status() == 0
