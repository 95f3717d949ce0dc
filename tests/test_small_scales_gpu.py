"""Queries and scales so small that every score is 0 to fp32: attention is the mean of the
values that a row sees, its LSE the logarithm of their number."""
import ctypes

import numpy as np
import pytest
import torch

import synthetic
from gpu_util import DeviceWorkload


@pytest.fixture(scope="module")
def va():
    import __graft_entry__
    __graft_entry__.build()
    import speculative_decoding_verify_gqa_gb300 as m
    return m


def _workload(fp8, **kw):
    return synthetic.make_custom(batch=2, h_q=8, h_kv=2, d=128, prefix=("fixed", [300, 0]), qo=("fixed", [17, 30]), mask="tree",
                                 kv_dtype=synthetic.FP8 if fp8 else synthetic.BF16, seed=9, **kw)


def _values(wl):
    raw = torch.from_numpy(wl.v_tok.view(np.uint8 if wl.kv_dtype == synthetic.FP8 else np.int16))
    v = raw.view(torch.float8_e4m3fn if wl.kv_dtype == synthetic.FP8 else torch.bfloat16)
    return v.float().double().numpy() * wl.v_scale


def _check(wl, out, lse, tol):
    """Uniform attention over the visible keys, in 64 bits."""
    v = _values(wl)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(wl.batch):
        pre, t0 = int(wl.prefix_lens[b]), int(wl.tok_indptr[b])
        for t in range(int(wl.qo_lens[b])):
            sees = np.r_[np.arange(pre), pre + np.flatnonzero(wl.mask_dense[b][t])]
            mean = np.repeat(v[t0 + sees].mean(0), wl.group, 0)
            row = int(wl.qo_indptr[b]) + t
            assert np.abs(lse[row] - np.log(len(sees))).max() <= 1e-6 * max(1.0, np.log(len(sees)))
            # p = 1 is exact in every operand type; sums fp32, out rounded to bf16
            assert (np.abs(out[row] - mean) <= tol + 2.0 ** -8 * np.abs(mean)).all()


# 330 additions in fp32 of values below 6, relative to the sum 2^-24 each: 330 * 2^-24 * 6
TOL = 1.2e-4


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", [1, 2, 3, 4])
@pytest.mark.parametrize("form", ["bf16", "fp8", "e4m3"])
def test_small_scales(va, kernel, form):
    """sm_scale * k_scale below the smallest fp32 number: masked keys stay masked."""
    if form == "e4m3" and kernel < 3:
        pytest.skip("tcgen05 kernels only")
    wl = _workload(form != "bf16")
    wl.sm_scale, wl.k_scale = 1e-30, 1e-20
    dw = DeviceWorkload(wl)
    opts = dict(q_fp8=True) if form == "e4m3" else {}
    for splits in (1, 0):
        out, lse, _ = dw.run(kernel=kernel, max_splits=splits, target_ctas=200, min_chunk=64, **opts)
        _check(wl, out, lse, TOL)


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", [3, 4])
@pytest.mark.parametrize("size", [1e-28, 1e-31, 1e-37, 3e-39, 1e-40])
def test_small_queries_with_e4m3_operands(va, kernel, size):
    """Rows whose largest element is far below the e4m3 scale's range, zeros among them."""
    wl = _workload(True)
    dw = DeviceWorkload(wl)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = (torch.rand(dw.q.shape, generator=g, device="cuda") - 0.5) * 2 * size
    q[..., ::3] = 0
    dw.q.copy_(q.to(torch.bfloat16))
    for splits in (1, 0):
        out, lse, _ = dw.run(kernel=kernel, q_fp8=True, max_splits=splits, target_ctas=200, min_chunk=64)
        _check(wl, out, lse, TOL)


def test_scales_whose_product_overflows_are_refused(va):
    plan = va.verify_attn_plan_host([0, 2], [0, 3], [5], None, 4, 2, 128, 16, num_sms=152)
    fake = ctypes.c_void_p(4096)   # never dereferenced: the check fails first
    args = [fake] * 7 + [None, None]
    rc = va.lib().verify_attn_run(*args, 4, 2, 128, 16, 1e20, 1e20, 1.0, fake, None, 10, va._hp(plan.host), fake, 1 << 30, None)
    assert rc == -1
