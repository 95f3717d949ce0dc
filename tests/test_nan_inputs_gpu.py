"""NaN in what a row sees makes that row NaN, in out and in lse, and no other
row's bits change: as softmax(q k^T) v has it, whichever kernel, split, group
or merge the row went through.  Each case runs one plan on clean values and
again with a NaN put into them."""
import numpy as np
import pytest
import torch

import synthetic
from gpu_util import DeviceWorkload
from test_shared_prefix_gpu import group_items, make_shared, shared_plan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def va():
    import __graft_entry__
    __graft_entry__.build()
    import speculative_decoding_verify_gqa_gb300 as m
    return m


def _sees(wl, b, pos):
    """Tokens of request b that see its key at position pos."""
    n, pre = int(wl.qo_lens[b]), int(wl.prefix_lens[b])
    u = pos - pre
    return [t for t in range(n) if u < 0 or (wl.mask_dense[b][t, u] if wl.mask_dense else u <= t)]


def _poke(wl, dw, cache, b, pos, h, e):
    """NaN into element e of head h of request b's row at this position; the rows [T, h_q] that see it."""
    page = int(wl.kv_indices[int(wl.kv_indptr[b]) + pos // wl.page_size])
    at = (page, pos % wl.page_size, h, e) if wl.nhd else (page, h, pos % wl.page_size, e)
    cache[at] = float("nan")
    assert bool(cache[at].isnan())
    rows = np.zeros((wl.total_qo, wl.h_q), bool)
    for c in range(wl.batch):
        pages = wl.kv_indices[int(wl.kv_indptr[c]):int(wl.kv_indptr[c + 1])].tolist()
        if page in pages:
            p = pages.index(page) * wl.page_size + pos % wl.page_size
            if p < int(wl.kv_lens[c]):
                for t in _sees(wl, c, p):
                    rows[int(wl.qo_indptr[c]) + t, h * wl.group:(h + 1) * wl.group] = True
    return rows


def _pair(wl, dw, plan):
    out, lse, _ = dw.run(plan=plan)
    return out.clone(), lse.clone()


def _check(va, wl, dw, plan, clean, rows, col=None):
    """rows: all NaN (or in column col alone, lse untouched); the others: the clean run's bits."""
    out, lse, _ = dw.run(plan=plan)
    torch.cuda.synchronize()
    assert va.verify_attn_device_status(plan) == 0
    hit = torch.from_numpy(rows).cuda()
    bits = lambda x: x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32)  # noqa: E731
    assert torch.equal(bits(out[~hit]), bits(clean[0][~hit])) and torch.equal(bits(lse[~hit]), bits(clean[1][~hit]))
    if col is None:
        assert out[hit].isnan().all() and lse[hit].isnan().all()
        return
    keep = torch.arange(wl.dv, device="cuda") != col
    assert torch.equal(bits(lse[hit]), bits(clean[1][hit]))
    assert torch.equal(bits(out[hit][:, keep]), bits(clean[0][hit][:, keep])) and out[hit][:, col].isnan().all()


def _cases(wl, dw, plan, va, keys):
    clean = _pair(wl, dw, plan)
    assert clean[0].isfinite().all()
    k0, v0, q0 = dw.k_cache.clone(), dw.v_cache.clone(), dw.q.clone()
    for n, (b, pos) in enumerate(keys):
        h, e = n % wl.h_kv, (37 * n) % wl.d
        _check(va, wl, dw, plan, clean, _poke(wl, dw, dw.k_cache, b, pos, h, e))
        dw.k_cache.view(torch.uint8).copy_(k0.view(torch.uint8))
        if len(_sees(wl, b, pos)) == int(wl.qo_lens[b]):
            e = (37 * n) % wl.dv
            _check(va, wl, dw, plan, clean, _poke(wl, dw, dw.v_cache, b, pos, h, e), col=e)
            dw.v_cache.view(torch.uint8).copy_(v0.view(torch.uint8))
    t, qh = wl.total_qo // 2, wl.h_q - 1
    dw.q[t, qh, 5] = float("nan")
    rows = np.zeros((wl.total_qo, wl.h_q), bool)
    rows[t, qh] = True
    _check(va, wl, dw, plan, clean, rows)
    dw.q.copy_(q0)


FORMS = {
    "d64_mma64": dict(d=64, kernel=1), "d64_mma128_fp8": dict(d=64, kernel=2, kv_dtype=synthetic.FP8),
    "mma64": dict(kernel=1), "mma128": dict(kernel=2), "mma64_fp8": dict(kernel=1, kv_dtype=synthetic.FP8, kv_layout="nhd"),
    "tc128": dict(kernel=3), "tc256": dict(kernel=4), "tc128_fp8": dict(kernel=3, kv_dtype=synthetic.FP8),
    "tc256_fp8_nhd": dict(kernel=4, kv_dtype=synthetic.FP8, kv_layout="nhd"),
    "tc128_e4m3": dict(kernel=3, kv_dtype=synthetic.FP8, q_fp8=True),
    "tc256_e4m3": dict(kernel=4, kv_dtype=synthetic.FP8, q_fp8=True),
}


def _split(form):
    form = dict(form)
    opts = {k: form.pop(k) for k in ("kernel", "q_fp8") if k in form}
    return dict(dict(d=128), **form), opts


@pytest.mark.parametrize("splits", [1, 0], ids=["whole", "split"])
@pytest.mark.parametrize("form", FORMS)
def test_plans_without_groups(va, form, splits):
    """Trees behind prefixes of three lengths; a request of one key; a key in the first, a middle and the last part."""
    shape, opts = _split(FORMS[form])
    wl = synthetic.make_custom(batch=4, h_q=8, h_kv=2, prefix=("fixed", [900, 0, 130, 3000]), qo=("fixed", [17, 1, 40, 5]),
                               mask="tree", seed=3, **shape)
    dw = DeviceWorkload(wl)
    plan = dw.plan(max_splits=splits, target_ctas=300, min_chunk=64, **opts)
    assert (plan.header()["max_nsplit"] > 4) == (splits == 0)
    keys = [(0, 0), (0, 500), (0, 899), (0, 900), (0, 905), (1, 0), (2, 129), (2, 150), (2, 169), (3, 2999), (3, 1400)]
    _cases(wl, dw, plan, va, keys)


@pytest.mark.parametrize("form", FORMS)
def test_plans_with_groups(va, form):
    """A NaN in a page that a group shares, in a request's own keys, and in a draft."""
    shape, opts = _split(FORMS[form])
    wl, gi, sp = make_shared(groups=[4, 3], shared=[1024, 2048], own=[10, 0, 90, 300, 5, 128, 1], qo=[17, 9, 17, 30, 6, 17, 64],
                             h_q=8, h_kv=2, mask="tree", seed=4, **shape)
    dw = DeviceWorkload(wl)
    plan = shared_plan(va, dw, gi, sp, **opts)
    assert group_items(plan) > 0
    keys = [(0, 0), (2, 1023), (3, 1100), (3, 1323), (3, 1329), (5, 2047), (4, 0), (6, 700), (6, 2048), (6, 2060), (1, 1024)]
    _cases(wl, dw, plan, va, keys)


@pytest.mark.parametrize("kernel", [1, 3])
def test_infinite_keys_in_masked_places_change_nothing(va, kernel):
    """Infinite and NaN keys of drafts: the rows that do not see them keep their bits, and those that do have no number."""
    wl = synthetic.make_custom(batch=2, h_q=8, h_kv=2, d=128, prefix=("fixed", [300, 40]), qo=("fixed", [17, 30]), mask="tree",
                               seed=6)
    dw = DeviceWorkload(wl)
    plan = dw.plan(kernel=kernel)
    clean = _pair(wl, dw, plan)
    b, u = 1, 11
    rows = _poke(wl, dw, dw.k_cache, b, 40 + u, 1, 3)
    page = int(wl.kv_indices[int(wl.kv_indptr[b]) + (40 + u) // wl.page_size])
    dw.k_cache[page, 1, (40 + u) % wl.page_size] = float("inf")
    out, lse, _ = dw.run(plan=plan)
    torch.cuda.synchronize()
    hit = torch.from_numpy(rows).cuda()
    assert 0 < int(hit.sum()) < hit.numel()
    assert torch.equal(out[~hit], clean[0][~hit]) and torch.equal(lse[~hit], clean[1][~hit])
    assert out[hit].isnan().all()
