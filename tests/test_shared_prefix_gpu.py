"""GPU parity of attention over shared prefixes (plans with groups) with the
fp64 oracle, which knows nothing of groups: it walks every request's own page
list.  Tolerances are those of the other plans (tests/gpu_util.py): a row's
parts are joined in fp32 like split partials."""
import numpy as np
import pytest
import torch

import synthetic
from gpu_util import DeviceWorkload, compare, to_dev
from test_fp8_mma_gpu import check as check_e4m3

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def va():
    import __graft_entry__
    __graft_entry__.build()
    import speculative_decoding_verify_gqa_gb300 as m
    return m


def make_shared(groups, shared, own, qo, page_size=16, **kw):
    """A workload whose requests (groups: members of each) start with shared[g] keys on the same pages."""
    of = [g for g, m in enumerate(groups) for _ in range(m)]
    wl = synthetic.make_custom(batch=len(of), page_size=page_size, qo=("fixed", qo),
                               prefix=("fixed", [shared[g] + o for g, o in zip(of, own)]), **kw)
    gi = np.concatenate([[0], np.cumsum(groups)]).astype(np.int32)
    sp = np.array([s // page_size for s in shared], np.int32)
    for g, m in enumerate(groups):
        r0 = int(gi[g])
        for b in range(r0 + 1, r0 + m):
            n, a, z = int(sp[g]), int(wl.kv_indptr[r0]), int(wl.kv_indptr[b])
            wl.kv_indices[z:z + n] = wl.kv_indices[a:a + n]
            ta, tz, k = int(wl.tok_indptr[r0]), int(wl.tok_indptr[b]), int(sp[g]) * page_size
            for x in (wl.k_tok, wl.v_tok):
                x[tz:tz + k] = x[ta:ta + k]
    return wl, gi, sp


def shared_plan(va, dw, gi, sp, **opts):
    wl = dw.wl
    o = dw.features()
    o.update(opts)
    return va.verify_attn_plan_shared(wl.kv_indptr, wl.qo_indptr, wl.last_page_len, wl.mask_indptr, gi, sp, wl.h_q,
                                      wl.h_kv, wl.d, wl.page_size, kv_dtype=wl.kv_dtype, device=dw.dev, **o)


def group_items(plan):
    return int((plan.items()[:, 0] >= plan.batch).sum())


def _run(va, wl, gi, sp, shares=True, **opts):
    dw = DeviceWorkload(wl)
    plan = shared_plan(va, dw, gi, sp, **opts)
    assert (group_items(plan) > 0) == shares
    out, lse, _ = dw.run(plan=plan)
    torch.cuda.synchronize()
    assert va.verify_attn_device_status(plan) == 0
    return dw, plan, out, lse


CASES = {
    "decode": dict(groups=[6], shared=[1024], own=[200, 3, 0, 77, 16, 500], qo=[1] * 6, h_q=32, h_kv=8, d=128),
    "chains": dict(groups=[9], shared=[768], own=[17 * i for i in range(9)], qo=[1, 5, 8, 3, 0, 8, 7, 1, 4], h_q=16, h_kv=2, d=128),
    "trees": dict(groups=[4, 3], shared=[640, 1280], own=[10, 0, 90, 300, 5, 128, 1], qo=[17, 9, 17, 30, 6, 17, 64], h_q=8,
                  h_kv=2, d=128, mask="tree"),
    "random_masks": dict(groups=[5], shared=[512], own=[0, 0, 7, 130, 60], qo=[9, 40, 12, 70, 3], h_q=8, h_kv=2, d=128,
                         mask="random"),
    "random_masks_shared": dict(groups=[5], shared=[4096], own=[0, 0, 7, 130, 60], qo=[9, 40, 12, 70, 3], h_q=8, h_kv=2, d=128,
                                mask="random"),
    "no_draft_visible": dict(groups=[4], shared=[512], own=[0, 5, 40, 0], qo=[9, 4, 12, 7], h_q=8, h_kv=2, d=128,
                             mask="none_visible"),
    "fp8": dict(groups=[6], shared=[2048], own=[200, 3, 0, 77, 16, 500], qo=[17] * 6, h_q=32, h_kv=8, d=128, mask="tree",
                kv_dtype=synthetic.FP8),
    "fp8_nhd": dict(groups=[3, 2], shared=[1024, 512], own=[31, 3, 0, 77, 16], qo=[5, 4, 3, 2, 1], h_q=16, h_kv=4, d=128,
                    kv_dtype=synthetic.FP8, kv_layout="nhd", page_size=32),
    "nhd": dict(groups=[5], shared=[1024], own=[31, 3, 0, 77, 16], qo=[5, 4, 3, 2, 1], h_q=16, h_kv=4, d=128, kv_layout="nhd"),
    "page_8": dict(groups=[5], shared=[1000], own=[31, 3, 0, 77, 16], qo=[5, 4, 3, 2, 1], h_q=16, h_kv=4, d=128, page_size=8),
    "page_1": dict(groups=[5], shared=[517], own=[31, 3, 0, 77, 16], qo=[5, 4, 3, 2, 1], h_q=4, h_kv=2, d=64, page_size=1),
    "page_256": dict(groups=[4], shared=[1024], own=[300, 3, 0, 77], qo=[5, 4, 3, 2], h_q=16, h_kv=4, d=128, page_size=256),
    "d64": dict(groups=[4, 1, 5], shared=[1000, 64, 512], own=[9] * 10, qo=[6, 5, 4, 3, 2, 1, 6, 5, 4, 3], h_q=14, h_kv=2,
                d=64, page_size=8),
    "d64_fp8": dict(groups=[8], shared=[1536], own=[40 * i for i in range(8)], qo=[4] * 8, h_q=8, h_kv=1, d=64,
                    kv_dtype=synthetic.FP8, mask="tree"),
    "group_3": dict(groups=[7], shared=[640], own=[33] * 7, qo=[3] * 7, h_q=12, h_kv=4, d=128),
    "value_width": dict(groups=[5], shared=[1024], own=[31, 3, 0, 77, 16], qo=[5, 4, 3, 2, 1], h_q=8, h_kv=4, d=128, dv=64),
    "rope": dict(groups=[5], shared=[1024], own=[31, 3, 0, 77, 16], qo=[5, 9, 3, 2, 1], h_q=16, h_kv=4, d=128, mask="tree",
                 rope_theta=10000.0),
    "mha": dict(groups=[8], shared=[1024], own=[20] * 8, qo=[2] * 8, h_q=4, h_kv=4, d=128),
    "long_rows": dict(groups=[2], shared=[768], own=[100, 0], qo=[150, 90], h_q=8, h_kv=2, d=128),
    "long_rows_shared": dict(groups=[2], shared=[9216], own=[100, 0], qo=[150, 90], h_q=8, h_kv=2, d=128),
    "uneven_tiles": dict(groups=[3], shared=[16 * 9], own=[1, 2, 3], qo=[1, 2, 1], h_q=4, h_kv=4, d=128),
}


# many rows over few shared keys: their partials would cost more than the keys, so the planner leaves them apart
APART = {"random_masks", "long_rows"}


@pytest.mark.parametrize("name", CASES)
def test_matches_oracle(va, name):
    c = dict(CASES[name])
    wl, gi, sp = make_shared(seed=3, **c)
    _, _, out, lse = _run(va, wl, gi, sp, shares=name not in APART)
    compare(wl, out, lse)


@pytest.mark.parametrize("kernel", [1, 2, 3, 4])
@pytest.mark.parametrize("opts", [dict(), dict(max_splits=1), dict(max_splits=7, min_chunk=128), dict(target_ctas=600)],
                         ids=["auto", "unsplit", "split", "many"])
def test_every_kernel_and_split(va, kernel, opts):
    wl, gi, sp = make_shared(groups=[6, 2], shared=[1536, 784], own=[200, 3, 0, 77, 16, 500, 40, 0], qo=[5, 1, 8, 17, 2, 3, 4, 6],
                             h_q=16, h_kv=2, d=128, mask="tree", seed=5)
    _, plan, out, lse = _run(va, wl, gi, sp, kernel=kernel, **opts)
    assert plan.header()["kernel"] == kernel
    compare(wl, out, lse)


@pytest.mark.parametrize("kernel", [3, 4])
def test_e4m3_mmas(va, kernel):
    """q_fp8 on a plan with groups: each part's P is rounded to e4m3 against its own maximum, so the
    bounds of tests/test_fp8_mma_gpu.py hold for each, and for their join, a weighted mean of them:
    sum e_j |v_j| over a part is at most that part's share of the row's, e_j falling with the
    distance of a part's maximum below the row's."""
    wl, gi, sp = make_shared(groups=[5], shared=[1024], own=[200, 3, 0, 77, 16], qo=[17, 5, 9, 1, 30], h_q=16, h_kv=4, d=128,
                             mask="tree", kv_dtype=synthetic.FP8, seed=6)
    _, _, out, lse = _run(va, wl, gi, sp, kernel=kernel, q_fp8=True)
    check_e4m3(wl, out, lse)


def test_equals_the_plan_without_groups_to_rounding(va):
    wl, gi, sp = make_shared(groups=[6], shared=[1024], own=[200, 3, 0, 77, 16, 500], qo=[5] * 6, h_q=32, h_kv=8, d=128, seed=8)
    dw, _, out, lse = _run(va, wl, gi, sp)
    ref, ref_lse, _ = dw.run()
    assert (lse - ref_lse).abs().max() < 1e-4
    assert (out.float() - ref.float()).abs().max() < 1e-2


def test_groups_not_worth_sharing_run_bit_equal(va):
    """No group shares: the items are those of one request at a time, unsplit -- the same bits."""
    wl, gi, sp = make_shared(groups=[3], shared=[16], own=[20, 3, 50], qo=[17, 9, 17], h_q=8, h_kv=2, d=128, seed=9)
    dw, _, out, lse = _run(va, wl, gi, sp, shares=False, max_splits=1)
    ref, ref_lse, _ = dw.run(max_splits=1)
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


def test_only_the_first_requests_pages_are_read(va):
    """The shared pages come from the group's first request: a page that the pool does not have
    in another request's list goes unnoticed, one in the first request's is flagged."""
    wl, gi, sp = make_shared(groups=[4], shared=[512], own=[20, 3, 50, 0], qo=[4] * 4, h_q=8, h_kv=2, d=128, seed=10)
    dw = DeviceWorkload(wl)
    plan = shared_plan(va, dw, gi, sp)
    good, _, _ = dw.run(plan=plan)
    for b, bits in ((2, 0), (0, 1)):
        kv = dw.kv_indices.clone()
        kv[int(wl.kv_indptr[b]) + 3] = wl.num_pages + 5
        out, _ = va.verify_attn_run(dw.q, dw.k_cache, dw.v_cache, dw.kv_indptr, kv, dw.last_page_len, dw.qo_indptr, None,
                                    None, plan, sm_scale=wl.sm_scale)
        torch.cuda.synchronize()
        assert va.verify_attn_device_status(plan) == bits
        assert torch.equal(out, good) == (bits == 0)


def test_tables_that_disagree_with_the_plan_are_flagged(va):
    """Device tables of another batch: items are skipped, nothing outside is read."""
    wl, gi, sp = make_shared(groups=[4], shared=[512], own=[20, 3, 50, 0], qo=[4] * 4, h_q=8, h_kv=2, d=128, seed=11)
    dw = DeviceWorkload(wl)
    plan = shared_plan(va, dw, gi, sp)
    short = torch.tensor([0, 8, 16, 24, 32], dtype=torch.int32, device="cuda")   # fewer pages than shared
    va.verify_attn_run(dw.q, dw.k_cache, dw.v_cache, short, dw.kv_indices, dw.last_page_len, dw.qo_indptr, None, None, plan)
    torch.cuda.synchronize()
    assert va.verify_attn_device_status(plan) & 2


def test_a_step_with_append_graph_and_side_stream(va):
    """verify_attn_append_run over a plan with groups, captured and replayed: the drafts' K/V
    written in the same call, new queries each replay."""
    for kv in (synthetic.BF16, synthetic.FP8):
        wl, gi, sp = make_shared(groups=[5], shared=[1024], own=[31, 3, 0, 77, 16], qo=[5, 9, 3, 2, 17], h_q=16, h_kv=4,
                                 d=128, mask="tree", kv_dtype=kv, seed=12)
        ref = DeviceWorkload(wl)
        plan = shared_plan(va, ref, gi, sp)
        want, want_lse, _ = ref.run(plan=plan)
        # a pool without the drafts
        dw = DeviceWorkload(wl, append=False)
        k_tok = to_dev(wl.k_tok.view(np.uint8 if kv == synthetic.FP8 else np.int16), "cuda", dw.kvd)
        v_tok = to_dev(wl.v_tok.view(np.uint8 if kv == synthetic.FP8 else np.int16), "cuda", dw.kvd)
        va.paged_kv_append(k_tok, v_tok, to_dev(wl.tok_indptr.astype(np.int32), "cuda"), dw.kv_indptr, dw.kv_indices,
                           dw.last_page_len, dw.k_cache, dw.v_cache)
        raw = dw.k_cache.view(torch.uint8)
        pre = raw.clone()
        out, lse = torch.empty_like(want), torch.empty_like(want_lse)
        side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()

        def step():
            va.verify_attn_append_run(dw.k_new, dw.v_new, dw.q, dw.k_cache, dw.v_cache, dw.kv_indptr, dw.kv_indices,
                                      dw.last_page_len, dw.qo_indptr, dw.mask, dw.mask_indptr, plan, sm_scale=wl.sm_scale,
                                      k_scale=wl.k_scale, v_scale=wl.v_scale, out=out, lse=lse)

        with torch.cuda.graph(g, stream=side):
            step()
        for _ in range(2):
            raw.fill_(255)
            raw.copy_(pre)
            # wipe the drafts' slots: the step has to write them
            for b in range(wl.batch):
                for i in range(int(wl.qo_lens[b])):
                    pos = int(wl.prefix_lens[b]) + i
                    page = int(wl.kv_indices[int(wl.kv_indptr[b]) + pos // wl.page_size])
                    dw.k_cache.view(torch.uint8)[page, :, pos % wl.page_size] = 255
                    dw.v_cache.view(torch.uint8)[page, :, pos % wl.page_size] = 255
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert va.verify_attn_device_status(plan) == 0
            assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_static_scratch_runs_a_plan_with_groups(va):
    wl, gi, sp = make_shared(groups=[5], shared=[512], own=[31, 3, 0, 77, 16], qo=[2] * 5, h_q=8, h_kv=2, d=128, seed=13)
    dw, plan, out, lse = _run(va, wl, gi, sp)
    got, got_lse = va.verify_attn_run_static_scratch(dw.q, dw.k_cache, dw.v_cache, dw.kv_indptr, dw.kv_indices,
                                                     dw.last_page_len, dw.qo_indptr, None, None, plan, sm_scale=wl.sm_scale)
    torch.cuda.synchronize()
    assert va.verify_attn_static_scratch_status() == 0
    assert torch.equal(out, got) and torch.equal(lse, got_lse)


def test_partial_and_merge_apart(va):
    wl, gi, sp = make_shared(groups=[5], shared=[512], own=[31, 3, 0, 77, 16], qo=[2] * 5, h_q=8, h_kv=2, d=128, seed=14)
    dw, plan, out, lse = _run(va, wl, gi, sp)
    got, got_lse = torch.zeros_like(out), torch.zeros_like(lse)
    va.verify_attn_partial(dw.q, dw.k_cache, dw.v_cache, dw.kv_indptr, dw.kv_indices, dw.last_page_len, dw.qo_indptr, None,
                           None, plan, sm_scale=wl.sm_scale, out=got, lse=got_lse)
    va.verify_attn_merge(dw.qo_indptr, plan, got, got_lse)
    torch.cuda.synchronize()
    assert torch.equal(out, got) and torch.equal(lse, got_lse)


@pytest.mark.parametrize("kernel", [2, 3, 4])
def test_plans_taking_turns_in_one_workspace(va, kernel):
    """Upload, append, run, upload the other plan, append, run, ... without a wait between: each run reads its own lists."""
    sets = [make_shared(groups=[7], shared=[1024], own=[31, 3, 0, 77, 16, 300, 9], qo=[5, 9, 3, 2, 17, 1, 4], h_q=16, h_kv=4,
                        d=128, mask="tree", seed=20),
            make_shared(groups=[3, 2], shared=[512, 2048], own=[100, 0, 5, 44, 700], qo=[1, 2, 30, 4, 6], h_q=16, h_kv=4,
                        d=128, mask="tree", seed=21)]
    dws, want = [], []
    for wl, gi, sp in sets:
        dw, plan, out, lse = _run(va, wl, gi, sp, kernel=kernel)
        dws.append(dw)
        want.append((out.clone(), lse.clone(), plan))
    ws = torch.empty(max(w[2].workspace_bytes for w in want), dtype=torch.uint8, device="cuda")
    got = []
    for turn in range(12):
        dw, (wl, gi, sp) = dws[turn % 2], sets[turn % 2]
        plan = shared_plan(va, dw, gi, sp, kernel=kernel, workspace=ws)
        va.paged_kv_append(dw.k_new, dw.v_new, dw.qo_indptr, dw.kv_indptr, dw.kv_indices, dw.last_page_len, dw.k_cache,
                           dw.v_cache)
        out, lse, _ = dw.run(plan=plan)
        got.append((out, lse))
    torch.cuda.synchronize()
    assert va.verify_attn_device_status(plan) == 0
    for turn, (out, lse) in enumerate(got):
        assert torch.equal(out, want[turn % 2][0]) and torch.equal(lse, want[turn % 2][1])


def test_workspace_of_the_bounds_serves_later_plans(va):
    wl, gi, sp = make_shared(groups=[5], shared=[512], own=[31, 3, 0, 77, 16], qo=[2] * 5, h_q=8, h_kv=2, d=128, seed=15)
    dw = DeviceWorkload(wl)
    _, n = va.verify_attn_plan_shared_bounds(wl.batch, 1, wl.total_qo, wl.h_q, wl.h_kv, wl.d)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for opts in ({}, dict(target_ctas=600), dict(max_splits=2), dict(kernel=1)):
        out, lse, _ = dw.run(plan=shared_plan(va, dw, gi, sp, workspace=ws, **opts))
        compare(wl, out, lse)
    with pytest.raises(va.VerifyAttnError):
        shared_plan(va, dw, gi, sp, workspace=ws[:256])
