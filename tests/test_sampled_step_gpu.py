"""One serving step through the operators together, as a server uses them:
requests behind a shared prompt -> groups found from the page tables -> plan
-> the drafts' append and their attention in one call -> the target's logits
(a random LM head here) -> sampled acceptance -> compaction -> the next token
of every request over the compacted cache.  Acceptance against its oracle,
attention (both steps) against the attention oracle, which builds its own
cache from the tokens that were accepted."""
import numpy as np
import pytest
import torch

import synthetic
from gpu_util import DeviceWorkload, compare, to_dev
from oracle.accept_sample import accept_sampled
from test_shared_prefix_gpu import make_shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def va():
    import __graft_entry__
    __graft_entry__.build()
    import speculative_decoding_verify_gqa_gb300 as m
    return m


@pytest.mark.parametrize("kv,layout,d", [(synthetic.BF16, "hnd", 128), (synthetic.FP8, "nhd", 128), (synthetic.BF16, "nhd", 64)])
@pytest.mark.parametrize("peak", [0.4, 6.0], ids=["flat", "peaked"])
def test_step(va, kv, layout, d, peak):
    raw = np.uint8 if kv == synthetic.FP8 else np.int16
    wl, _, _ = make_shared(groups=[5, 2], shared=[512, 256], own=[31, 3, 0, 77, 16, 40, 9], qo=[9, 17, 5, 12, 1, 30, 8], h_q=8,
                           h_kv=2, d=d, mask="tree", kv_dtype=kv, kv_layout=layout, seed=20)
    B, T, V = wl.batch, wl.total_qo, 1000
    rng = np.random.default_rng(7)
    gen = torch.Generator(device="cuda").manual_seed(7)

    # the cache as the last step left it: every prefix, no drafts
    dw = DeviceWorkload(wl, append=False)
    tok = lambda x: to_dev(x.view(raw), "cuda", dw.kvd)  # noqa: E731
    va.paged_kv_append(tok(wl.k_tok), tok(wl.v_tok), to_dev(wl.tok_indptr.astype(np.int32), "cuda"), dw.kv_indptr,
                       dw.kv_indices, dw.last_page_len, dw.k_cache, dw.v_cache, kv_layout=layout)
    for x in (dw.k_cache.view(torch.uint8), dw.v_cache.view(torch.uint8)):
        for b in range(B):
            for i in range(int(wl.qo_lens[b])):
                pos = int(wl.prefix_lens[b]) + i
                page = int(wl.kv_indices[int(wl.kv_indptr[b]) + pos // wl.page_size])
                if layout == "nhd":
                    x[page, pos % wl.page_size] = 255
                else:
                    x[page, :, pos % wl.page_size] = 255

    # groups, plan, append + attention
    gi, sp = va.verify_attn_shared_groups(wl.kv_indptr, wl.kv_indices, wl.qo_indptr, wl.last_page_len, wl.page_size)
    assert gi.tolist() == [0, 5, 7] and sp.tolist() == [32, 16]
    plan = va.verify_attn_plan_shared(wl.kv_indptr, wl.qo_indptr, wl.last_page_len, wl.mask_indptr, gi, sp, wl.h_q, wl.h_kv,
                                      d, wl.page_size, kv_dtype=kv, kv_layout=layout)
    out, lse = va.verify_attn_append_run(dw.k_new, dw.v_new, dw.q, dw.k_cache, dw.v_cache, dw.kv_indptr, dw.kv_indices,
                                         dw.last_page_len, dw.qo_indptr, dw.mask, dw.mask_indptr, plan,
                                         sm_scale=wl.sm_scale, k_scale=wl.k_scale, v_scale=wl.v_scale, kv_layout=layout)
    assert va.verify_attn_device_status(plan) == 0
    compare(wl, out, lse)

    # the target's logits, and drafts that often are what it would emit
    head = torch.randn((wl.h_q * d, V), generator=gen, device="cuda") * peak
    logits = (out.float().view(T, -1) @ head).to(torch.bfloat16)
    host = logits.double().cpu().numpy()
    parents = np.concatenate([np.array(p, np.int32) for p in wl.parents])
    toks = np.zeros(T, np.int32)
    for b in range(B):
        o = int(wl.qo_indptr[b])
        for i in range(1, int(wl.qo_lens[b])):
            toks[o + i] = host[o + parents[o + i]].argmax() if rng.random() < 0.7 else rng.integers(V)
    temp = np.full(B, 0.5, np.float32)
    temp[2] = 0.0
    for _ in range(20):   # numbers that leave every decision clear of its border, by the oracle alone
        u, noise = rng.random(T).astype(np.float32), rng.exponential(size=(B, V)).astype(np.float32)
        r_acc, r_paths, r_bonus, _, margin = accept_sampled(host, wl.qo_indptr, toks, parents, u, noise, temp)
        if margin > 1e-4:
            break
    assert margin > 1e-4
    cu = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    acc, path, bonus, _ = va.verify_accept_sample(logits, dw.qo_indptr, cu(toks), cu(parents), cu(u), cu(noise),
                                                  temperature=cu(temp), status=status)
    assert acc.tolist() == r_acc.tolist() and bonus.tolist() == r_bonus.tolist()
    # flat logits accept little; peaked ones most of what was planted
    assert (r_acc > 1).sum() >= (1 if peak < 1 else 4)
    kv_len = torch.empty(B, dtype=torch.int32, device="cuda")
    va.paged_kv_compact(acc, path, dw.qo_indptr, dw.kv_indptr, dw.kv_indices, dw.last_page_len, dw.k_cache, dw.v_cache,
                        kv_layout=layout, kv_len_out=kv_len, status=status)
    assert int(status) == 0
    assert kv_len.tolist() == [int(p + a) for p, a in zip(wl.prefix_lens, r_acc)]

    # the next step, as a workload of its own: prefix and accepted drafts, then one new token
    nxt = synthetic.make_custom(batch=B, h_q=wl.h_q, h_kv=wl.h_kv, d=d, page_size=wl.page_size, kv_dtype=kv, kv_layout=layout,
                                prefix=("fixed", (wl.prefix_lens + r_acc).tolist()), qo=("fixed", [1] * B), seed=21)
    nxt.k_scale, nxt.v_scale = wl.k_scale, wl.v_scale
    for b in range(B):
        s, t = int(wl.tok_indptr[b]), int(nxt.tok_indptr[b])
        pre = int(wl.prefix_lens[b])
        rows = np.concatenate([np.arange(pre), pre + r_paths[b]])
        for x, y in ((nxt.k_tok, wl.k_tok), (nxt.v_tok, wl.v_tok)):
            x[t:t + len(rows)] = y[s + rows]
    # its pages: the requests' own, as many as it needs (a new one where the next token starts a page)
    n_pages = wl.num_pages
    ids, ptr = [], [0]
    pool = [x for x in (dw.k_cache, dw.v_cache)]
    spare = [i for i in range(n_pages) if i not in set(wl.kv_indices.tolist())]
    for b in range(B):
        need = -(-int(nxt.kv_lens[b]) // wl.page_size)
        own = wl.kv_indices[int(wl.kv_indptr[b]):int(wl.kv_indptr[b + 1])].tolist()[:need]
        while len(own) < need:
            own.append(spare.pop())
        ids += own
        ptr.append(len(ids))
    kvp, kvi = np.array(ptr, np.int32), np.array(ids, np.int32)
    last = ((nxt.kv_lens - 1) % wl.page_size + 1).astype(np.int32)
    kn, vn = nxt.new_tokens()
    qd = cu(nxt.q.view(np.int16)).view(torch.bfloat16)
    plan2 = va.verify_attn_plan(kvp, nxt.qo_indptr, last, None, wl.h_q, wl.h_kv, d, wl.page_size, kv_dtype=kv, kv_layout=layout)
    out2, lse2 = va.verify_attn_append_run(tok(kn), tok(vn), qd, pool[0], pool[1], cu(kvp), cu(kvi), cu(last),
                                           cu(nxt.qo_indptr), None, None, plan2, sm_scale=nxt.sm_scale, k_scale=wl.k_scale,
                                           v_scale=wl.v_scale, kv_layout=layout)
    assert va.verify_attn_device_status(plan2) == 0
    compare(nxt, out2, lse2)
