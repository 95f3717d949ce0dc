"""Cases of the operators around one verification step: sampled acceptance of
drafted tokens, attention over a prefix that the requests of a batch share,
and compaction of the accepted path in the paged cache.

``run`` computes an operator in plain torch operations, or, with ``own``
true, through the package's calls; ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}


def _va():
    import speculative_decoding_verify_gqa_gb300 as va
    return va


# ----------------------------------------------------------------- the cases

def listed():
    """Sampled acceptance.
    sample_one: one chat stream with a 4-token chain; latency is all.
    sample_chains: a serving batch of ragged chains with the draft model's
      distributions, over a Llama-3-sized vocabulary, mixed temperatures.
    sample_wide_tree: 8 requests x 64-node trees of top-k drafts (no draft
      distributions), the wide tree of this repository's own workloads.
    sample_odd: fp32 logits over an odd vocabulary (rows off every 16-byte
      boundary), trees whose siblings are drawn from bf16 draft distributions.

    Attention over a shared prefix.
    shared_parallel: 4 samples of one prompt, one token each (plain decode).
    shared_system: a serving batch behind one system prompt, ragged chains.
    shared_trees: three prompts of a long-context service, their answers
      drafted as 17-node trees over an fp8 cache (head layout NHD).
    shared_d64: head_dim 64 and 8-token pages (the warp-level kernels).
    shared_big: the CodeLLaMA-34B-shaped batch behind a long prompt.

    Compaction after acceptance.
    keep_one: one 17-node tree, one layer's cache.
    keep_layers: a serving batch of chains, every layer of a 32-layer cache.
    keep_fp8: wide trees over an fp8 cache, NHD, 16 layers.
    """
    return [
        dict(name="sample_one", op="sample", batch=1, nodes=5, ragged=False, tree=False, vocab=32016,
             logits="bf16", draft="f32", temps="one", shape_seed=1),
        dict(name="sample_chains", op="sample", batch=64, nodes=8, ragged=True, tree=False, vocab=128256,
             logits="bf16", draft="f32", temps="mixed", shape_seed=2),
        dict(name="sample_wide_tree", op="sample", batch=8, nodes=64, ragged=False, tree=True, vocab=128256,
             logits="bf16", draft="none", temps="none", shape_seed=3),
        dict(name="sample_odd", op="sample", batch=12, nodes=17, ragged=True, tree=True, vocab=50257,
             logits="f32", draft="bf16", temps="mixed", shape_seed=4),
        dict(name="shared_parallel", op="shared", groups=1, members=4, own=200, nodes=1, ragged=False, tree=False,
             shared=2048, h_q=32, h_kv=8, d=128, page=16, kv="bf16", nhd=False, shape_seed=5),
        dict(name="shared_system", op="shared", groups=1, members=32, own=500, nodes=5, ragged=True, tree=False,
             shared=4096, h_q=32, h_kv=8, d=128, page=16, kv="bf16", nhd=False, shape_seed=6),
        dict(name="shared_trees", op="shared", groups=3, members=8, own=700, nodes=17, ragged=True, tree=True,
             shared=16384, h_q=32, h_kv=8, d=128, page=32, kv="fp8", nhd=True, shape_seed=7),
        dict(name="shared_d64", op="shared", groups=2, members=5, own=90, nodes=6, ragged=True, tree=False,
             shared=1000, h_q=14, h_kv=2, d=64, page=8, kv="bf16", nhd=False, shape_seed=8),
        dict(name="shared_big", op="shared", groups=1, members=64, own=1024, nodes=8, ragged=True, tree=False,
             shared=8192, h_q=64, h_kv=8, d=128, page=16, kv="bf16", nhd=False, shape_seed=9),
        dict(name="keep_one", op="keep", batch=1, nodes=17, layers=1, h_kv=8, d=128, page=16, kv="bf16", nhd=False,
             shape_seed=10),
        dict(name="keep_layers", op="keep", batch=64, nodes=8, layers=32, h_kv=8, d=128, page=16, kv="bf16",
             nhd=False, shape_seed=11),
        dict(name="keep_fp8", op="keep", batch=8, nodes=64, layers=16, h_kv=8, d=64, page=32, kv="fp8", nhd=True,
             shape_seed=12),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: any operator, sizes over the listed cases' ranges."""
    op = rng.choice(["sample", "shared", "keep"])
    seed = rng.randrange(1 << 20)
    if op == "sample":
        batch, vocab = _log(rng, 1, 64), _log(rng, 1000, 128256)
        nodes = _log(rng, 1, max(1, min(64, 512 // batch)))
        return dict(op=op, batch=batch, nodes=nodes, ragged=rng.random() < 0.5, tree=rng.random() < 0.5, vocab=vocab,
                    logits=rng.choice(["bf16", "f32"]), draft=rng.choice(["none", "bf16", "f32"]),
                    temps=rng.choice(["none", "one", "mixed"]), shape_seed=seed)
    if op == "shared":
        d = rng.choice([64, 128, 128])
        h_kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4, 8])
        groups, nodes = _log(rng, 1, 4), _log(rng, 1, 16)
        members = _log(rng, 1, max(1, 64 // (groups * group)))
        page = rng.choice([1, 8, 16, 32, 64])
        shared = _log(rng, 64, 16384) // page * page
        return dict(op=op, groups=groups, members=members, own=_log(rng, 1, 1024), nodes=nodes,
                    ragged=rng.random() < 0.7, tree=rng.random() < 0.5, shared=shared, h_q=h_kv * group, h_kv=h_kv,
                    d=d, page=page, kv=rng.choice(["bf16", "fp8"]), nhd=rng.random() < 0.5, shape_seed=seed)
    batch = _log(rng, 1, 64)
    return dict(op=op, batch=batch, nodes=_log(rng, 1, 64), layers=_log(rng, 1, max(1, 512 // batch // 4)),
                h_kv=rng.choice([1, 2, 8]), d=rng.choice([64, 128]), page=rng.choice([1, 4, 16, 64]),
                kv=rng.choice(["bf16", "fp8"]), nhd=rng.random() < 0.5, shape_seed=seed)


def _lens(case, n):
    """Query tokens of each of n requests: the case's own shape, the same for every seed."""
    r = random.Random(case["shape_seed"])
    return [r.randint(1, case["nodes"]) if case.get("ragged", True) else case["nodes"] for _ in range(n)]


def _own_lens(case, n):
    """Keys of each request between the shared prefix and its drafts."""
    r = random.Random(case["shape_seed"] + 77)
    return [r.randint(0, case["own"]) if case["ragged"] else case["own"] for _ in range(n)]


def _indptr(lens):
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return out


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tree(lens, tree, r):
    """Parents of each request's nodes: a chain, or node i below a node drawn from 0 .. i - 1."""
    out = []
    for n in lens:
        out += [-1] + [r.randrange(i) if tree else i - 1 for i in range(1, n)]
    return out


def _paths(lens, parents, r):
    """A root path of each request, as acceptance leaves it: from a drawn node up."""
    acc, path, o = [], [], 0
    for n in lens:
        v, p = r.randrange(n), []
        while v >= 0:
            p.append(v)
            v = parents[o + v]
        acc.append(len(p))
        path += p[::-1] + [-1] * (n - len(p))
        o += n
    return acc, path


# ---------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    return {"sample": _prepare_sample, "shared": _prepare_shared, "keep": _prepare_keep}[case["op"]](case, g, r)


def _prepare_sample(case, g, r):
    lens = _lens(case, case["batch"])
    total, V = sum(lens), case["vocab"]
    parents = _tree(lens, case["tree"], r)
    indptr = _indptr(lens)
    # peaked like a language model's: a few likely tokens over a broad tail
    x = torch.randn((total, V), generator=g, device="cuda") * 2
    hot = torch.randint(0, V, (total, 8), generator=g, device="cuda")
    x.scatter_(1, hot, math.log(V) + torch.randn((total, 8), generator=g, device="cuda") * 2)
    logits = x.to(_DT[case["logits"]])
    temps = None
    if case["temps"] == "one":
        temps = torch.full((case["batch"],), 0.8, device="cuda")
    elif case["temps"] == "mixed":
        temps = torch.rand(case["batch"], generator=g, device="cuda") * 0.8 + 0.5
        temps[torch.rand(case["batch"], generator=g, device="cuda") < 0.125] = 0.0
    # the draft model: near the target; drafts drawn from it, or its top tokens
    x = logits.float()
    if temps is not None:
        x /= temps.clamp(min=0.5).repeat_interleave(torch.tensor(lens, device="cuda"))[:, None]
    x += torch.randn((total, V), generator=g, device="cuda") * 0.5
    q = torch.softmax(x, 1)
    par = torch.tensor([max(p, 0) + indptr[b] for b, n in enumerate(lens) for p in parents[indptr[b]:indptr[b] + n]],
                       device="cuda")
    if case["draft"] == "none":
        seen, rank = {}, []
        for p in par.tolist():
            rank.append(seen.get(p, -1))   # a root counts first: its own entry is no child
            seen[p] = rank[-1] + 1
        k = min(V, max(1, max(rank) + 1))
        top = q.topk(k, 1).indices
        toks = top[par, torch.tensor(rank, device="cuda").clamp(0, k - 1)]
        probs = None
    else:
        probs = q.to(_DT[case["draft"]])
        toks = torch.empty(total, dtype=torch.int64, device="cuda")
        for a in range(0, total, 64):
            e = torch.empty((min(64, total - a), V), device="cuda").exponential_(generator=g)
            toks[a:a + 64] = (q[par[a:a + 64]] / e).argmax(1)
    return dict(op="sample", case=case, logits=logits, probs=probs, temps=temps, toks=toks.to(torch.int32),
                parents=_i32(parents), indptr=_i32(indptr), max_nodes=max(lens),
                u=torch.rand(total, generator=g, device="cuda"),
                noise=torch.empty((case["batch"], V), device="cuda").exponential_(generator=g))


def _pool(case, pages, g, layers=None):
    """K or V pages; every slot holds something, as a pool in use does."""
    mid = (case["page"], case["h_kv"]) if case["nhd"] else (case["h_kv"], case["page"])
    shape = (() if layers is None else (layers,)) + (pages,) + mid + (case["d"],)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _prepare_shared(case, g, r):
    B, P = case["groups"] * case["members"], case["page"]
    lens, mid = _lens(case, B), _own_lens(case, B)
    kv_lens = [case["shared"] + a + n for a, n in zip(mid, lens)]
    sp = case["shared"] // P
    need = [-(-k // P) - sp for k in kv_lens]
    n_pages = case["groups"] * sp + sum(need)
    n_pages += n_pages // 8 + 1
    ids = list(range(n_pages))
    r.shuffle(ids)
    indices, kv_indptr, at = [], [0], case["groups"] * sp
    for b in range(B):
        grp = b // case["members"]
        indices += ids[grp * sp:(grp + 1) * sp] + ids[at:at + need[b]]
        at += need[b]
        kv_indptr.append(len(indices))
    last = [(k - 1) % P + 1 for k in kv_lens]
    indptr = _indptr(lens)
    bits, mask_indptr = [], None
    if case["tree"]:
        parents = _tree(lens, True, r)
        mask_indptr = [0]
        for b, n in enumerate(lens):
            rows = []
            for i in range(n):
                p = parents[indptr[b] + i]
                row = list(rows[p]) if p >= 0 else [0] * n
                row[i] = 1
                rows.append(row)
            bits += [x for row in rows for x in row]
            mask_indptr.append(len(bits))
        bits += [0] * (-len(bits) % 8)
        w = torch.tensor(bits, dtype=torch.int32).view(-1, 8) << torch.arange(8, dtype=torch.int32)
        mask = w.sum(1).to(torch.uint8).cuda()
    k, v = _pool(case, n_pages, g), _pool(case, n_pages, g)
    ks = vs = 1.0
    if case["kv"] == "fp8":
        ks = vs = 6.0 / 448.0   # randn stays below 6
        k, v = (k.float() / ks).to(_DT["fp8"]), (v.float() / vs).to(_DT["fp8"])
    q = torch.randn((indptr[-1], case["h_q"], case["d"]), generator=g, device="cuda", dtype=torch.bfloat16)
    s = dict(op="shared", case=case, q=q, k=k, v=v, k_scale=ks, v_scale=vs, kv_indptr=_i32(kv_indptr),
             kv_indices=_i32(indices), last=_i32(last), indptr=_i32(indptr), max_nodes=max(lens), max_kv=max(kv_lens),
             mask=mask if case["tree"] else None, mask_indptr=_i32(mask_indptr) if case["tree"] else None, plan=None)
    if own:   # the plan that a program keeps for all layers of a step
        s["plan"] = _va().verify_attn_plan_shared(
            kv_indptr, indptr, last, mask_indptr, [i * case["members"] for i in range(case["groups"] + 1)],
            [sp] * case["groups"], case["h_q"], case["h_kv"], case["d"], P,
            kv_dtype="fp8_e4m3" if case["kv"] == "fp8" else "bf16", kv_layout="nhd" if case["nhd"] else "hnd")
    return s


def _prepare_keep(case, g, r):
    lens, P = _lens(dict(case, ragged=case["batch"] > 1), case["batch"]), case["page"]
    # the prefix before the drafts stays where it is: only its last pages are listed
    pre = [random.Random(case["shape_seed"] + b).randrange(2 * P) for b in range(case["batch"])]
    kv_lens = [a + n for a, n in zip(pre, lens)]
    need = [-(-k // P) for k in kv_lens]
    n_pages = sum(need) + 3
    ids = list(range(n_pages))
    r.shuffle(ids)
    parents = _tree(lens, True, r)
    acc, path = _paths(lens, parents, r)
    k, v = _pool(case, n_pages, g, case["layers"]), _pool(case, n_pages, g, case["layers"])
    if case["kv"] == "fp8":
        k, v = k.to(_DT["fp8"]), v.to(_DT["fp8"])
    return dict(op="keep", case=case, k=k, v=v, acc=_i32(acc), path=_i32(path), indptr=_i32(_indptr(lens)),
                kv_indptr=_i32(_indptr(need)), kv_indices=_i32(ids[:sum(need)]),
                last=_i32([(n - 1) % P + 1 for n in kv_lens]), max_nodes=max(lens),
                kv_len=torch.empty(case["batch"], dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------------ one pass

def run(s):
    return {"sample": _run_sample, "shared": _run_shared, "keep": _run_keep}[s["op"]](s)


def _run_sample(s):
    if own:
        acc, path, bonus, logp = _va().verify_accept_sample(
            s["logits"], s["indptr"], s["toks"], s["parents"], s["u"], s["noise"], temperature=s["temps"],
            draft_probs=s["probs"], want_logprobs=True)
        return dict(accept_len=acc, path=path, bonus=bonus, logp=logp)
    B, (total, V) = s["noise"].shape[0], s["logits"].shape
    dev = s["logits"].device
    indptr, toks = s["indptr"].long(), s["toks"].long()
    node = torch.arange(total, device=dev)
    req = torch.searchsorted(indptr, node, right=True) - 1
    first = indptr[:-1]
    par = torch.where(s["parents"] < 0, node, first[req] + s["parents"])
    child = s["parents"] >= 0
    # the target's probabilities
    x = s["logits"].float()
    greedy = torch.zeros(B, dtype=torch.bool, device=dev)
    if s["temps"] is not None:
        greedy = s["temps"] == 0
        t = torch.where(greedy, torch.ones_like(s["temps"]), s["temps"])
        x = x - x.max(1, keepdim=True).values
        x = x / t[req][:, None]
    x = x - x.max(1, keepdim=True).values
    e = torch.exp(x)
    z = e.sum(1, dtype=torch.float64)
    p = e / z.float()[:, None]
    if s["temps"] is not None:
        col = torch.arange(V, device=dev)
        am = torch.where(x == 0, col, V).min(1).values       # the first of equal maxima
        p = torch.where(greedy[req][:, None], (col == am[:, None]).float(), p)
    # siblings in index order; (A, B) of each parent as its children are rejected
    sib = (par[:, None] == par[None, :]) & child[:, None] & child[None, :]
    rank = (sib & (node[None, :] < node[:, None])).sum(1)
    pt = torch.exp(x[par, toks].double()) / z[par]
    u = s["u"].double()
    a = torch.zeros(total, dtype=torch.float64, device=dev)
    b = torch.ones(total, dtype=torch.float64, device=dev)
    ok = torch.zeros(total, dtype=torch.bool, device=dev)
    q = None if s["probs"] is None else s["probs"].float()
    if q is None:
        same = sib & (toks[:, None] == toks[None, :]) & (node[None, :] < node[:, None])
        pt = torch.where(same.any(1), torch.zeros_like(pt), pt)   # an equal sibling was rejected before
        gone = torch.where(sib & (node[None, :] < node[:, None]), pt[None, :], torch.zeros_like(pt)[None, :]).sum(1)
        ok = child & (u * (1 - gone) < pt)
    else:
        qt = q[par, toks].double()
        for k in range(int(rank.max()) + 1):
            i = node[child & (rank == k)]
            v = par[i]
            ok[i] = u[i] * b[v] * qt[i] < pt[i] - a[v] * qt[i]
            a[v] += b[v]
            b[v] = (p[v] - a[v].float()[:, None] * q[v]).clamp(min=0).sum(1, dtype=torch.float64)
    # at temperature 0 a child is accepted where its token is the argmax
    if s["temps"] is not None:
        ok = torch.where(greedy[req], child & (toks == am[par]), ok)
    # the first accepted child of each node; then down from the roots
    nxt = torch.full((total,), total, device=dev).scatter_reduce(0, par[ok], node[ok], "amin")
    path = torch.full((total + 1,), -1, dtype=torch.int32, device=dev)
    logp = torch.zeros(total + 1, dtype=torch.float64, device=dev)
    cur, acc = first.clone(), torch.ones(B, dtype=torch.int32, device=dev)
    path[first] = 0
    for k in range(1, s["max_nodes"]):
        to = nxt[cur]
        go = (to < total) & (acc == k)
        to = torch.where(go, to, cur)
        slot = torch.where(go, first + k, total)
        path[slot] = (to - first).to(torch.int32)
        raw = x[cur, toks[to]].double() - torch.log(z[cur])
        logp[torch.where(go, first + k - 1, total)] = torch.where(greedy, torch.zeros_like(raw), raw)
        acc += go.to(torch.int32)
        cur = to
    # the bonus token: a race of exponentials over what is left of the last row
    w = p[cur]
    if q is None:
        out = child & (cur[req] == par)
        left = w.clone()
        left[req[out], toks[out]] = 0
    else:
        left = (w - a[cur].float()[:, None] * q[cur]).clamp(min=0)
    left = torch.where(((left > 0).any(1) & ~greedy)[:, None], left, w)
    key = torch.where(left > 0, left / s["noise"], -1.0)
    col = torch.arange(V, device=dev)
    bonus = torch.where(key == key.max(1, keepdim=True).values, col, V).min(1).values
    raw = x[cur, bonus].double() - torch.log(z[cur])
    logp[first + acc - 1] = torch.where(greedy, torch.zeros_like(raw), raw)
    return dict(accept_len=acc, path=path[:total], bonus=bonus.to(torch.int32), logp=logp[:total].float())


def _gather(cache, pages, slots, nhd):
    """[..., h, d] rows of a paged cache at (page, slot), in fp32."""
    raw = cache.view(torch.uint8) if cache.element_size() == 1 else cache
    rows = raw[pages, slots] if nhd else raw[pages, :, slots]
    return (rows.view(cache.dtype) if cache.element_size() == 1 else rows).float()


def _run_shared(s):
    if own:
        out, lse = _va().verify_attn_run(
            s["q"], s["k"], s["v"], s["kv_indptr"], s["kv_indices"], s["last"], s["indptr"], s["mask"],
            s["mask_indptr"], s["plan"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return dict(out=out, lse=lse)
    c = s["case"]
    P, h, G, d, L, N = c["page"], c["h_kv"], c["h_q"] // c["h_kv"], c["d"], s["max_nodes"], s["max_kv"]
    dev = s["q"].device
    indptr, kvp = s["indptr"].long(), s["kv_indptr"].long()
    n, np_ = indptr[1:] - indptr[:-1], kvp[1:] - kvp[:-1]
    kv_len = (np_ - 1) * P + s["last"]
    B = n.shape[0]
    pos = torch.arange(N, device=dev)
    live = pos < kv_len[:, None]
    page = s["kv_indices"][torch.where(live, kvp[:-1, None] + pos // P, 0)].long()
    slot = (pos % P).expand(B, N)
    k = _gather(s["k"], page, slot, c["nhd"])                     # [B, N, h, d]
    v = _gather(s["v"], page, slot, c["nhd"])
    t = torch.arange(L, device=dev)
    tok = torch.where(t < n[:, None], indptr[:-1, None] + t, 0)   # [B, L]
    q = s["q"][tok].float().view(B, L, h, G, d).permute(0, 2, 1, 3, 4).reshape(B, h, L * G, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * (s["k_scale"] / math.sqrt(d))
    draft = pos - (kv_len - n)[:, None]                           # [B, N]: < 0 in the prefix
    if s["mask"] is None:
        vis = draft[:, None] <= t[:, None]
    else:
        col = torch.minimum(draft.clamp(min=0), (n - 1)[:, None])
        bit = s["mask_indptr"][:-1].long()[:, None, None] + torch.minimum(t, (n - 1)[:, None])[:, :, None] * n[:, None, None]
        bit = bit + col[:, None]
        vis = (draft[:, None] < 0) | ((s["mask"][bit >> 3] >> (bit & 7)) & 1).bool()
    vis = vis & live[:, None]                                     # [B, L, N]
    vis = vis[:, None, :, None].expand(B, 1, L, G, N).reshape(B, 1, L * G, N)
    x = x.masked_fill(~vis, -math.inf)
    m = x.max(-1, keepdim=True).values
    e = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    z = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v.permute(0, 2, 1, 3)) * s["v_scale"] / torch.where(z > 0, z, torch.ones_like(z))
    lse = (m + torch.log(z)).squeeze(-1)
    o = o.view(B, h, L, G, d).permute(0, 2, 1, 3, 4).reshape(B, L, h * G, d)
    lse = lse.view(B, h, L, G).permute(0, 2, 1, 3).reshape(B, L, h * G)
    rows = t < n[:, None]
    return dict(out=o[rows].to(torch.bfloat16), lse=lse[rows])


def _run_keep(s):
    c = s["case"]
    if own:
        _va().paged_kv_compact(s["acc"], s["path"], s["indptr"], s["kv_indptr"], s["kv_indices"], s["last"], s["k"],
                               s["v"], kv_layout="nhd" if c["nhd"] else "hnd", kv_len_out=s["kv_len"])
        return dict(k=s["k"], v=s["v"], kv_len=s["kv_len"])
    P, dev = c["page"], s["k"].device
    indptr, kvp = s["indptr"].long(), s["kv_indptr"].long()
    pre = (kvp[1:] - kvp[:-1] - 1) * P + s["last"] - (indptr[1:] - indptr[:-1])
    k = torch.arange(s["max_nodes"], device=dev)
    on = k < s["acc"][:, None]
    src = pre[:, None] + s["path"][torch.where(on, indptr[:-1, None] + k, 0)]
    dst = pre[:, None] + k
    on = on & (src != dst)
    base = kvp[:-1, None].expand_as(on)[on]
    src, dst = src[on], dst[on]
    sp, dp = s["kv_indices"][base + src // P].long(), s["kv_indices"][base + dst // P].long()
    for cache in (s["k"], s["v"]):
        x = cache.view(torch.uint8) if cache.element_size() == 1 else cache
        if c["nhd"]:
            x[:, dp, dst % P] = x[:, sp, src % P]
        else:
            x[:, dp, :, dst % P] = x[:, sp, :, src % P]
    s["kv_len"].copy_(pre + s["acc"])
    return dict(k=s["k"], v=s["v"], kv_len=s["kv_len"])


# ------------------------------------------------------------- what it needs

def work(case):
    if case["op"] == "sample":
        lens, V = _lens(case, case["batch"]), case["vocab"]
        es = {"bf16": 2, "f32": 4}
        # Rows that no accepted node leads to cannot change the answer, so they
        # need not be read: a request needs one row of logits for each node it
        # accepts.  A chain drafted by the inputs' draft model accepts about
        # three drafts in four; a tree's best branch about two nodes.
        rows = sum(min(1 + 2, n) if case["tree"] else (1 - 0.75 ** n) / 0.25 for n in lens)
        q = 0 if case["draft"] == "none" else es[case["draft"]] * V
        return {"bytes": rows * V * es[case["logits"]] + len(lens) * (q + 4 * V) + 24 * sum(lens),
                "flops": 4 * rows * V + 4 * len(lens) * V}
    if case["op"] == "shared":
        B = case["groups"] * case["members"]
        lens, mid = _lens(case, B), _own_lens(case, B)
        es = 1 if case["kv"] == "fp8" else 2
        keys = case["groups"] * case["shared"] + sum(a + n for a, n in zip(mid, lens))
        seen = sum(n * (case["shared"] + a) + n * (n + 1) / 2 for a, n in zip(mid, lens))
        return {"bytes": keys * case["h_kv"] * case["d"] * 2 * es + sum(lens) * case["h_q"] * (4 * case["d"] + 4),
                "flops": 4.0 * case["d"] * case["h_q"] * seen}
    lens = _lens(dict(case, ragged=case["batch"] > 1), case["batch"])
    # a drawn node of a random tree of n nodes lies about ln n below the root,
    # and all of its path but the root (and a node 1) has to move
    rows = sum(max(0.0, math.log(n) - 0.5) for n in lens)
    row = case["h_kv"] * case["d"] * (1 if case["kv"] == "fp8" else 2)
    return {"bytes": 4 * rows * row * case["layers"] + 16 * len(lens) + 4 * sum(lens), "flops": 0}


# ------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"sample": _exact_sample, "shared": _exact_shared, "keep": _exact_keep}[case["op"]](s)


def _exact_sample(s):
    """The walk as it is defined, request by request, residual by residual."""
    B, total = s["noise"].shape[0], s["logits"].shape[0]
    indptr, toks, parents = s["indptr"].tolist(), s["toks"].tolist(), s["parents"].tolist()
    u = s["u"].tolist()
    accept, bonus = [0] * B, [-1] * B
    path, logp = [-1] * total, [0.0] * total
    for b in range(B):
        o, n = indptr[b], indptr[b + 1] - indptr[b]
        t = 1.0 if s["temps"] is None else float(s["temps"][b])
        v, k = 0, 0
        while True:
            path[o + k] = v
            row = s["logits"][o + v].double()
            if t == 0:
                lp = torch.full_like(row, -math.inf)
                lp[(row == row.max()).nonzero()[0, 0]] = 0
            else:
                lp = torch.log_softmax(row / t, 0)
            p = torch.exp(lp)
            left, to = p.clone(), -1
            for c in [i for i in range(v + 1, n) if parents[o + i] == v]:
                x = toks[o + c]
                if t == 0:
                    if float(p[x]) > 0:
                        to = c
                        break
                    continue
                q = None if s["probs"] is None else s["probs"][o + v].double()
                if u[o + c] * (1.0 if q is None else float(q[x])) < float(left[x]):
                    to = c
                    break
                nxt = left.clone()
                if q is None:
                    nxt[x] = 0
                else:
                    nxt = (left - q).clamp(min=0)
                mass = nxt.sum()
                left = nxt / mass if mass > 0 else nxt
            if to < 0:
                left = left if bool((left > 0).any()) else p
                bonus[b] = int((left / s["noise"][b].double()).argmax())
                logp[o + k] = float(lp[bonus[b]])
                accept[b] = k + 1
                break
            logp[o + k] = float(lp[toks[o + to]])
            v, k = to, k + 1
    i = dict(dtype=torch.int32, device="cuda")
    return dict(accept_len=torch.tensor(accept, **i), path=torch.tensor(path, **i), bonus=torch.tensor(bonus, **i),
                logp=torch.tensor(logp, dtype=torch.float64, device="cuda"))


def _exact_shared(s):
    """Dense attention of each request over its own list of keys."""
    c = s["case"]
    P, h, d = c["page"], c["h_kv"], c["d"]
    G = c["h_q"] // h
    indptr, kvp, last = s["indptr"].tolist(), s["kv_indptr"].tolist(), s["last"].tolist()
    outs, lses = [], []
    for b in range(len(last)):
        n = indptr[b + 1] - indptr[b]
        pages = s["kv_indices"][kvp[b]:kvp[b + 1]].long()
        kv_len = (len(pages) - 1) * P + last[b]
        kv = []
        for cache, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
            x = cache.view(torch.uint8)[pages].view(cache.dtype) if cache.element_size() == 1 else cache[pages]
            x = x.transpose(1, 2) if not c["nhd"] else x          # [pages, P, h, d]
            kv.append(x.reshape(-1, h, d)[:kv_len].double() * scale)
        vis = torch.ones((n, kv_len), dtype=torch.bool, device="cuda")
        if s["mask"] is None:
            vis[:, kv_len - n:] = torch.ones((n, n), device="cuda").tril().bool()
        else:
            m0 = int(s["mask_indptr"][b])
            bits = torch.arange(m0, m0 + n * n, device="cuda")
            vis[:, kv_len - n:] = ((s["mask"].int()[bits // 8] >> (bits % 8)) % 2).view(n, n).bool()
        q = s["q"][indptr[b]:indptr[b + 1]].double().view(n, h, G, d)
        x = torch.einsum("nhgd,khd->nhgk", q, kv[0]) / math.sqrt(d)
        x = x.masked_fill(~vis[:, None, None], -math.inf)
        lse = torch.logsumexp(x, -1)
        outs.append(torch.einsum("nhgk,khd->nhgd", torch.exp(x - lse[..., None]), kv[1]).reshape(n, h * G, d))
        lses.append(lse.reshape(n, h * G))
    return dict(out=torch.cat(outs), lse=torch.cat(lses))


def _exact_keep(s):
    """Slot after slot, front to back."""
    c = s["case"]
    P = c["page"]
    indptr, kvp, last = s["indptr"].tolist(), s["kv_indptr"].tolist(), s["last"].tolist()
    acc, path, ids = s["acc"].tolist(), s["path"].tolist(), s["kv_indices"].tolist()
    kv_len = []
    for b in range(len(acc)):
        pre = (kvp[b + 1] - kvp[b] - 1) * P + last[b] - (indptr[b + 1] - indptr[b])
        kv_len.append(pre + acc[b])
        for k in range(acc[b]):
            a, z = pre + path[indptr[b] + k], pre + k
            if a == z:
                continue
            for cache in (s["k"], s["v"]):
                x = cache.view(torch.uint8) if cache.element_size() == 1 else cache
                x = x if c["nhd"] else x.transpose(2, 3)
                x[:, ids[kvp[b] + z // P], z % P] = x[:, ids[kvp[b] + a // P], a % P].clone()
    # what is held in 8 bits as the values it stands for
    return dict(k=s["k"].float(), v=s["v"].float(), kv_len=torch.tensor(kv_len, dtype=torch.int32, device="cuda"))
