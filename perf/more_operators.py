"""Cases of the operators around a cache that is kept within a budget: the norm
and the rotation of queries and keys with their append, the attention weight
that every cached key has received, and the eviction of the keys that received
least.

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
    """Norm, rotation and append of a step's queries, keys and values.
    prep_one: one token of one stream (plain decode); latency is all.
    prep_chains: a serving batch of ragged chains, quantised into an fp8 cache.
    prep_odd: head_dim 64, a value width of its own, an odd number of heads per
      KV head, half of each head rotated in pairs of neighbours, far positions.
    prep_prompt: the prompts of the varlen prefill.

    Attention weight per cached key.
    weigh_one: after one 17-node tree step, the accepted path's weights.
    weigh_chains: the CodeLLaMA-34B-shaped batch, chains over long prefixes.
    weigh_trees: the wide trees over an fp8 cache (NHD), every node counted.
    weigh_odd: head_dim 64, pages of one token, 7 query heads per KV head.
    weigh_prompt: every query of the varlen prefill's prompts.

    Eviction.
    evict_one: one request, one layer, a cache of 4,113 keys to half.
    evict_layers: a serving batch, 16 layers at once, to half of the keys.
    evict_long: two long contexts over an fp8 cache (NHD), to a quarter.
    """
    return [
        dict(name="prep_one", op="prep", batch=1, nodes=1, ragged=False, far=4096, h_q=32, h_kv=8, d=128, dv=128,
             page=16, kv="bf16", nhd=False, fused=True, weight="bf16", offset=0.0, rot=128, inter=False, shape_seed=1),
        dict(name="prep_chains", op="prep", batch=64, nodes=8, ragged=True, far=8192, h_q=64, h_kv=8, d=128, dv=128,
             page=16, kv="fp8", nhd=False, fused=True, weight="bf16", offset=0.0, rot=128, inter=False, shape_seed=2),
        dict(name="prep_odd", op="prep", batch=9, nodes=33, ragged=True, far=900000, h_q=14, h_kv=2, d=64, dv=128,
             page=8, kv="bf16", nhd=True, fused=False, weight="f32", offset=1.0, rot=32, inter=True, shape_seed=3),
        dict(name="prep_prompt", op="prep", batch=10, nodes=1024, ragged=False, far=0, h_q=64, h_kv=8, d=128, dv=128,
             page=16, kv="bf16", nhd=False, fused=True, weight="bf16", offset=0.0, rot=128, inter=False, shape_seed=4),
        dict(name="weigh_one", op="weigh", batch=1, nodes=17, ragged=False, tree=True, path=True, prefix=4096,
             h_q=32, h_kv=8, d=128, page=16, kv="bf16", nhd=False, decay=1.0, shape_seed=5),
        dict(name="weigh_chains", op="weigh", batch=64, nodes=8, ragged=True, tree=False, path=False, prefix=8192,
             h_q=64, h_kv=8, d=128, page=16, kv="bf16", nhd=False, decay=0.98, shape_seed=6),
        dict(name="weigh_trees", op="weigh", batch=8, nodes=64, ragged=False, tree=True, path=False, prefix=32768,
             h_q=32, h_kv=8, d=128, page=32, kv="fp8", nhd=True, decay=1.0, shape_seed=7),
        dict(name="weigh_odd", op="weigh", batch=5, nodes=19, ragged=True, tree=True, path=False, prefix=1500,
             h_q=14, h_kv=2, d=64, page=1, kv="bf16", nhd=False, decay=1.0, shape_seed=8),
        dict(name="weigh_prompt", op="weigh", batch=10, nodes=1024, ragged=False, tree=False, path=False, prefix=0,
             h_q=64, h_kv=8, d=128, page=16, kv="bf16", nhd=False, decay=0.0, shape_seed=9),
        dict(name="evict_one", op="evict", batch=1, layers=1, keys=4113, ragged=False, share=0.5, sinks=4, recent=64,
             h_kv=8, d=128, page=16, kv="bf16", nhd=False, shape_seed=10),
        dict(name="evict_layers", op="evict", batch=8, layers=16, keys=8192, ragged=True, share=0.5, sinks=4,
             recent=256, h_kv=8, d=128, page=16, kv="bf16", nhd=False, shape_seed=11),
        dict(name="evict_long", op="evict", batch=2, layers=4, keys=131072, ragged=False, share=0.25, sinks=4,
             recent=1024, h_kv=8, d=128, page=32, kv="fp8", nhd=True, shape_seed=12),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: any operator, sizes over the listed cases' ranges."""
    op = rng.choice(["prep", "weigh", "evict"])
    c = dict(op=op, ragged=rng.random() < 0.6, h_kv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128, 128]),
             page=rng.choice([1, 8, 16, 32, 64]), kv=rng.choice(["bf16", "fp8"]), nhd=rng.random() < 0.5,
             shape_seed=rng.randrange(1 << 20))
    group = rng.choice([1, 3, 4, 7, 8])
    if op == "prep":
        batch = _log(rng, 1, 64)
        return dict(c, batch=batch, nodes=_log(rng, 1, 8192 // batch), far=_log(rng, 1, 1 << 20), h_q=c["h_kv"] * group,
                    dv=rng.choice([c["d"], c["d"], 64, 128]), fused=rng.random() < 0.5,
                    weight=rng.choice(["none", "bf16", "f32"]), offset=rng.choice([0.0, 1.0]),
                    rot=rng.choice([c["d"], c["d"], c["d"] // 2, c["d"] // 4]), inter=rng.random() < 0.3)
    if op == "weigh":
        batch = _log(rng, 1, 64)
        nodes = _log(rng, 1, 256 // batch)
        prefix = _log(rng, 16, min(32768, (1 << 18) // batch))
        if rng.random() < 0.25:   # whole prompts
            batch, nodes, prefix = _log(rng, 1, 10), _log(rng, 1, 1024), 0
        tree = rng.random() < 0.5 and nodes <= 64
        return dict(c, batch=batch, nodes=nodes, tree=tree, path=rng.random() < 0.4, prefix=prefix,
                    h_q=c["h_kv"] * group, decay=rng.choice([0.0, 0.9, 1.0]))
    batch, layers = _log(rng, 1, 16), _log(rng, 1, 16)
    return dict(c, batch=batch, layers=layers, keys=_log(rng, 16, min(131072, (1 << 20) // (batch * layers))),
                share=rng.choice([0.1, 0.25, 0.5, 0.9]), sinks=rng.choice([0, 1, 4]), recent=rng.choice([0, 16, 100]))


def _lens(case):
    """Query tokens of each request: the case's own shape, the same for every seed."""
    r = random.Random(case["shape_seed"])
    return [r.randint(1, case["nodes"]) if case["ragged"] else case["nodes"] for _ in range(case["batch"])]


def _prefixes(case):
    """Keys of each request before its new tokens."""
    r = random.Random(case["shape_seed"] + 77)
    if case["op"] == "prep":   # the pages before the last ones are not listed: the operator does not come near them
        return [r.randrange(2 * case["page"]) for _ in range(case["batch"])]
    return [r.randint(case["prefix"] // 16, case["prefix"]) if case["ragged"] else case["prefix"]
            for _ in range(case["batch"])]


def _keys(case):
    """Keys of each request of an eviction, and how many of them are kept."""
    r = random.Random(case["shape_seed"])
    n = [r.randint(max(1, case["keys"] // 4), case["keys"]) if case["ragged"] else case["keys"]
         for _ in range(case["batch"])]
    return n, [max(1, int(x * case["share"])) for x in n]


def _indptr(lens):
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return out


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pages(case, kv_lens, r):
    """Page tables over a shuffled pool: (pages of the pool, the device tables)."""
    P = case["page"]
    need = [-(-k // P) for k in kv_lens]
    n_pages = sum(need) + max(1, sum(need) // 16)
    ids = list(range(n_pages))
    r.shuffle(ids)
    return n_pages, dict(kv_indptr=_i32(_indptr(need)), kv_indices=_i32(ids[:sum(need)]),
                         last=_i32([(k - 1) % P + 1 if k else 0 for k in kv_lens]), n_keys=_i32(kv_lens),
                         max_kv=max(kv_lens))


def _pool(case, pages, g, width, layers=()):
    """K or V pages; every slot holds something, as a pool in use does."""
    mid = (case["page"], case["h_kv"]) if case["nhd"] else (case["h_kv"], case["page"])
    x = torch.randn(layers + (pages,) + mid + (width,), generator=g, device="cuda", dtype=torch.bfloat16)
    return x if case["kv"] == "bf16" else (x * 64).to(_DT["fp8"])


def _weights(case, pages, g, layers=()):
    """Attention weight so far of the key in every slot: a few keys have received most of it."""
    mid = (case["page"], case["h_kv"]) if case["nhd"] else (case["h_kv"], case["page"])
    return torch.exp(2 * torch.randn(layers + (pages,) + mid, generator=g, device="cuda"))


# ---------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    return {"prep": _prepare_prep, "weigh": _prepare_weigh, "evict": _prepare_evict}[case["op"]](case, g, r)


def _prepare_prep(case, g, r):
    lens, pre = _lens(case), _prefixes(case)
    total, hq, h, d, dv = sum(lens), case["h_q"], case["h_kv"], case["d"], case["dv"]
    n_pages, tables = _pages(case, [a + n for a, n in zip(pre, lens)], r)
    rand = dict(generator=g, device="cuda", dtype=torch.bfloat16)
    if case["fused"]:   # slices of one projection's rows
        rows = torch.randn((total, hq * d + h * d + h * dv), **rand) * 1.5
        q, k, v = rows.split([hq * d, h * d, h * dv], 1)
        q, k, v = q.view(total, hq, d), k.view(total, h, d), v.view(total, h, dv)
    else:
        q, k, v = (torch.randn((total, a, b), **rand) * 1.5 for a, b in ((hq, d), (h, d), (h, dv)))
    qw = kw = None
    if case["weight"] != "none":
        qw, kw = ((torch.rand(d, generator=g, device="cuda") + 0.5 - case["offset"]).to(_DT[case["weight"]])
                  for _ in range(2))
    start = [r.randint(0, case["far"]) if case["far"] else 0 for _ in lens]
    return dict(op="prep", case=case, q=q, k=k, v=v, qw=qw, kw=kw, indptr=_i32(_indptr(lens)),
                positions=_i32([s + i for s, n in zip(start, lens) for i in range(n)]), theta=5e5, eps=1e-6,
                k_cache=_pool(case, n_pages, g, d), v_cache=_pool(case, n_pages, g, dv), k_scale=0.0171,
                v_scale=0.0163, **tables)


def _tree_masks(lens, r, tree):
    """Bit-packed ancestor masks of random trees (or chains), their bit offsets, and a root path of each."""
    bits, indptr, acc, path = [], [0], [], []
    for n in lens:
        parent = [-1] + [r.randrange(i) if tree else i - 1 for i in range(1, n)]
        rows = []
        for i in range(n):
            row = list(rows[parent[i]]) if i else [0] * n
            row[i] = 1
            rows.append(row)
        if tree:
            bits += [x for row in rows for x in row]
        indptr.append(indptr[-1] + n * n)
        last = r.randrange(n)
        up = [j for j in range(n) if rows[last][j]] if tree else list(range(last + 1))
        acc.append(len(up))
        path += up + [-1] * (n - len(up))
    if not tree:
        return None, None, acc, path
    bits += [0] * (-len(bits) % 8)
    w = torch.tensor(bits, dtype=torch.int32).view(-1, 8) << torch.arange(8, dtype=torch.int32)
    return w.sum(1).to(torch.uint8).cuda(), _i32(indptr), acc, path


def _prepare_weigh(case, g, r):
    lens, pre = _lens(case), _prefixes(case)
    total, hq, h, d = sum(lens), case["h_q"], case["h_kv"], case["d"]
    n_pages, tables = _pages(case, [a + n for a, n in zip(pre, lens)], r)
    mask, mask_indptr, acc, path = _tree_masks(lens, r, case["tree"])
    k = _pool(case, n_pages, g, d)
    s = dict(op="weigh", case=case, k=k, k_scale=1.0 if case["kv"] == "bf16" else 1 / 64,
             q=torch.randn((total, hq, d), generator=g, device="cuda", dtype=torch.bfloat16),
             w=_weights(case, n_pages, g), indptr=_i32(_indptr(lens)), max_nodes=max(lens), mask=mask,
             mask_indptr=mask_indptr, acc=_i32(acc) if case["path"] else None,
             path=_i32(path) if case["path"] else None, **tables)
    x, _ = _logits(s)   # the attention's own log-sum-exp, which its call has returned
    s["lse"] = torch.logsumexp(x, -1)[_new_rows(s)]
    return s


def _prepare_evict(case, g, r):
    n, keep = _keys(case)
    n_pages, tables = _pages(case, n, r)
    layers = (case["layers"],)
    return dict(op="evict", case=case, k=_pool(case, n_pages, g, case["d"], layers),
                v=_pool(case, n_pages, g, case["d"], layers), w=_weights(case, n_pages, g, layers), keep=_i32(keep),
                kv_len=torch.empty(case["batch"], dtype=torch.int32, device="cuda"), **tables)


# ------------------------------------------------------------------ one pass

def run(s):
    return {"prep": _run_prep, "weigh": _run_weigh, "evict": _run_evict}[s["op"]](s)


def _raw(x):
    """fp8 as bytes: torch indexes those."""
    return x.view(torch.uint8) if x.element_size() == 1 else x


def _normed(x, w, offset, eps):
    x = x.float()
    if w is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * (w.float() + offset)


def _rotated(x, cos, sin, inter):
    """The first 2 * cos.shape[-1] elements of each head rotated, pair by pair."""
    n = cos.shape[-1]
    a, b = (x[..., :2 * n:2], x[..., 1:2 * n:2]) if inter else (x[..., :n], x[..., n:2 * n])
    y, z = a * cos - b * sin, a * sin + b * cos
    y = torch.stack((y, z), -1).flatten(-2) if inter else torch.cat((y, z), -1)
    return torch.cat((y, x[..., 2 * n:]), -1)


def _run_prep(s):
    c = s["case"]
    if own:
        q = _va().paged_qkv_append(
            s["q"], s["k"], s["v"], s["indptr"], s["kv_indptr"], s["kv_indices"], s["last"], s["k_cache"],
            s["v_cache"], q_weight=s["qw"], k_weight=s["kw"], weight_offset=c["offset"], eps=s["eps"],
            positions=s["positions"], rope_theta=s["theta"], rotary_dim=c["rot"], interleaved=c["inter"],
            kv_layout="nhd" if c["nhd"] else "hnd", **(dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
                                                       if c["kv"] == "fp8" else {}))
        return dict(q=q, k=s["k_cache"], v=s["v_cache"])
    P, dev, total = c["page"], s["q"].device, s["q"].shape[0]
    i = torch.arange(0, c["rot"], 2, device=dev, dtype=torch.float64)
    angle = s["positions"].double()[:, None] * torch.pow(s["theta"], -i / c["rot"])
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q = _rotated(_normed(s["q"], s["qw"], c["offset"], s["eps"]), cos, sin, c["inter"])
    k = _rotated(_normed(s["k"], s["kw"], c["offset"], s["eps"]), cos, sin, c["inter"])
    v = s["v"].float()
    if c["kv"] == "fp8":
        k, v = (k / s["k_scale"]).clamp(-448, 448), (v / s["v_scale"]).clamp(-448, 448)
    t = torch.arange(total, device=dev)
    indptr = s["indptr"].long()
    req = torch.searchsorted(indptr, t, right=True) - 1
    pos = s["n_keys"].long()[req] - indptr[req + 1] + t
    page = s["kv_indices"][s["kv_indptr"].long()[req] + pos // P].long()
    for cache, x in ((s["k_cache"], k), (s["v_cache"], v)):
        x = _raw(x.to(_DT[c["kv"]]))
        if c["nhd"]:
            _raw(cache)[page, pos % P] = x
        else:
            _raw(cache)[page, :, pos % P] = x
    return dict(q=q.to(torch.bfloat16), k=s["k_cache"], v=s["v_cache"])


def _slots(s):
    """(page, slot, whether there is a key) of every position of every request: [B, N]."""
    P = s["case"]["page"]
    pos = torch.arange(s["max_kv"], device="cuda")
    live = pos < s["n_keys"][:, None]
    page = s["kv_indices"][torch.where(live, s["kv_indptr"][:-1].long()[:, None] + pos // P, 0)].long()
    return page, (pos % P).expand_as(page), live


def _new_rows(s):
    """Which of the padded [B, L] rows are query tokens."""
    n = s["indptr"][1:] - s["indptr"][:-1]
    return torch.arange(s["max_nodes"], device="cuda") < n[:, None]


def _logits(s):
    """Scaled logits [B, L, h_q, N], -inf where a key is not seen, and what is seen [B, L, N]."""
    c = s["case"]
    h, G, d, L = c["h_kv"], c["h_q"] // c["h_kv"], c["d"], s["max_nodes"]
    indptr = s["indptr"].long()
    n, B = indptr[1:] - indptr[:-1], c["batch"]
    page, slot, live = _slots(s)
    k = _raw(s["k"])[page, slot] if c["nhd"] else _raw(s["k"])[page, :, slot]
    k = k.view(s["k"].dtype).float()
    rows = _new_rows(s)
    tok = torch.where(rows, indptr[:-1, None] + torch.arange(L, device="cuda"), 0)
    q = s["q"][tok].float().view(B, L, h, G, d).permute(0, 2, 1, 3, 4).reshape(B, h, L * G, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * (s["k_scale"] / math.sqrt(d))
    x = x.view(B, h, L, G, -1).permute(0, 2, 1, 3, 4)                        # [B, L, h, G, N]
    t = torch.arange(L, device="cuda")
    draft = torch.arange(s["max_kv"], device="cuda") - (s["n_keys"] - n)[:, None]
    if s["mask"] is None:
        vis = draft[:, None] <= t[:, None]
    else:
        top = (n - 1)[:, None]
        bit = torch.minimum(t, top)[:, :, None] * n[:, None, None] + torch.minimum(draft.clamp(min=0), top)[:, None]
        bit = bit + s["mask_indptr"][:-1].long()[:, None, None]
        vis = (draft[:, None] < 0) | ((s["mask"][bit >> 3] >> (bit & 7)) & 1).bool()
    vis = vis & live[:, None] & rows[:, :, None]
    return x.masked_fill(~vis[:, :, None, None], -math.inf).flatten(2, 3), vis


def _run_weigh(s):
    c = s["case"]
    if own:
        return _va().verify_attn_key_weights(
            s["q"], s["k"], s["kv_indptr"], s["kv_indices"], s["last"], s["indptr"], s["lse"], s["w"],
            mask=None if c["path"] else s["mask"], mask_indptr=None if c["path"] else s["mask_indptr"],
            accept_len=s["acc"], accepted_nodes=s["path"], k_scale=s["k_scale"], decay=c["decay"],
            kv_layout="nhd" if c["nhd"] else "hnd")
    h, L, B, N = c["h_kv"], s["max_nodes"], c["batch"], s["max_kv"]
    indptr = s["indptr"].long()
    n = indptr[1:] - indptr[:-1]
    x, _ = _logits(s)
    rows = _new_rows(s)
    tok = torch.where(rows, indptr[:-1, None] + torch.arange(L, device="cuda"), 0)
    e = torch.exp(x - s["lse"][tok][..., None])
    e = torch.where(x == -math.inf, torch.zeros_like(e), e)
    pre = s["n_keys"].long() - n
    pos = torch.arange(N, device="cuda")
    page, slot, live = _slots(s)
    if c["path"]:
        # only the accepted nodes' queries count, and key path[k] is weighed in slot k of the drafts
        path = torch.where(rows, s["path"][tok].long(), -1)                  # [B, L]
        on = (torch.arange(L, device="cuda") < s["acc"][:, None])
        counted = torch.zeros((B, L + 1), device="cuda").scatter_(1, torch.where(on, path, L), 1.0)[:, :L]
        e = e * counted[:, :, None, None]
        live = live & (pos < (pre + s["acc"])[:, None])
        j = (pos - pre[:, None]).clamp(min=0, max=L - 1)
        src = torch.where(pos < pre[:, None], pos, pre[:, None] + path.gather(1, j).clamp(min=0))
    else:
        src = pos.expand(B, N)
    got = e.sum(1).view(B, h, -1, N).sum(2).permute(0, 2, 1)                 # [B, N, h]
    got = got.gather(1, src[..., None].expand(B, N, h))
    old = s["w"][page, slot] if c["nhd"] else s["w"][page, :, slot]
    got = got + torch.where((pos < pre[:, None])[..., None], old * c["decay"], torch.zeros_like(old))
    page, slot = page[live], slot[live]
    if c["nhd"]:
        s["w"][page, slot] = got[live]
    else:
        s["w"][page, :, slot] = got[live]
    return s["w"]


def _run_evict(s):
    c = s["case"]
    if own:
        _va().paged_kv_evict(s["w"], s["keep"], s["kv_indptr"], s["kv_indices"], s["last"], s["k"], s["v"],
                             max_kv_len=s["max_kv"], sinks=c["sinks"], recent=c["recent"],
                             kv_layout="nhd" if c["nhd"] else "hnd", kv_len_out=s["kv_len"])
        return dict(k=s["k"], v=s["v"], w=s["w"], kv_len=s["kv_len"])
    n, B, h, N = s["n_keys"].long(), c["batch"], c["h_kv"], s["max_kv"]
    keep = torch.minimum(s["keep"].long(), n)
    page, slot, live = _slots(s)
    w = s["w"][:, page, slot] if c["nhd"] else s["w"][:, page, :, slot].permute(2, 0, 1, 3)   # [layers, B, N, h]
    w = w.transpose(2, 3)
    pos = torch.arange(N, device="cuda")
    sinks = keep.clamp(max=c["sinks"])
    recent = torch.minimum(keep - sinks, torch.full_like(keep, c["recent"]))
    held = (pos < sinks[:, None]) | ((pos >= (n - recent)[:, None]) & live)
    w = torch.where(held[:, None], math.inf, torch.where(live[:, None], w, -math.inf))
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices       # equal weights: the first position first
    on = torch.zeros(w.shape, dtype=torch.bool, device="cuda").scatter_(
        -1, order, (pos < keep[:, None])[:, None].expand(w.shape))
    to = on.cumsum(-1) - 1
    layer, b, head, frm = (on & (to != pos)).nonzero(as_tuple=True)
    to = to[layer, b, head, frm]
    sp, ss, dp, ds = page[b, frm], slot[b, frm], page[b, to], slot[b, to]
    for x in (_raw(s["k"]), _raw(s["v"]), s["w"]):
        if c["nhd"]:
            x[layer, dp, ds, head] = x[layer, sp, ss, head]
        else:
            x[layer, dp, head, ds] = x[layer, sp, head, ss]
    s["kv_len"].copy_(keep)
    return dict(k=s["k"], v=s["v"], w=s["w"], kv_len=s["kv_len"])


# ------------------------------------------------------------- what it needs

def work(case):
    es, h, d = 1 if case["kv"] == "fp8" else 2, case["h_kv"], case["d"]
    if case["op"] == "prep":
        n = sum(_lens(case))
        row = case["h_q"] * d * 4 + h * (d + case["dv"]) * (2 + es)
        return {"bytes": n * (row + 8), "flops": 10.0 * n * (case["h_q"] + h) * d}
    if case["op"] == "weigh":
        lens, pre = _lens(case), _prefixes(case)
        if case["path"]:   # a drawn node of a random tree lies about ln n below the root, of a chain about n / 2
            used = [min(n, 1 + math.log(n)) if case["tree"] else (n + 1) / 2 for n in lens]
        else:
            used = lens
        keys = sum(a + n for a, n in zip(pre, used))
        seen = sum(n * a + (n * (n + 1) / 2 if not case["tree"] or case["path"] else n * min(n, 1 + math.log(n)))
                   for a, n in zip(pre, used))
        old = 4 if case["decay"] else 0
        return {"bytes": keys * h * (d * es + 4) + sum(pre) * h * old + sum(used) * case["h_q"] * (2 * d + 4),
                "flops": 2.0 * d * case["h_q"] * seen}
    n, keep = _keys(case)
    # the sinks stay where they are, and so do the few keys before the first one that goes
    moved = sum(max(0, k - case["sinks"]) for k, x in zip(keep, n) if k < x)
    return {"bytes": case["layers"] * h * (4.0 * sum(n) + 2.0 * moved * (2 * d * es + 4)), "flops": 0}


# ------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"prep": _exact_prep, "weigh": _exact_weigh, "evict": _exact_evict}[case["op"]](s)


def _exact_prep(s):
    """Head by head: divided by its root mean square, then turned as complex numbers."""
    c = s["case"]
    half = c["rot"] // 2
    freq = torch.tensor([s["theta"] ** (-2.0 * i / c["rot"]) for i in range(half)], dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["positions"].double()[:, None] * freq)

    def head(x, w):
        x = x.double()
        if w is not None:
            ms = torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1]
            x = x / torch.sqrt(ms + s["eps"]) * (w.double() + c["offset"])
        part = x[..., :2 * half]
        z = torch.complex(part[..., 0::2], part[..., 1::2]) if c["inter"] else torch.complex(
            part[..., :half], part[..., half:])
        z = z * turn[:, None]
        done = torch.zeros_like(x)
        done[..., 2 * half:] = x[..., 2 * half:]
        if c["inter"]:
            done[..., 0:2 * half:2], done[..., 1:2 * half:2] = z.real, z.imag
        else:
            done[..., :half], done[..., half:2 * half] = z.real, z.imag
        return done

    q, k, v = head(s["q"], s["qw"]), head(s["k"], s["kw"]), s["v"].double()
    if c["kv"] == "fp8":
        k, v = (k / s["k_scale"]).clamp(-448, 448), (v / s["v_scale"]).clamp(-448, 448)
    out = dict(q=q)
    indptr, kvp = s["indptr"].tolist(), s["kv_indptr"].tolist()
    n_keys, ids = s["n_keys"].tolist(), s["kv_indices"].long()
    for name, x in (("k", k), ("v", v)):
        cache = s[name + "_cache"].double()
        flat = cache if c["nhd"] else cache.transpose(1, 2)                   # a view: [pages, P, h, width]
        for b in range(c["batch"]):
            pos = torch.arange(n_keys[b] - (indptr[b + 1] - indptr[b]), n_keys[b], device="cuda")
            flat[ids[kvp[b] + pos // c["page"]], pos % c["page"]] = x[indptr[b]:indptr[b + 1]]
        out[name] = cache
    return out


def _exact_weigh(s):
    """Request by request: exp(logit - lse) of every pair that the masks allow, added up over the queries."""
    c = s["case"]
    P, h, d = c["page"], c["h_kv"], c["d"]
    G = c["h_q"] // h
    indptr, kvp, n_keys = s["indptr"].tolist(), s["kv_indptr"].tolist(), s["n_keys"].tolist()
    out = s["w"].double()
    w = out if c["nhd"] else out.transpose(1, 2)                              # a view: [pages, P, h]
    for b in range(c["batch"]):
        o, n, m = indptr[b], indptr[b + 1] - indptr[b], n_keys[b]
        pos = torch.arange(m, device="cuda")
        page, slot = s["kv_indices"][kvp[b]:kvp[b + 1]].long()[pos // P], pos % P
        k = _raw(s["k"])[page, slot] if c["nhd"] else _raw(s["k"])[page, :, slot]          # [m, h, d]
        k = k.view(s["k"].dtype).double() * s["k_scale"]
        seen = torch.ones((n, m), dtype=torch.bool, device="cuda")
        if s["mask"] is None:
            seen[:, m - n:] = torch.ones((n, n), device="cuda").tril().bool()
        else:
            bits = torch.arange(int(s["mask_indptr"][b]), int(s["mask_indptr"][b + 1]), device="cuda")
            seen[:, m - n:] = ((s["mask"].int()[bits // 8] >> (bits % 8)) % 2).view(n, n).bool()
        nodes = list(range(n)) if s["acc"] is None else s["path"][o:o + int(s["acc"][b])].tolist()
        sums = torch.zeros((m, h), dtype=torch.float64, device="cuda")
        for a in range(0, len(nodes), 128):
            at = torch.tensor(nodes[a:a + 128], device="cuda")
            x = torch.einsum("nhgd,khd->nhgk", s["q"][o + at].double().view(-1, h, G, d), k) / math.sqrt(d)
            x = torch.exp(x - s["lse"][o + at].double().view(-1, h, G, 1))
            sums += torch.where(seen[at][:, None, None], x, 0.0).sum((0, 2)).T
        last = m - n + len(nodes)
        new = torch.cat((torch.arange(m - n, device="cuda"), m - n + torch.tensor(nodes, device="cuda")))
        before = w[page[:m - n], slot[:m - n]] * c["decay"] if c["decay"] else 0
        w[page[:last], slot[:last]] = sums[new]
        w[page[:m - n], slot[:m - n]] += before
    return out


def _exact_evict(s):
    """Request by request: every weight above the last one kept, then the first of its equals; moved one by one."""
    c = s["case"]
    P, h, Y = c["page"], c["h_kv"], c["layers"]
    kvp, n_keys, keep = s["kv_indptr"].tolist(), s["n_keys"].tolist(), s["keep"].tolist()
    pools = [_raw(s["k"]), _raw(s["v"]), s["w"]]
    kv_len = []
    for b in range(c["batch"]):
        n, left = n_keys[b], min(keep[b], n_keys[b])
        kv_len.append(left)
        if left == n:
            continue
        pos = torch.arange(n, device="cuda")
        page, slot = s["kv_indices"][kvp[b]:kvp[b + 1]].long()[pos // P], pos % P
        first = min(c["sinks"], left)
        tail = min(c["recent"], left - first)
        for layer in range(Y):
            for head in range(h):
                at = (page, slot, head) if c["nhd"] else (page, head, slot)
                w = s["w"][layer][at].double()
                on = (pos < first) | (pos >= n - tail)
                rest = left - first - tail
                if rest:
                    mid = w[first:n - tail]
                    edge = torch.kthvalue(mid, mid.numel() - rest + 1).values
                    more, same = mid > edge, mid == edge
                    on[first:n - tail] = more | (same & (same.cumsum(0) <= rest - more.sum()))
                rows = pos[on]
                to = pos[:left]
                for x in pools:
                    y = x[layer]
                    if c["nhd"]:
                        y[page[to], slot[to], head] = y[page[rows], slot[rows], head].clone()
                    else:
                        y[page[to], head, slot[to]] = y[page[rows], head, slot[rows]].clone()
    # what is held in 8 bits as the values it stands for
    return dict(k=s["k"].float(), v=s["v"].float(), w=s["w"].double(),
                kv_len=torch.tensor(kv_len, dtype=torch.int32, device="cuda"))
