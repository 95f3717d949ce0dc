"""GPU test of paged_kv_compact against a host copy of the whole pool: the
accepted rows at the front of their request's draft slots bit for bit, every
other slot as it was."""
import numpy as np
import pytest
import torch

from oracle.accept_sample import compact_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def va():
    import __graft_entry__
    __graft_entry__.build()
    import speculative_decoding_verify_gqa_gb300 as m
    return m


def _case(seed, lens, pre, acc, page, h_kv, d, dv=None, fp8=False, nhd=False, layers=None, spare=4):
    rng = np.random.default_rng(seed)
    need = [-(-(a + n) // page) for a, n in zip(pre, lens)]
    pages = sum(need) + spare
    ids = rng.permutation(pages)[:sum(need)].astype(np.int32)
    path = np.full(sum(lens), -1, np.int32)
    o = 0
    for n, a in zip(lens, acc):
        if a:
            path[o:o + a] = np.sort(np.concatenate([[0], 1 + rng.choice(n - 1, a - 1, replace=False)]) if a > 1 else [0])
        o += n
    mid = (page, h_kv) if nhd else (h_kv, page)
    shape = (() if layers is None else (layers,)) + (pages,) + mid
    bits = lambda w: rng.integers(0, 256, shape + (w * (1 if fp8 else 2),), dtype=np.uint8)  # noqa: E731
    ptr = lambda x: np.concatenate([[0], np.cumsum(x)]).astype(np.int32)  # noqa: E731
    return dict(k=bits(d), v=bits(dv or d), acc=np.array(acc, np.int32), path=path, qo=ptr(lens), kvp=ptr(need), ids=ids,
                last=np.array([(a + n - 1) % page + 1 if a + n else 0 for a, n in zip(pre, lens)], np.int32), page=page,
                fp8=fp8, nhd=nhd, layers=layers)


def _dev(c):
    dt = torch.float8_e4m3fn if c["fp8"] else torch.bfloat16
    t = {n: torch.from_numpy(c[n].copy()).cuda() for n in ("acc", "path", "qo", "kvp", "ids", "last")}
    t["k"], t["v"] = (torch.from_numpy(c[n].copy()).cuda().view(dt) for n in ("k", "v"))
    return t


def _expect(c):
    moves, new = compact_rows(c["qo"], c["kvp"], c["last"], c["page"], c["ids"], c["acc"], c["path"])
    out = []
    for n in ("k", "v"):
        x = c[n].copy()
        x5 = x if c["layers"] is not None else x[None]
        for (sp, ss), (dp, ds) in moves:
            if c["nhd"]:
                x5[:, dp, ds] = x5[:, sp, ss]
            else:
                x5[:, dp, :, ds] = x5[:, sp, :, ss]
        out.append(x)
    return out[0], out[1], new, len(moves)


def _run(va, c, t=None, **kw):
    t = t or _dev(c)
    kv_len = torch.full((len(c["acc"]),), -7, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    va.paged_kv_compact(t["acc"], t["path"], t["qo"], t["kvp"], t["ids"], t["last"], t["k"], t["v"],
                        kv_layout="nhd" if c["nhd"] else "hnd", kv_len_out=kv_len, status=status, **kw)
    torch.cuda.synchronize()
    return t["k"].view(torch.uint8).cpu().numpy(), t["v"].view(torch.uint8).cpu().numpy(), kv_len.cpu().numpy(), int(status)


CASES = {
    "tree_17": dict(lens=[17], pre=[300], acc=[5], page=16, h_kv=8, d=128),
    "batch": dict(lens=[8, 1, 5, 0, 12], pre=[10, 3, 0, 20, 33], acc=[4, 1, 5, 0, 2], page=16, h_kv=2, d=128),
    "all_accepted": dict(lens=[6, 9], pre=[2, 7], acc=[6, 9], page=8, h_kv=4, d=64),
    "none_accepted": dict(lens=[6, 9], pre=[2, 7], acc=[0, 0], page=8, h_kv=4, d=64),
    "page_1": dict(lens=[9, 4], pre=[2, 0], acc=[6, 3], page=1, h_kv=3, d=64, nhd=True),
    "fp8_nhd": dict(lens=[64, 40], pre=[31, 0], acc=[9, 20], page=32, h_kv=2, d=64, fp8=True, nhd=True),
    "layers": dict(lens=[9, 4, 7], pre=[5, 100, 0], acc=[6, 2, 3], page=4, h_kv=2, d=128, layers=5),
    "layers_fp8": dict(lens=[17], pre=[1], acc=[9], page=256, h_kv=1, d=128, fp8=True, layers=3),
    "value_width": dict(lens=[9, 4], pre=[5, 2], acc=[6, 2], page=16, h_kv=2, d=128, dv=64),
    "value_width_wider": dict(lens=[9, 4], pre=[5, 2], acc=[6, 2], page=16, h_kv=3, d=64, dv=128, fp8=True, nhd=True),
    "long_path": dict(lens=[700], pre=[9], acc=[400], page=16, h_kv=1, d=64),
}


@pytest.mark.parametrize("name", CASES)
def test_matches_host_copy(va, name):
    c = _case(7, **CASES[name])
    k, v, new, n = _expect(c)
    assert n > 0 or name in ("all_accepted", "none_accepted")
    got = _run(va, c)
    assert got[3] == 0
    assert np.array_equal(got[0], k) and np.array_equal(got[1], v) and np.array_equal(got[2], new)


def test_pools_side_by_side_in_one_tensor(va):
    c = _case(3, **CASES["layers"])
    k, v, new, _ = _expect(c)
    t = _dev(c)
    t["k"], t["v"] = torch.stack([t["k"], t["v"]])
    got = _run(va, c, t)
    assert got[3] == 0
    assert np.array_equal(got[0], k) and np.array_equal(got[1], v) and np.array_equal(got[2], new)
    with pytest.raises(RuntimeError):
        va.paged_kv_compact(t["acc"], t["path"], t["qo"], t["kvp"], t["ids"], t["last"], t["k"], t["k"])


def test_bad_paths_move_nothing(va):
    """A path that does not ascend, leaves the request or is longer than it:
    its request keeps its slots and length, the others are compacted."""
    base = dict(lens=[8, 8], pre=[10, 3], acc=[3, 4], page=16, h_kv=2, d=64)
    for kind in range(4):
        c = _case(3, **base)
        want = dict(c)
        want["acc"] = np.array([0, 4], np.int32)   # request 0 left alone
        k, v, new, _ = _expect(want)
        new[0] = 18
        bad = {k2: (x.copy() if isinstance(x, np.ndarray) else x) for k2, x in c.items()}
        if kind == 0:
            bad["path"][:3] = [0, 5, 5]
        elif kind == 1:
            bad["path"][:3] = [0, 2, 8]
        elif kind == 2:
            bad["path"][:3] = [-1, 2, 3]
        else:
            bad["acc"][0] = 9
        got = _run(va, bad)
        assert got[3] == 2
        assert np.array_equal(got[0], k) and np.array_equal(got[1], v) and np.array_equal(got[2], new)


def test_page_ids_outside_the_pool_are_skipped(va):
    c = _case(5, lens=[6], pre=[3], acc=[4], page=4, h_kv=2, d=64)
    c["path"][:4] = [0, 2, 3, 5]       # positions 3, 5, 6, 8: pages 0, 1, 1, 2 of the request
    c["ids"][2] = 1000                 # node 5's source
    want = dict(c, acc=np.array([3], np.int32))
    k, v, new, _ = _expect(want)
    got = _run(va, c)
    assert got[3] == 1 and np.array_equal(got[0], k) and np.array_equal(got[1], v) and got[2][0] == 7


def test_tables_that_disagree_are_flagged(va):
    c = _case(6, lens=[6, 5], pre=[3, 2], acc=[2, 3], page=4, h_kv=2, d=64)
    c["last"][0] = 9                   # more than a page holds
    got = _run(va, c)
    want = dict(c, acc=np.array([0, 3], np.int32))
    k, v, new, _ = _expect(want)
    assert got[3] == 2 and np.array_equal(got[0], k) and np.array_equal(got[1], v) and list(got[2]) == [0, int(new[1])]


def test_graph_replay_and_side_stream(va):
    cs = [_case(s, lens=[12, 9], pre=[4, 40], acc=a, page=16, h_kv=2, d=128) for s, a in ((1, [5, 3]), (2, [2, 7]))]
    cs[1].update(kvp=cs[0]["kvp"], last=cs[0]["last"])
    t = _dev(cs[0])
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    _run(va, cs[0], t, stream=side)
    kv_len = torch.zeros(2, dtype=torch.int32, device="cuda")
    with torch.cuda.graph(g, stream=side):
        va.paged_kv_compact(t["acc"], t["path"], t["qo"], t["kvp"], t["ids"], t["last"], t["k"], t["v"], kv_len_out=kv_len)
    for c in (cs[1], cs[0]):
        for n, x in _dev(c).items():
            t[n].copy_(x)
        g.replay()
        torch.cuda.synchronize()
        k, v, new, _ = _expect(c)
        assert np.array_equal(t["k"].view(torch.uint8).cpu().numpy(), k)
        assert np.array_equal(t["v"].view(torch.uint8).cpu().numpy(), v)
        assert np.array_equal(kv_len.cpu().numpy(), new)


def test_offsets_past_32_bits(va):
    """Rows beyond 4 GB of a pool (the slots are compared, not the pool)."""
    pages, h, P, d = 140000, 8, 16, 128
    pool = [torch.empty((pages, h, P, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    assert pool[0].numel() * 2 > 1 << 32
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    last = pages - 1
    for x in pool:
        x[last].normal_()
        x[2].normal_()
    want = [(x[last, :, 3].clone(), x[2, :, 1].clone()) for x in pool]
    # prefix 13: drafts 0 .. 2 on the last page's slots 13 .. 15, 3 .. 5 on page 2's 0 .. 2
    keep = [x[last, :, 13].clone() for x in pool]
    va.paged_kv_compact(i(2), i(0, 4, -1, -1, -1, -1), i(0, 6), i(0, 2), i(last, 2), i(3), *pool)
    for x, (a, b), k in zip(pool, want, keep):
        assert torch.equal(x[last, :, 13], k) and torch.equal(x[last, :, 14], b) and torch.equal(x[last, :, 3], a)


def test_refusals(va):
    c = _case(4, lens=[3], pre=[1], acc=[2], page=16, h_kv=2, d=64)
    t = _dev(c)
    names = ["acc", "path", "qo", "kvp", "ids", "last", "k", "v"]

    def call(n, x):
        a = dict(t)
        a[n] = x
        va.paged_kv_compact(*[a[m] for m in names])

    for n, x in (("acc", t["acc"].long()), ("acc", t["acc"].cpu()), ("path", t["path"].long()), ("qo", t["qo"].cpu()),
                 ("kvp", t["kvp"][:1]), ("ids", t["ids"][None]), ("last", t["last"].float()), ("k", t["k"].half()),
                 ("k", t["k"].transpose(1, 2)), ("v", t["v"][:2]), ("v", t["v"].view(torch.float8_e4m3fn)), ("k", t["k"][0])):
        with pytest.raises((ValueError, KeyError)):
            call(n, x)
    with pytest.raises(va.VerifyAttnError):   # a head width that is not served
        va.paged_kv_compact(*[t[m] for m in names[:6]], t["k"][..., :32].contiguous(), t["v"][..., :32].contiguous())
