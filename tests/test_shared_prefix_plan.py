"""Host planner for shared prefixes: every row sees each of its keys through
exactly one partial that its merge reads, partials do not overlap, sizes stay
below the bounds, and the argument checks."""
import ctypes

import numpy as np
import pytest


@pytest.fixture(scope="module")
def va():
    from speculative_decoding_verify_gqa_gb300 import build as b
    b.build()
    import speculative_decoding_verify_gqa_gb300 as m
    m.lib()
    return m


def _groups_of(plan, n):
    hd = plan.header()
    off = 184 + 32 * (hd["n_items"] + hd["n_merge"])
    return np.frombuffer(plan.host[off:off + 32 * n].tobytes(), np.int32).reshape(-1, 8)


def _tables(rng, groups, page, max_shared, max_own, max_L, masked):
    """groups: members of each.  Page ids are drawn so that nothing but the shared pages coincides."""
    kvp, qo, last, ids, gi, sp, mi = [0], [0], [], [], [0], [], [0]
    nxt = 0
    for m in groups:
        s = int(rng.integers(0, max_shared // page + 1))
        shared = list(range(nxt, nxt + s))
        nxt += s
        for _ in range(m):
            L = int(rng.integers(0, max_L + 1))
            own = int(rng.integers(0, max_own + 1)) + L
            n = -(-own // page)
            ids += shared + list(range(nxt, nxt + n))
            nxt += n
            kv = s * page + own
            kvp.append(kvp[-1] + s + n)
            qo.append(qo[-1] + L)
            last.append((kv - 1) % page + 1 if kv else 0)
            mi.append(mi[-1] + L * L)
        gi.append(gi[-1] + m)
        sp.append(s)
    a = lambda x: np.array(x, np.int32)  # noqa: E731
    return a(kvp), a(ids), a(qo), a(last), a(mi) if masked else None, a(gi), a(sp)


def _check_plan(va, tables, h_q, h_kv, d, page, num_sms, **opts):
    kvp, ids, qo, last, mi, gi, sp = tables
    batch, ng, G = len(qo) - 1, len(sp), h_q // h_kv
    plan = va.verify_attn_plan_shared_host(kvp, qo, last, mi, gi, sp, h_q, h_kv, d, page, num_sms=num_sms, **opts)
    hd = plan.header()
    recs, items, merges = _groups_of(plan, ng), plan.items(), plan.merges()
    pb, wb = va.verify_attn_plan_shared_bounds(batch, ng, int(qo[-1]), h_q, h_kv, d, num_sms)
    assert 184 + 32 * (hd["n_items"] + hd["n_merge"] + ng) <= pb and plan.workspace_bytes <= wb
    kv = [(int(kvp[b + 1] - kvp[b]) - 1) * page + int(last[b]) if kvp[b + 1] > kvp[b] else 0 for b in range(batch)]
    # every partial row is written once: part row -> (lo, hi) of the item, per (request, head, row) or group row
    part = {}
    final = set()
    for b, h, row0, nrows, lo, hi, pr, _ in items.tolist():
        assert 0 <= h < h_kv and nrows > 0 and lo < hi
        if b >= batch:
            g = recs[b - batch]
            assert pr >= 0 and row0 + nrows <= g[3] and hi <= g[2] * page
        else:
            assert row0 + nrows <= G * int(qo[b + 1] - qo[b]) and hi <= kv[b]
        for r in range(nrows):
            if pr < 0:
                assert (b, h, row0 + r) not in final
                final.add((b, h, row0 + r))
                if mi is None:
                    assert lo == 0 and hi >= kv[b] - int(qo[b + 1] - qo[b]) + (row0 + r) // G + 1
                else:
                    assert (lo, hi) == (0, kv[b])
            else:
                assert pr + r not in part and pr + r < hd["part_rows"]
                part[pr + r] = (b, h, row0 + r, lo, hi)
    # the merge of each row reads partials that tile its keys
    used, shared_rows = set(), 0
    most = 0
    for b, h, row0, nrows, base, ns, grp, _ in merges.tolist():
        for r in range(nrows):
            src = [base + s * nrows + r for s in range(ns)]
            assert all(part[x][:3] == (b, h, row0 + r) for x in src)
            if grp:
                g = recs[grp - 1]
                rg = (int(qo[b]) - int(qo[g[0]])) * G + row0 + r
                more = [int(g[4]) + (h * int(g[5]) + s) * int(g[3]) + rg for s in range(int(g[5]))]
                assert all(part[x][:3] == (batch + grp - 1, h, rg) for x in more)
                src += more
                shared_rows += 1
            used.update(src)
            most = max(most, len(src))
            spans = sorted(part[x][3:] for x in src)
            t = (row0 + r) // G
            end = kv[b] if mi is not None else kv[b] - int(qo[b + 1] - qo[b]) + t + 1
            assert spans[0][0] == 0 and spans[-1][1] >= end and spans[-1][1] <= kv[b]
            assert all(x[1] == y[0] for x, y in zip(spans, spans[1:]))
            assert (b, h, row0 + r) not in final
            final.add((b, h, row0 + r))
    assert used == set(part) and most == hd["max_nsplit"]
    assert final == {(b, h, r) for b in range(batch) for h in range(h_kv) for r in range(G * int(qo[b + 1] - qo[b]))}
    if hd["n_ctas"]:
        # every item on exactly one chain
        seen = []
        for c in range(hd["n_ctas"]):
            i = c
            while i >= 0:
                seen.append(i)
                i = int(items[i][7])
        assert sorted(seen) == list(range(hd["n_items"]))
    return plan, shared_rows


CASES = [
    dict(groups=[4], page=16, max_shared=2048, max_own=200, max_L=1, h_q=32, h_kv=8, d=128),
    dict(groups=[32], page=16, max_shared=4096, max_own=500, max_L=5, h_q=32, h_kv=8, d=128),
    dict(groups=[8, 8, 8], page=32, max_shared=9000, max_own=700, max_L=17, h_q=32, h_kv=8, d=128, masked=True),
    dict(groups=[5, 1, 0, 5], page=8, max_shared=1000, max_own=90, max_L=6, h_q=14, h_kv=2, d=64),
    dict(groups=[1, 1, 1], page=16, max_shared=500, max_own=50, max_L=3, h_q=8, h_kv=2, d=128),
    dict(groups=[30, 20], page=1, max_shared=300, max_own=30, max_L=9, h_q=3, h_kv=1, d=128, masked=True),
    dict(groups=[], page=16, max_shared=0, max_own=0, max_L=0, h_q=8, h_kv=2, d=128),
]


@pytest.mark.parametrize("num_sms", [1, 7, 152])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_plan_covers_every_row_and_key_once(va, case, num_sms):
    c = dict(CASES[case])
    dims = [c.pop(k) for k in ("h_q", "h_kv", "d")]
    page = c["page"]
    t = _tables(np.random.default_rng(case), c["groups"], page, c["max_shared"], c["max_own"], c["max_L"],
                c.get("masked", False))
    for opts in ({}, dict(max_splits=1), dict(min_chunk=512), dict(target_ctas=300), dict(kv_dtype="fp8_e4m3")):
        _check_plan(va, t, *dims, page, num_sms, **opts)


@pytest.mark.parametrize("seed", range(40))
def test_random_plans(va, seed):
    rng = np.random.default_rng(seed)
    page = int(2 ** rng.integers(0, 7))
    h_kv, G = int(rng.integers(1, 5)), int(rng.choice([1, 2, 3, 4, 8]))
    t = _tables(rng, rng.integers(0, 12, rng.integers(1, 5)).tolist(), page, int(rng.integers(page, 6000)),
                int(rng.integers(0, 400)), int(rng.integers(1, 20)), bool(rng.integers(0, 2)))
    _check_plan(va, t, G * h_kv, h_kv, int(rng.choice([64, 128])), page, int(rng.choice([4, 100, 152])))


def test_a_long_shared_prefix_is_shared(va):
    rng = np.random.default_rng(1)
    t = list(_tables(rng, [32], 16, 4096, 100, 5, False))
    while t[6][0] < 200:
        t = list(_tables(rng, [32], 16, 4096, 100, 5, False))
    plan, rows = _check_plan(va, t, 32, 8, 128, 16, 152)
    assert rows == 32 * int(t[2][-1])
    # and a tiny one is not: the partials would cost more than the keys
    t = _tables(rng, [2], 16, 16, 100, 17, False)
    _, rows = _check_plan(va, t, 32, 8, 128, 16, 152)
    assert rows == 0


def test_a_group_of_one_plans_like_no_group(va):
    t = _tables(np.random.default_rng(4), [1, 1], 16, 3000, 100, 17, False)
    _, rows = _check_plan(va, t, 32, 8, 128, 16, 152)
    assert rows == 0


def test_plan_validation(va):
    kvp, qo, last, gi, sp = [0, 4, 8], [0, 2, 4], [3, 3], [0, 2], [3]
    # kv_len 51: prefix 49, three whole pages of 16
    ok = dict(kv=kvp, qo=qo, last=last, mi=None, gi=gi, sp=sp)

    def call(h_q=8, h_kv=2, d=128, page=16, opts=None, **kw):
        a = dict(ok, **kw)
        return va.verify_attn_plan_shared_host(a["kv"], a["qo"], a["last"], a["mi"], a["gi"], a["sp"], h_q, h_kv, d, page,
                                               num_sms=152, **(opts or {}))

    call()
    for bad, code in ((dict(sp=[4]), -1), (dict(sp=[-1]), -1), (dict(gi=[0, 1]), -1), (dict(gi=[1, 2]), -1),
                      (dict(gi=[0, 2, 1, 2], sp=[0, 0, 0]), -1), (dict(last=[1, 3]), -1), (dict(last=[17, 3]), -1),
                      (dict(qo=[0, 60, 62]), -1), (dict(kv=[0, 4, 3]), -1), (dict(mi=[0, 4, 9]), -1),
                      (dict(opts=dict(mask_layout="full"), mi=[0, 4, 8]), -2), (dict(opts=dict(draft_items=1)), -2),
                      (dict(opts=dict(draft_items=2)), -1), (dict(opts=dict(kernel=9)), -1), (dict(page=24), -2),
                      (dict(d=96), -2), (dict(h_q=9), -1), (dict(opts=dict(q_fp8=True)), -2),
                      (dict(opts=dict(kernel=3), page=8, last=[3, 3], sp=[2]), -2), (dict(opts=dict(max_splits=-1)), -1)):
        with pytest.raises(va.VerifyAttnError) as e:
            call(**bad)
        assert e.value.status == code, bad
    with pytest.raises(ValueError):
        call(sp=[1, 1])
    with pytest.raises(ValueError):
        call(last=[3])
    # a plan buffer that is too small reports the bytes it needs
    need = ctypes.c_size_t(0)
    a = [np.array(x, np.int32) for x in (kvp, qo, last, gi, sp)]
    rc = va.lib().verify_attn_plan_shared_host(a[0].ctypes.data, a[1].ctypes.data, a[2].ctypes.data, None, 2,
                                               a[3].ctypes.data, a[4].ctypes.data, 1, 8, 2, 128, 16, 0, 0, 0, 152, None,
                                               a[0].ctypes.data, 8, ctypes.byref(need))
    assert rc == -7 and need.value > 184


def test_found_groups(va):
    f = lambda ids, lens, L, page=4, **kw: [  # noqa: E731
        x.tolist() for x in va.verify_attn_shared_groups(
            np.concatenate([[0], np.cumsum([len(i) for i in ids])]), sum(ids, []), np.concatenate([[0], np.cumsum(L)]),
            lens, page, **kw)]
    # three requests share 2, 2 and 2 pages; the fourth starts elsewhere
    a = [[1, 2, 3], [1, 2, 4], [1, 2, 5, 6], [7, 8]]
    assert f(a, [1, 2, 3, 4], [1, 1, 1, 1]) == [[0, 3, 4], [2, 0]]
    # drafts that reach into the second page: only one whole page is before them
    assert f(a, [1, 2, 3, 4], [1, 3, 1, 1]) == [[0, 3, 4], [1, 0]]
    # joining a third with one common page would save less (2 < 5): it starts anew
    b = [[1, 2, 3, 4, 5, 6], [1, 2, 3, 4, 5, 7], [1, 8, 9], [1, 8, 10]]
    assert f(b, [4] * 4, [1] * 4) == [[0, 2, 4], [5, 2]]
    assert f(a, [1, 2, 3, 4], [1, 1, 1, 1], min_pages=3) == [[0, 1, 2, 3, 4], [0, 0, 0, 0]]
    assert f([], [], []) == [[0], []]
    with pytest.raises(va.VerifyAttnError):
        f(a, [1, 2, 3, 9], [1, 1, 1, 1])
    with pytest.raises(ValueError):
        va.verify_attn_shared_groups([0, 3], [1], [0, 1], [1], 4)


@pytest.mark.parametrize("seed", range(10))
def test_found_groups_plan(va, seed):
    """What verify_attn_shared_groups finds is what the planner accepts, and truly shared."""
    rng = np.random.default_rng(seed)
    kvp, ids, qo, last, mi, gi, sp = _tables(rng, [3, 1, 5, 2], 8, 600, 60, 5, False)
    g, s = va.verify_attn_shared_groups(kvp, ids, qo, last, 8)
    for i in range(len(s)):
        for b in range(g[i], g[i + 1]):
            assert (ids[kvp[b]:kvp[b] + s[i]] == ids[kvp[g[i]]:kvp[g[i]] + s[i]]).all()
    _check_plan(va, (kvp, ids, qo, last, None, g, s), 16, 4, 128, 8, 152)
