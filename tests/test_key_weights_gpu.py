"""GPU test of verify_attn_key_weights against the definition in double
precision, element by element within a bound of what fp32 may lose; every slot
that no key of a request lies in stays as it was."""
import math

import numpy as np
import pytest
import torch

from oracle import budget

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def va():
    import __graft_entry__
    __graft_entry__.build()
    import speculative_decoding_verify_gqa_gb300 as m
    return m


class Case:
    def __init__(self, seed, lens, pre, page=16, hq=8, h=2, d=128, fp8=False, nhd=False, mask=None, path=False,
                 decay=1.0, scale=0.0, peak=1.0):
        rng = np.random.default_rng(seed)
        self.rng = rng
        self.lens, self.pre, self.page, self.hq, self.h, self.d = lens, pre, page, hq, h, d
        self.fp8, self.nhd, self.kind, self.decay, self.scale = fp8, nhd, mask, decay, scale
        need = [-(-(a + n) // page) for a, n in zip(pre, lens)]
        pages = sum(need) + 2
        ptr = lambda x: np.concatenate([[0], np.cumsum(x)]).astype(np.int32)  # noqa: E731
        self.ids = rng.permutation(pages)[:max(1, sum(need))].astype(np.int32)
        self.kvp, self.indptr = ptr(need), ptr(lens)
        self.last = np.array([(a + n - 1) % page + 1 if a + n else 0 for a, n in zip(pre, lens)], np.int32)
        total = sum(lens)
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        self.q = t(rng.standard_normal((total, hq, d)).astype(np.float32) * peak).to(torch.bfloat16)
        mid = (page, h) if nhd else (h, page)
        k = t(rng.standard_normal((pages,) + mid + (d,)).astype(np.float32))
        self.k_scale = 1 / 64 if fp8 else 1.0
        self.kc = (k * 64).to(torch.float8_e4m3fn) if fp8 else k.to(torch.bfloat16)
        self.w0 = rng.lognormal(0, 1, (pages,) + mid).astype(np.float32)
        self.w = t(self.w0.copy())
        # masks: random bits ("holes": some rows and some keys are seen by nobody)
        self.mask = self.mask_indptr = None
        if mask:
            full = mask.startswith("full")
            widths = [a + n if full else n for a, n in zip(pre, lens)]
            self.mask_indptr = ptr([n * x for n, x in zip(lens, widths)])
            bits = rng.random(int(self.mask_indptr[-1])) < (0.3 if "holes" in mask else 0.7)
            if "holes" in mask:
                for b, (n, x) in enumerate(zip(lens, widths)):
                    view = bits[self.mask_indptr[b]:self.mask_indptr[b + 1]].reshape(n, x)
                    view[::3] = False
                    view[:, ::4] = False
            self.mask = np.packbits(np.concatenate([bits, np.zeros(-len(bits) % 8 + 8, bool)]), bitorder="little")
        self.acc = self.path = None
        if path:
            self.acc = np.array([rng.integers(0, n + 1) for n in lens], np.int32)
            self.path = np.full(total, -1, np.int32)
            for b, a in enumerate(self.acc):
                self.path[self.indptr[b]:self.indptr[b] + a] = np.sort(rng.choice(lens[b], a, replace=False))
        self.full = bool(mask) and mask.startswith("full")
        self.dev = {n: t(getattr(self, n)) for n in ("ids", "kvp", "indptr", "last")}
        for n in ("mask", "mask_indptr", "acc", "path"):
            self.dev[n] = None if getattr(self, n) is None else t(getattr(self, n))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.set_lse()

    def request(self, b):
        pages, slots = budget.slots_of(self.kvp, self.ids, self.last, self.page, b)
        k = self.kc.float().double().cpu().numpy()
        k = k[pages, slots] if self.nhd else k[pages, :, slots]
        n = self.lens[b]
        seen = budget.visible(n, len(pages), self.mask, 0 if self.mask is None else int(self.mask_indptr[b]), self.full)
        q = self.q[self.indptr[b]:self.indptr[b + 1]].double().cpu().numpy()
        scale = (self.scale or 1 / math.sqrt(self.d)) * self.k_scale
        return q, k, seen, scale, pages, slots

    def set_lse(self):
        lse = np.zeros((sum(self.lens), self.hq), np.float32)
        G = self.hq // self.h
        for b, n in enumerate(self.lens):
            q, k, seen, scale, _, _ = self.request(b)
            s = np.einsum("nhgd,mhd->nhgm", q.reshape(n, self.h, G, self.d), k) * scale
            s = np.where(seen[:, None, None], s, -np.inf)
            with np.errstate(divide="ignore", invalid="ignore"):
                m = s.max(-1, keepdims=True, initial=-np.inf)
                l = np.log(np.exp(s - np.where(np.isfinite(m), m, 0)).sum(-1)) + m[..., 0]
            lse[self.indptr[b]:self.indptr[b + 1]] = np.where(np.isfinite(l), l, -np.inf).reshape(n, self.hq)
        self.lse = torch.from_numpy(lse).cuda()

    def run(self, va, **kw):
        x = self.dev
        args = dict(mask=x["mask"], mask_indptr=x["mask_indptr"], accept_len=x["acc"], accepted_nodes=x["path"],
                    sm_scale=self.scale, k_scale=self.k_scale, decay=self.decay, kv_layout="nhd" if self.nhd else "hnd",
                    mask_layout="full" if self.full else "qlen", status=self.status)
        args.update(kw)
        return va.verify_attn_key_weights(self.q, self.kc, x["kvp"], x["ids"], x["last"], x["indptr"], self.lse, self.w,
                                          **args)

    def check(self, skip=(), skip_pages=(), times=1):
        got = self.w.cpu().numpy()
        touched = np.zeros(got.shape, bool)
        for b, n in enumerate(self.lens):
            if b in skip:
                continue
            q, k, seen, scale, pages, slots = self.request(b)
            path = None if self.acc is None else self.path[self.indptr[b]:self.indptr[b] + self.acc[b]]
            w, loss = budget.key_weights(q, k, self.lse[self.indptr[b]:self.indptr[b + 1]].cpu().numpy(), seen, scale, path)
            m = len(w)
            at = (pages[:m], slots[:m]) if self.nhd else (pages[:m], slice(None), slots[:m])
            old = self.w0[at].astype(np.float64)
            if not self.nhd:
                old = old.reshape(m, self.h)
            base = np.where((np.arange(m) < self.pre[b])[:, None], old, 0.0)
            decay = np.float64(np.float32(self.decay))
            want = w
            base = np.where(base != 0, base * decay, 0.0) if self.decay else np.zeros_like(base)
            want = base + w
            tol = loss + 2.0 ** -23 * np.abs(want) + 1e-38
            have = got[at].astype(np.float64)
            ok = np.ones(m, bool) & ~np.isin(pages[:m], list(skip_pages))
            if self.nhd:
                touched[pages[:m][ok], slots[:m][ok]] = True
            else:
                touched[pages[:m][ok], :, slots[:m][ok]] = True
            err = np.abs(have - want)[ok]
            assert np.all(err <= tol[ok]), (b, float(err.max()), float((err / tol[ok]).max()))
        assert np.array_equal(got[~touched], self.w0[~touched])


CASES = [
    dict(lens=[1], pre=[0]),
    dict(lens=[1], pre=[127]),
    dict(lens=[1], pre=[128], hq=32, h=8),
    dict(lens=[17], pre=[300], hq=32, h=8, mask="qlen"),
    dict(lens=[17, 0, 3], pre=[300, 40, 0], hq=32, h=8, path=True),
    dict(lens=[4, 8, 1, 2], pre=[513, 2, 1030, 77], hq=64, h=8, decay=0.97),
    dict(lens=[9, 33], pre=[100, 1000], fp8=True, nhd=True, page=32, mask="qlen-holes"),
    dict(lens=[5, 19], pre=[200, 31], d=64, hq=14, h=2, page=1, mask="qlen"),
    dict(lens=[5, 19], pre=[200, 31], d=64, hq=6, h=6, page=8, fp8=True, decay=0.0),
    dict(lens=[300], pre=[0], hq=8, h=1),
    dict(lens=[130, 257, 1], pre=[0, 5, 600], hq=6, h=2, nhd=True, decay=0.0),
    dict(lens=[64], pre=[700], hq=8, h=2, mask="full-holes", page=64),
    dict(lens=[12, 3], pre=[0, 140], hq=4, h=2, mask="full-holes", d=64, fp8=True),
    dict(lens=[11], pre=[0], hq=4, h=4, mask="qlen-holes"),
    dict(lens=[2] * 200, pre=[3] * 200, hq=2, h=1, d=64, page=4),
    dict(lens=[1] * 3, pre=[2000, 1, 500], hq=16, h=1, path=True, fp8=True, page=256),
    dict(lens=[7], pre=[400], hq=5, h=5, scale=0.3, peak=2.0),
    dict(lens=[40], pre=[90], hq=96, h=12, path=True, nhd=True),
    dict(lens=[0], pre=[50], decay=0.5),
    dict(lens=[1], pre=[40000], hq=2, h=1),
    dict(lens=[700], pre=[300], hq=14, h=2, d=64, mask="qlen", page=2),
]


@pytest.mark.parametrize("n", range(len(CASES)))
def test_against_definition(va, n):
    c = Case(n, **CASES[n])
    assert c.run(va) is c.w
    torch.cuda.synchronize()
    assert int(c.status) == 0
    c.check()


def test_decay_zero_does_not_read(va):
    c = Case(60, [3], [200], decay=0.0)
    c.w.fill_(float("nan"))
    c.run(va)
    got = c.w.clone()
    c.w0 = np.full_like(c.w0, np.nan)
    pages, slots = budget.slots_of(c.kvp, c.ids, c.last, c.page, 0)
    assert not bool(got[torch.from_numpy(pages).cuda().long(), :, torch.from_numpy(slots).cuda().long()].isnan().any())
    # the step's own keys start at 0 with any decay
    c.decay = 1.0
    c.run(va)
    new = c.w[torch.from_numpy(pages[200:]).cuda().long(), :, torch.from_numpy(slots[200:]).cuda().long()]
    assert not bool(new.isnan().any())


@pytest.mark.parametrize("d", [64, 128])
def test_hidden_keys_may_hold_anything(va, d):
    for kind in ("qlen-holes", "full-holes"):
        c = Case(61, [12], [150], hq=8, h=2, d=d, mask=kind)
        pages, slots = budget.slots_of(c.kvp, c.ids, c.last, c.page, 0)
        _, _, seen, _, _, _ = c.request(0)
        hidden = np.nonzero(~seen.any(0))[0]
        assert len(hidden)
        clean = c.kc.clone()
        for x, j in zip([float("nan"), float("inf"), -float("inf")] * len(hidden), hidden):
            c.kc[int(pages[j]), :, int(slots[j])] = x
        c.run(va)
        c.kc = clean
        c.check()
    # slots behind the last key, and of other pages
    c = Case(62, [3], [70], hq=8, h=2, d=d)
    pages, slots = budget.slots_of(c.kvp, c.ids, c.last, c.page, 0)
    clean = c.kc.clone()
    free = np.ones(c.w0.shape, bool)
    free[pages, :, slots] = False
    c.kc[torch.from_numpy(free).cuda()] = float("nan")
    c.run(va)
    c.kc = clean
    c.check()


def test_nan_reaches_what_it_was_seen_with(va):
    c = Case(63, [4], [40], hq=8, h=2)
    c.q[2, 1] = float("nan")      # head 1: KV head 0; query 2 sees keys 0 .. 42
    c.run(va)
    pages, slots = budget.slots_of(c.kvp, c.ids, c.last, c.page, 0)
    w = c.w[torch.from_numpy(pages).cuda().long(), :, torch.from_numpy(slots).cuda().long()]
    assert bool(w[:43, 0].isnan().all()) and not bool(w[43:, 0].isnan().any()) and not bool(w[:, 1].isnan().any())


def test_skipped_requests(va):
    c = Case(64, [4, 5], [40, 60])
    c.dev["last"][0] = 0
    c.run(va)
    assert int(c.status) == 2
    c.check(skip=[0])
    c = Case(65, [6, 5], [40, 60], path=True)
    o = int(c.indptr[1])
    c.dev["acc"][1] = 2
    c.dev["path"][o], c.dev["path"][o + 1] = 3, 3
    c.run(va)
    assert int(c.status) == 2
    c.check(skip=[1])
    c = Case(66, [4, 5], [40, 60])
    bad = int(c.ids[1])
    c.dev["ids"][1] = 10 ** 8
    c.run(va)
    assert int(c.status) == 1
    c.check(skip_pages=[bad])


def test_graph_stream_and_repeats(va):
    c = Case(67, [5, 9], [300, 45], hq=32, h=8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.run(va)
    torch.cuda.current_stream().wait_stream(s)
    c.check()
    first = c.w.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(va)
    for _ in range(2):   # the same bits every time
        c.w.copy_(torch.from_numpy(c.w0))
        g.replay()
        assert torch.equal(c.w, first)


def test_weights_add_up(va):
    """With the attention's own lse a step hands out one unit of weight per query and head."""
    c = Case(68, [6, 1], [500, 2000], hq=16, h=4, decay=0.0)
    plan = va.verify_attn_plan(c.kvp, c.indptr, c.last, None, c.hq, c.h, c.d, c.page)
    _, c.lse = va.verify_attn_run(c.q, c.kc, c.kc, c.dev["kvp"], c.dev["ids"], c.dev["last"], c.dev["indptr"], None,
                                  None, plan)
    c.run(va)
    for b, n in enumerate(c.lens):
        pages, slots = budget.slots_of(c.kvp, c.ids, c.last, c.page, b)
        w = c.w[torch.from_numpy(pages).cuda().long(), :, torch.from_numpy(slots).cuda().long()].double()
        assert torch.allclose(w.sum(0), torch.full((c.h,), float(n * c.hq // c.h), dtype=torch.float64, device="cuda"),
                              rtol=1e-3)


def test_far_rows(va):
    """Cache rows behind 2^31 elements."""
    pages, P, d = 140000, 64, 128
    k = torch.zeros((pages, 2, P, d), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((pages, 2, P), device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    k[pages - 1] = torch.randn((2, P, d), generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn((1, 2, d), generator=g, device="cuda").to(torch.bfloat16)
    s = torch.einsum("hd,hpd->hp", q[0].double(), k[pages - 1].double()) / math.sqrt(d)
    lse = torch.logsumexp(s, -1)
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    va.verify_attn_key_weights(q, k, i([0, 1]), i([pages - 1]), i([P]), i([0, 1]), lse.float()[None], w)
    assert torch.allclose(w[pages - 1].double(), torch.exp(s - lse[:, None]), rtol=1e-4)
    assert int((w != 0).sum()) == 2 * P


# Calls whose CTAs have several units each: with the rows held, streamed in order
# of cost (some request has more than 256 rows), and streamed as they come (more
# than 512 units of a head besides).
MANY = [
    dict(lens=[8, 3, 1, 5] * 10, pre=list(range(300, 3500, 80)), hq=16, h=4),
    dict(lens=[8, 3, 1, 5] * 10, pre=list(range(300, 3500, 80)), hq=16, h=4, fp8=True, nhd=True, page=64, mask="qlen-holes"),
    dict(lens=[60, 2, 33] * 8, pre=[1500, 17, 900] * 8, hq=12, h=6, d=64, path=True, decay=0.9),
    dict(lens=[50, 2, 33] * 8, pre=[1500, 17, 900] * 8, hq=30, h=6, d=64, fp8=True, page=4, path=True),
    dict(lens=[300, 40, 1, 0], pre=[2500, 1000, 3000, 100], hq=32, h=8),
    dict(lens=[300, 40, 1, 0], pre=[2500, 1000, 3000, 100], hq=32, h=8, fp8=True, nhd=True, page=64),
    dict(lens=[0, 129, 260, 7], pre=[90, 2000, 1001, 2222], hq=40, h=8, d=64, mask="qlen-holes", page=4),
    dict(lens=[129, 260, 7], pre=[2000, 1001, 2222], hq=40, h=8, d=64, mask="full-holes", fp8=True, page=32),
    dict(lens=[200, 260, 7], pre=[2000, 1001, 2222], hq=40, h=8, path=True, decay=0.5),
    dict(lens=[200, 260, 7], pre=[2000, 1001, 2222], hq=40, h=8, path=True, fp8=True, d=64, page=128),
    dict(lens=[700, 900], pre=[0, 128], hq=64, h=16, nhd=True),
    dict(lens=[2] * 300 + [200] + [2] * 250, pre=[9] * 551, hq=4, h=2, d=64),
    dict(lens=[2] * 300 + [200] + [2] * 250, pre=[9] * 551, hq=4, h=2, fp8=True, page=8, path=True),
]


@pytest.mark.parametrize("n", range(len(MANY)))
def test_many_units(va, n):
    c = Case(100 + n, **MANY[n])
    c.run(va)
    torch.cuda.synchronize()
    assert int(c.status) == 0
    c.check()


def test_padded_batch(va):
    """Requests of no pages and no tokens behind the last one, and query rows behind the last request's."""
    c = Case(120, [5, 3, 0, 0, 0], [200, 31, 0, 0, 0])
    o = int(c.indptr[-1])
    c.q = torch.cat([c.q, torch.full_like(c.q[:4], float("nan"))])
    c.lse = torch.cat([c.lse, torch.full_like(c.lse[:4], float("nan"))])
    assert c.q.shape[0] == o + 4
    c.run(va)
    torch.cuda.synchronize()
    assert int(c.status) == 0
    c.q, c.lse = c.q[:o], c.lse[:o]
    c.check()


def test_two_calls_at_once(va):
    cases = [Case(121, **MANY[4]), Case(122, **MANY[1])]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                c.w.copy_(torch.from_numpy(c.w0))
                c.run(va)
    torch.cuda.synchronize()
    for c in cases:
        assert int(c.status) == 0
        c.check()


@pytest.mark.parametrize("mask", ["qlen", "full-holes"])
def test_mask_offsets_that_disagree(va, mask):
    """Mask offsets below 0, or of another span than L * L (L * kv_len for the
    full layout), leave their requests alone; the mask is not read there."""
    lens, pre = [5, 7, 300, 4], [40, 0, 60, 9]
    c = Case(130, lens, pre, mask=mask)
    c.dev["mask_indptr"][1] = -16           # the end of request 0's mask, the beginning of request 1's
    c.run(va)
    assert int(c.status) == 2
    c.check(skip=[0, 1])
    c = Case(131, lens, pre, mask=mask, fp8=True, nhd=True)
    c.dev["mask_indptr"][4] -= 1
    c.run(va)
    assert int(c.status) == 2
    c.check(skip=[3])
    c = Case(132, lens, pre, mask=mask, hq=16)
    c.dev["mask_indptr"][3:] += 1 << 30     # two spans too long
    c.dev["mask_indptr"][4] += 8
    c.run(va)
    assert int(c.status) == 2
    c.check(skip=[2, 3])
    c = Case(133, [0, 3], [10, 20], mask=mask)
    c.dev["mask_indptr"][0] = -1            # a request without tokens, too
    c.run(va)
    assert int(c.status) == 2
    c.check(skip=[0])


LEFT_OUT = [
    dict(lens=[4, 9, 1], pre=[40, 200, 0], hq=8, h=2),
    dict(lens=[4, 9, 1], pre=[40, 200, 0], hq=6, h=2, d=64, fp8=True, page=4, decay=0.5),
    dict(lens=[17, 30], pre=[300, 10], hq=32, h=8, mask="qlen-holes"),
    dict(lens=[12, 40], pre=[30, 140], hq=8, h=2, d=64, mask="full-holes", fp8=True, nhd=True, page=32),
    dict(lens=[40, 7], pre=[90, 500], hq=16, h=2, path=True),
    dict(lens=[700, 300], pre=[100, 2000], hq=16, h=4),
    dict(lens=[700, 300], pre=[100, 2000], hq=16, h=4, fp8=True, nhd=True, mask="qlen"),
    dict(lens=[8, 3, 1, 5] * 10, pre=list(range(300, 3500, 80)), hq=16, h=4),
]


@pytest.mark.parametrize("n", range(len(LEFT_OUT)))
def test_queries_left_out(va, n):
    """A query whose lse is -inf counts nothing, whatever its row and the keys that it would see hold."""
    c = Case(140 + n, **LEFT_OUT[n])
    out = torch.from_numpy(c.rng.random(c.lse.shape) < 0.2).cuda()
    out[::5] = True                          # whole tokens among them
    c.lse[out] = -float("inf")
    row = torch.from_numpy(c.rng.integers(0, 4, c.lse.shape)).cuda()
    for k, special in enumerate((float("nan"), float("inf"), -float("inf"), 3e38)):
        c.q[out & (row == k)] = special
    c.run(va)
    torch.cuda.synchronize()
    assert int(c.status) == 0
    c.check()


@pytest.mark.parametrize("fp8", [False, True])
def test_all_queries_left_out(va, fp8):
    """Nothing is added where every lse is -inf, whatever q holds; a key of NaN or
    infinity harms no weight but its own."""
    c = Case(150, [6, 300], [150, 40], hq=8, h=2, fp8=fp8, decay=0.5)
    c.lse.fill_(-float("inf"))
    c.q[::2] = float("nan")
    c.q[1::2] = float("inf")
    bad = []
    for b in range(2):
        pages, slots = budget.slots_of(c.kvp, c.ids, c.last, c.page, b)
        bad.append(torch.arange(b, len(pages), 3, device="cuda"))
        c.kc.view(torch.uint8)[torch.from_numpy(pages[b::3]).cuda().long(), :, torch.from_numpy(slots[b::3]).cuda().long()] = 0x7f   # NaN
    c.run(va)
    for b in range(2):
        pages, slots = budget.slots_of(c.kvp, c.ids, c.last, c.page, b)
        at = (torch.from_numpy(pages).cuda().long(), slice(None), torch.from_numpy(slots).cuda().long())
        want = 0.5 * torch.from_numpy(c.w0).cuda()[at]
        want[c.pre[b]:] = 0
        got = c.w[at]
        good = torch.ones(len(pages), dtype=torch.bool, device="cuda")
        good[bad[b]] = False
        assert torch.equal(got[good], want[good])


def test_no_pages_at_all(va):
    """An idle step: requests, none of which has a page or a token."""
    c = Case(151, [0, 0, 0], [0, 0, 0])
    c.dev["ids"] = c.dev["ids"][:0]
    assert c.run(va) is c.w
    torch.cuda.synchronize()
    assert int(c.status) == 0
    assert torch.equal(c.w, torch.from_numpy(c.w0).cuda())
