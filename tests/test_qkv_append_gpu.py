"""GPU test of paged_qkv_append against the definition in double precision:
normalised and rotated queries, keys and values in their slots, every other
slot and row as it was."""
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


def _tables(rng, lens, pre, page, spare=3):
    need = [-(-(a + n) // page) for a, n in zip(pre, lens)]
    pages = sum(need) + spare
    ids = rng.permutation(pages)[:max(1, sum(need))].astype(np.int32)
    ptr = lambda x: np.concatenate([[0], np.cumsum(x)]).astype(np.int32)  # noqa: E731
    last = np.array([(a + n - 1) % page + 1 if a + n else 0 for a, n in zip(pre, lens)], np.int32)
    return pages, dict(indptr=ptr(lens), kvp=ptr(need), ids=ids, last=last)


class Case:
    def __init__(self, seed, lens, pre, page=16, hq=8, h=2, d=128, dv=None, fp8=False, nhd=False, fused=True,
                 weights="bf16", offset=0.0, rot=None, inter=False, far=5000, pad=0, theta=5e5, eps=1e-6):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.page, self.hq, self.h, self.d, self.dv = page, hq, h, d, dv or d
        self.fp8, self.nhd, self.offset, self.inter, self.theta, self.eps = fp8, nhd, offset, inter, theta, eps
        self.total = sum(lens) + pad
        self.used = sum(lens)
        self.lens, self.pre = lens, pre
        self.rot = d if rot is None else rot
        pages, self.t = _tables(rng, lens, pre, page)
        wq, wk, wv = hq * d, h * d, h * self.dv
        rows = torch.randn((self.total, wq + wk + wv), generator=g).to(torch.bfloat16)
        rows[:, ::7] *= 3
        parts = rows.split([wq, wk, wv], 1)
        if fused:
            rows = rows.cuda()
            parts = rows.split([wq, wk, wv], 1)
        else:
            parts = [p.contiguous().cuda() for p in parts]
        self.q, self.k, self.v = (p.view(self.total, n, w) for p, n, w in zip(parts, (hq, h, h), (d, d, self.dv)))
        self.qw = self.kw = None
        if weights:
            dt = torch.bfloat16 if weights == "bf16" else torch.float32
            self.qw, self.kw = ((torch.rand(d, generator=g) + 0.5 - offset).to(dt).cuda() for _ in range(2))
        self.positions = torch.from_numpy(rng.integers(0, far + 1, self.total).astype(np.int32)).cuda()
        mid = (page, h) if nhd else (h, page)
        raw = lambda w: torch.from_numpy(rng.integers(0, 256, (pages,) + mid + (w * (1 if fp8 else 2),), dtype=np.uint8))  # noqa: E731
        dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
        self.k0, self.v0 = raw(d), raw(self.dv)
        self.kc, self.vc = self.k0.clone().cuda().view(dt), self.v0.clone().cuda().view(dt)
        self.scales = (0.0231, 0.0187) if fp8 else (None, None)
        self.dev = {n: torch.from_numpy(x).cuda() for n, x in self.t.items()}
        self.q_out = torch.full((self.total, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, va, **kw):
        args = dict(q_weight=self.qw, k_weight=self.kw, weight_offset=self.offset, eps=self.eps,
                    positions=self.positions if self.rot else None, rope_theta=self.theta, rotary_dim=self.rot or None,
                    interleaved=self.inter, k_scale=self.scales[0], v_scale=self.scales[1],
                    kv_layout="nhd" if self.nhd else "hnd", q_out=self.q_out, status=self.status)
        args.update(kw)
        return va.paged_qkv_append(self.q, self.k, self.v, self.dev["indptr"], self.dev["kvp"], self.dev["ids"],
                                   self.dev["last"], self.kc, self.vc, **args)

    def expect(self, freq=None):
        f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
        if freq is None:
            freq = float(np.float32(self.theta)) ** (-2.0 * np.arange(self.rot // 2) / max(1, self.rot))
        pos = self.positions.cpu().numpy() if self.rot else None
        a = (self.offset, float(np.float32(self.eps)), pos, freq, self.rot, self.inter)
        return (budget.prepare_heads(f(self.q), f(self.qw), *a), budget.prepare_heads(f(self.k), f(self.kw), *a),
                f(self.v))

    def check(self, skipped=(), freq=None):
        (q, qs), (k, ks), v = self.expect(freq)
        live = np.zeros(self.total, bool)
        live[:self.used] = True
        for i in skipped:
            live[i] = False
        got = self.q_out.double().cpu().numpy()
        assert np.all(got[~live] == 7.0)
        # fp32: the mean of squares, its root, the weight, the angle's sine and cosine
        # and the two products lose below 32 half steps of what is added; then one
        # rounding, half a step of bf16
        tol = 2.0 ** -8 * np.abs(q) + 32 * 2.0 ** -24 * qs + 1e-38
        assert np.all((np.abs(got - q) <= tol)[live]), np.abs((got - q) / tol)[live].max()
        want_k, want_v = self.k0.clone(), self.v0.clone()
        P = self.page
        for x, size, cache, raw, scale in ((k, ks, self.kc, want_k, self.scales[0]),
                                           (v, np.abs(v), self.vc, want_v, self.scales[1])):
            have = cache.cpu()
            hb = have.view(torch.uint8).numpy()
            touched = np.zeros(hb.shape[:3], bool)
            hv = have.float().double().numpy()
            for b, n in enumerate(self.lens):
                pages, slots = budget.slots_of(self.t["kvp"], self.t["ids"], self.t["last"], P, b)
                for u in range(n):
                    i = self.t["indptr"][b] + u
                    if not live[i]:
                        continue
                    page, slot = pages[self.pre[b] + u], slots[self.pre[b] + u]
                    at = (page, slot) if self.nhd else (page, slice(None), slot)
                    touched[at] = True
                    if self.fp8:
                        # the quotient rounds once more; half a step of e4m3, or of its subnormals
                        y = np.clip(x[i] / np.float64(np.float32(scale)), -448, 448)
                        tol = 2.0 ** -4 * np.abs(y) + 2.0 ** -10 + 34 * 2.0 ** -24 * size[i] / scale
                    else:
                        y, tol = x[i], 2.0 ** -8 * np.abs(x[i]) + 32 * 2.0 ** -24 * size[i] + 1e-38
                    if cache is self.vc and not self.fp8:
                        tol = 0.0
                    assert np.all(np.abs(hv[at] - y) <= tol)
            assert np.array_equal(hb[~touched], raw.numpy()[~touched])


CASES = [
    dict(lens=[1], pre=[0]),
    dict(lens=[1], pre=[4095], hq=32, h=8),
    dict(lens=[17], pre=[30], hq=32, h=8, weights="f32", offset=1.0),
    dict(lens=[3, 0, 8, 1], pre=[5, 9, 0, 31], hq=64, h=8, fp8=True, nhd=True),
    dict(lens=[5, 6], pre=[7, 8], d=64, hq=14, h=2, page=8, rot=32, inter=True, nhd=True, dv=128, fused=False),
    dict(lens=[40, 2], pre=[0, 1], d=64, hq=3, h=3, page=1, rot=16, weights=None),
    dict(lens=[9], pre=[2], rot=48, hq=5, h=1, page=256),
    dict(lens=[2, 2], pre=[1, 1], rot=0, hq=20, h=20, fused=False),
    dict(lens=[1, 70, 3], pre=[0, 0, 200], hq=48, h=24, dv=64, fp8=True, page=4),
    dict(lens=[4], pre=[0], hq=256, h=2),
    dict(lens=[6], pre=[3], far=2 ** 31 - 1, hq=16, h=2, inter=True),
    dict(lens=[1] * 300, pre=[3] * 300, hq=2, h=1, d=64),
    dict(lens=[5, 3], pre=[3, 0], hq=8, h=8, pad=11),
    # more tokens than CTAs: runs of tokens
    dict(lens=[700, 0, 1, 411], pre=[5, 0, 77, 0], hq=8, h=2, pad=9),
    dict(lens=[1500], pre=[0], hq=6, h=3, d=64, dv=128, fp8=True, nhd=True, rot=32, inter=True, weights="f32", offset=1.0),
    dict(lens=[460, 460], pre=[3, 0], hq=40, h=2, fused=False, page=64),
    dict(lens=[930], pre=[0], hq=128, h=8, page=32),
]


@pytest.mark.parametrize("n", range(len(CASES)))
def test_against_definition(va, n):
    c = Case(n, **CASES[n])
    out = c.run(va)
    assert out is c.q_out
    torch.cuda.synchronize()
    assert int(c.status) == 0
    c.check()


def test_one_side_normalised(va):
    c = Case(50, [4], [4])
    c.qw = None
    c.run(va)
    c.check()
    c = Case(51, [4], [4])
    c.kw = None
    c.run(va)
    c.check()


def test_inv_freq_replaces_the_formula(va):
    c = Case(52, [7], [20], far=131072)
    freq = 5e5 ** (-2.0 * np.arange(64) / 128) / np.where(np.arange(64) < 20, 1.0, 8.0)
    c.run(va, inv_freq=freq)
    c.check(freq=freq)


def test_same_as_append_where_both_apply(va):
    """Without weights the keys and values are those of paged_kv_append, bit for
    bit where no rotation rounds, and to one rounding where it does."""
    for fp8 in (False, True):
        c = Case(53, [6, 2], [11, 0], weights=None, rot=0, fused=False, fp8=fp8)
        c.run(va)
        k2 = c.k0.clone().cuda().view(c.kc.dtype)
        v2 = c.v0.clone().cuda().view(c.kc.dtype)
        va.paged_kv_append(c.k, c.v, c.dev["indptr"], c.dev["kvp"], c.dev["ids"], c.dev["last"], k2, v2,
                           k_scale=c.scales[0], v_scale=c.scales[1])
        assert torch.equal(k2.view(torch.uint8), c.kc.view(torch.uint8))
        assert torch.equal(v2.view(torch.uint8), c.vc.view(torch.uint8))
        assert torch.equal(c.q_out, c.q)


def test_in_place(va):
    c = Case(54, [9, 4], [1, 2], fused=False)
    (q, qs), _, _ = c.expect()
    c.q_out = c.q
    c.run(va)
    tol = 2.0 ** -8 * np.abs(q) + 32 * 2.0 ** -24 * qs + 1e-38
    assert np.all(np.abs(c.q_out.double().cpu().numpy() - q) <= tol)


def test_zero_and_special_rows(va):
    """An all-zero head stays zero with eps > 0; NaN and infinity stay in their head."""
    c = Case(55, [3], [0], hq=4, h=1)
    c.q[0, 1] = 0
    c.q[1, 2, 5] = float("nan")
    c.q[2, 0, 3] = float("inf")
    c.run(va)
    out = c.q_out
    assert bool((out[0, 1] == 0).all())
    assert bool(out[1, 2].isnan().all()) and not bool(out[1, [0, 1, 3]].isnan().any())
    assert bool(out[2, 0].isnan().any()) and not bool(out[2, 1:].isnan().any())


def test_bad_tables_skip_the_token(va):
    c = Case(56, [3, 4], [14, 0], page=16)
    c.dev["ids"][1] = 10 ** 6           # the page of request 0's position 16
    c.run(va)
    torch.cuda.synchronize()
    assert int(c.status) == 1
    c.check(skipped=[2])
    c = Case(57, [3, 4], [14, 0], page=16)
    c.dev["last"][1] = 17
    c.run(va)
    torch.cuda.synchronize()
    assert int(c.status) == 4
    c.check(skipped=[3, 4, 5, 6])


def test_graph_and_streams(va):
    c = Case(58, [5, 3], [3, 0], hq=8, h=2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.run(va)
    torch.cuda.current_stream().wait_stream(s)
    c.check()
    c = Case(59, [5, 3], [3, 0], hq=8, h=2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(va)
    c.q.mul_(0.5)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    c.check()


def test_far_slots(va):
    """Cache rows behind 2^31 elements."""
    pages = (1 << 31) // (16 * 128) // 2 + 40
    k = torch.zeros((pages, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q, kn, vn = (torch.randn((1, n, 128), device="cuda").to(torch.bfloat16) for n in (4, 2, 2))
    va.paged_qkv_append(q, kn, vn, i([0, 1]), i([0, 1]), i([pages - 1]), i([16]), k, v)
    assert torch.equal(k[pages - 1, :, 15], kn[0]) and torch.equal(v[pages - 1, :, 15], vn[0])
    assert int((k != 0).any(-1).sum()) == 2


@pytest.mark.parametrize("kw", [dict(lens=[3, 5, 0, 0, 0], pre=[40, 2, 0, 0, 0], pad=6),
                                dict(lens=[500, 300] + [0] * 140, pre=[40, 2] + [0] * 140, pad=30, fp8=True)])
def test_padded_batch(va, kw):
    """Requests of no pages and no tokens behind the last one, and rows behind the last token."""
    c = Case(40, **kw)
    c.q[c.used:] = float("nan")
    c.run(va)
    c.check()


def test_two_calls_at_once(va):
    cases = [Case(41, [700, 411], [5, 0], fp8=True), Case(42, [4, 1, 9], [5, 60, 0], hq=32, h=8)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                c.run(va)
    torch.cuda.synchronize()
    for c in cases:
        c.check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("lens, d, rot", [([3], 64, 32), ([2, 200], 128, 48), ([700, 411], 64, 16), ([640, 9], 128, 112)])
def test_special_values_past_the_rotation(va, lens, d, rot, inter, fp8):
    """Columns behind rotary_dim go as they are, whatever they hold: infinity and
    NaN reach neither their neighbours nor the columns that turn."""
    c = Case(60, lens, [5] * len(lens), hq=5, h=5, d=d, rot=rot, inter=inter, fp8=fp8, weights=None)
    gen = torch.Generator().manual_seed(61)
    for x in (c.q, c.k):
        at = torch.rand((c.total, 5, d - rot), generator=gen).cuda()
        for n, special in enumerate((float("inf"), -float("inf"), float("nan"), -0.0)):
            x[..., rot:][(at >= n / 16) & (at < (n + 1) / 16)] = special
    c.run(va)
    torch.cuda.synchronize()
    assert int(c.status) == 0
    same = lambda a, b: bool(((a == b) | (a.isnan() & b.isnan())).all())  # noqa: E731
    assert same(c.q_out[..., rot:], c.q[..., rot:])
    assert bool(c.q_out[..., :rot].isfinite().all())
    # the keys: as the append without rotation stores them, bit for bit but for NaN
    k2, v2 = (x.clone().cuda().view(c.kc.dtype) for x in (c.k0, c.v0))
    va.paged_kv_append(c.k.contiguous(), c.v.contiguous(), c.dev["indptr"], c.dev["kvp"], c.dev["ids"], c.dev["last"],
                       k2, v2, k_scale=c.scales[0], v_scale=c.scales[1])
    for b, n in enumerate(lens):
        pages, slots = (torch.from_numpy(x[5:]).cuda().long() for x in budget.slots_of(c.t["kvp"], c.t["ids"], c.t["last"], c.page, b))
        got, want = c.kc[pages, :, slots].float(), k2[pages, :, slots].float()
        assert same(got[..., rot:], want[..., rot:])
        assert bool(got[..., :rot].isfinite().all())
        assert torch.equal(torch.signbit(got[..., rot:]) | got[..., rot:].isnan(), torch.signbit(want[..., rot:]) | want[..., rot:].isnan())


def test_same_as_the_rotating_append(va):
    """Without weights the rotated keys are paged_kv_append's at the same positions,
    up to what both may lose: the angle and its sine and cosine (32 half steps of
    fp32 of what is added, the tolerance against the definition, in either), and
    half a step of bf16 or e4m3 in either."""
    for fp8 in (False, True):
        for nhd in (False, True):
            c = Case(62, [6, 2, 90], [11, 0, 300], weights=None, fused=False, fp8=fp8, nhd=nhd, far=8191)
            c.run(va)
            k2, v2 = (x.clone().cuda().view(c.kc.dtype) for x in (c.k0, c.v0))
            va.paged_kv_append(c.k, c.v, c.dev["indptr"], c.dev["kvp"], c.dev["ids"], c.dev["last"], k2, v2,
                               k_scale=c.scales[0], v_scale=c.scales[1], kv_layout="nhd" if nhd else "hnd",
                               positions=c.positions, rope_theta=c.theta)
            assert torch.equal(v2.view(torch.uint8), c.vc.view(torch.uint8))
            _, (k, size), _ = c.expect()
            for b, n in enumerate(c.lens):
                pages, slots = budget.slots_of(c.t["kvp"], c.t["ids"], c.t["last"], c.page, b)
                new = slice(c.pre[b], c.pre[b] + n)
                rows = slice(int(c.t["indptr"][b]), int(c.t["indptr"][b]) + n)
                pages, slots = (torch.from_numpy(x[new]).cuda().long() for x in (pages, slots))
                a, e = ((x[pages, slots] if nhd else x[pages, :, slots]).float().double().cpu().numpy() for x in (c.kc, k2))
                if fp8:
                    y = np.clip(k[rows] / np.float64(np.float32(c.scales[0])), -448, 448)
                    tol = 2 * (2.0 ** -4 * np.abs(y) + 2.0 ** -10 + 34 * 2.0 ** -24 * size[rows] / c.scales[0])
                else:
                    tol = 2 * (2.0 ** -8 * np.abs(k[rows]) + 32 * 2.0 ** -24 * size[rows] + 1e-38)
                assert np.all(np.abs(a - e) <= tol)
            free = torch.ones(c.kc.shape[:3], dtype=torch.bool, device="cuda")
            for b, n in enumerate(c.lens):
                pages, slots = budget.slots_of(c.t["kvp"], c.t["ids"], c.t["last"], c.page, b)
                pages, slots = (torch.from_numpy(x[c.pre[b]:]).cuda().long() for x in (pages, slots))
                free[(pages, slots) if nhd else (pages, slice(None), slots)] = False
            assert torch.equal(k2.view(torch.uint8)[free], c.kc.view(torch.uint8)[free])
