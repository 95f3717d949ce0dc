"""GPU test of paged_kv_evict against a host copy of all three pools: the
survivors at the front in their order bit for bit, every other slot as it was."""
import numpy as np
import pytest
import torch

from evict_modes import shapes
from oracle import budget

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def va():
    import __graft_entry__
    __graft_entry__.build()
    import speculative_decoding_verify_gqa_gb300 as m
    return m


class Case:
    def __init__(self, seed, lens, keep, sinks=0, recent=0, page=16, h=2, d=64, dv=None, fp8=False, nhd=False,
                 layers=None, values="spread"):
        rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 2
        self.ids = rng.permutation(pages)[:max(1, sum(need))].astype(np.int32)
        self.kvp = np.concatenate([[0], np.cumsum(need)]).astype(np.int32)
        self.last = np.array([(n - 1) % page + 1 if n else 0 for n in lens], np.int32)
        self.keep = np.array(keep, np.int32)
        self.lens, self.sinks, self.recent, self.page, self.nhd, self.layers = lens, sinks, recent, page, nhd, layers
        mid = (page, h) if nhd else (h, page)
        shape = (() if layers is None else (layers,)) + (pages,) + mid
        es = 1 if fp8 else 2
        self.k, self.v = (rng.integers(0, 256, shape + (w * es,), dtype=np.uint8) for w in (d, dv or d))
        w = rng.lognormal(0, 2, shape)
        if values == "equal":
            w[:] = 1.5
        elif values == "few":
            w = rng.integers(0, 4, shape) * 0.25 - 0.25
            w[w == 0] *= rng.choice([-1.0, 1.0], w[w == 0].shape)     # -0 equals 0
        elif values == "special":
            pick = rng.integers(0, 8, shape)
            w = np.select([pick == 0, pick == 1, pick == 2, pick == 3], [np.nan, np.inf, -np.inf, -w], w)
        elif values == "close":
            w = (1 + rng.integers(0, 3000, shape) * 2.0 ** -23)
        self.w = w.astype(np.float32)
        self.dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
        t = lambda x: torch.from_numpy(x.copy()).cuda()  # noqa: E731
        self.dev = dict(w=t(self.w), keep=t(self.keep), kvp=t(self.kvp), ids=t(self.ids), last=t(self.last),
                        k=t(self.k).view(self.dt), v=t(self.v).view(self.dt))
        self.kv_len = torch.full((len(lens),), -7, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, va, **kw):
        x = self.dev
        args = dict(sinks=self.sinks, recent=self.recent, kv_layout="nhd" if self.nhd else "hnd",
                    kv_len_out=self.kv_len, status=self.status)
        args.update(kw)
        va.paged_kv_evict(x["w"], x["keep"], x["kvp"], x["ids"], x["last"], x["k"], x["v"], **args)

    def expect(self, skip=()):
        out = []
        w5 = self.w if self.layers is not None else self.w[None]
        moves = []
        for layer in range(w5.shape[0]):
            for b in range(len(self.lens)):
                if b in skip:
                    continue
                pages, slots = budget.slots_of(self.kvp, self.ids, self.last, self.page, b)
                for h in range(w5.shape[2] if not self.nhd else w5.shape[3]):
                    at = [(layer, p, s, h) if self.nhd else (layer, p, h, s) for p, s in zip(pages, slots)]
                    rows = budget.survivors(np.array([w5[a] for a in at]), int(self.keep[b]), self.sinks, self.recent)
                    moves += [(at[j], at[i]) for i, j in enumerate(rows)]
        for x in (self.k, self.v, self.w):
            y = x.copy()
            x5, y5 = (x, y) if self.layers is not None else (x[None], y[None])
            for s, d in moves:
                y5[d] = x5[s]
            out.append(y)
        return out

    def check(self, skip=(), status=0):
        torch.cuda.synchronize()
        assert int(self.status) == status
        k, v, w = self.expect(skip)
        assert np.array_equal(self.dev["k"].view(torch.uint8).cpu().numpy(), k)
        assert np.array_equal(self.dev["v"].view(torch.uint8).cpu().numpy(), v)
        assert np.array_equal(self.dev["w"].cpu().numpy().view(np.uint32), w.view(np.uint32))
        want = [n if b in skip else min(n, int(c)) for b, (n, c) in enumerate(zip(self.lens, self.keep))]
        assert self.kv_len.tolist() == want


CASES = [
    dict(lens=[100], keep=[50]),
    dict(lens=[1], keep=[1]),
    dict(lens=[1, 0, 2], keep=[0, 0, 1]),
    dict(lens=[33, 700, 64, 5], keep=[32, 100, 64, 9], sinks=4, recent=16, h=3),
    dict(lens=[257, 31], keep=[128, 30], sinks=1, recent=300, page=1, nhd=True, d=128),
    dict(lens=[513], keep=[3], sinks=4, recent=4),
    dict(lens=[513], keep=[6], sinks=4, recent=4),
    dict(lens=[2000, 900], keep=[1999, 1], page=32, fp8=True, nhd=True, d=128, dv=64, layers=2),
    dict(lens=[300], keep=[100], values="equal", sinks=3),
    dict(lens=[1000, 450], keep=[333, 200], values="few", recent=7, page=8),
    dict(lens=[1000, 450], keep=[400, 100], values="special", sinks=2, recent=7, page=64),
    dict(lens=[1200], keep=[600], values="close", h=1, d=128, fp8=True),
    dict(lens=[40] * 40, keep=[13] * 40, layers=3, h=2),
    dict(lens=[3000], keep=[0]),
    dict(lens=[9000], keep=[4500], sinks=4, recent=100, h=1, page=128),
    # longer than what every CTA of a cluster ranks by itself
    dict(lens=[20001, 300], keep=[5000, 250], sinks=4, recent=100, h=1, d=64),
    dict(lens=[17000], keep=[9000], h=2, d=64, values="equal", nhd=True, page=8),
    dict(lens=[18500], keep=[6000], h=1, d=64, values="few", recent=33),
    dict(lens=[16500], keep=[12000], h=1, d=128, values="special", fp8=True),
    dict(lens=[30000], keep=[100], h=1, d=64, values="close", sinks=1),
    # many units: one CTA each
    dict(lens=[70, 50] * 40, keep=[30, 45] * 40, layers=4, h=2, d=64, values="few", recent=3),
]


@pytest.mark.parametrize("n", range(len(CASES)))
def test_against_definition(va, n):
    c = Case(n, **CASES[n])
    c.run(va)
    c.check()


def test_skipped_requests(va):
    """Lengths past max_kv_len, bad pages and bad tables leave their request alone."""
    c = Case(100, [90, 300, 40], [20, 20, 20])
    c.run(va, max_kv_len=299)
    c.check(skip=[1], status=2)
    c = Case(101, [90, 300, 40], [20, 20, 20])
    c.dev["ids"][int(c.kvp[1])] = -1
    c.run(va)
    c.check(skip=[1], status=1)
    c = Case(102, [90, 300, 40], [20, 20, 20])
    c.dev["keep"][2] = -1
    c.run(va)
    c.check(skip=[2], status=2)


def test_twice_and_graph(va):
    """A graph captured over one pool, replayed after the tables have moved on."""
    c = Case(103, [400, 77], [200, 50], sinks=2, recent=8)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(va, max_kv_len=1000)
    g.replay()
    c.check()
    k, v, w = c.expect()
    c.k, c.v, c.w = k, v, w
    c.lens, c.keep = [200, 50], np.array([60, 50], np.int32)
    page = c.page
    # the same pages listed, fewer keys: pages past the new length are dropped
    need = [-(-n // page) for n in c.lens]
    c.ids = np.concatenate([c.ids[c.kvp[b]:c.kvp[b] + need[b]] for b in range(2)]).astype(np.int32)
    c.kvp = np.concatenate([[0], np.cumsum(need)]).astype(np.int32)
    c.last = np.array([(n - 1) % page + 1 for n in c.lens], np.int32)
    c.dev["ids"][:len(c.ids)] = torch.from_numpy(c.ids)
    for n in ("kvp", "last", "keep"):
        c.dev[n].copy_(torch.from_numpy(getattr(c, n)))
    g.replay()
    c.check()


def test_longer_than_shared_memory_holds(va):
    """Slices that are read from the cache in every pass: 310,000 keys with the largest bound."""
    c = Case(104, [310000], [200000], sinks=3, recent=1000, h=1, d=64, fp8=True, page=256)
    c.run(va, max_kv_len=1 << 19)
    c.check()


def test_far_rows(va):
    """Rows of the last layer lie behind 2^31 bytes and 2^31 elements."""
    layers, pages, h, P, d = 3, 45000, 2, 64, 128
    k = torch.zeros((layers, pages, h, P, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    w = torch.zeros((layers, pages, h, P), device="cuda")
    at = pages - 2
    row = torch.arange(P, device="cuda").float()
    k[2, at] = row[:, None].to(torch.bfloat16)
    v[2, at] = -row[:, None].to(torch.bfloat16)
    w[2, at] = row % 7
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    va.paged_kv_evict(w, i([20]), i([0, 1]), i([at]), i([P]), k, v)
    rows = budget.survivors((np.arange(P) % 7).astype(np.float32), 20, 0, 0)
    for x, sign in ((k, 1), (v, -1)):
        assert x[2, at, 0, :20, 0].float().tolist() == [float(sign * r) for r in rows]
        assert x[2, at, 1, 20:, 5].float().tolist() == [float(sign * r) for r in range(20, P)]
        assert int((x[1] != 0).any()) == 0


def test_padded_batch(va):
    """Requests of no pages behind the last one: their new length is 0, whatever they may keep."""
    c = Case(90, [900, 40, 0, 0, 0], [300, 17, 0, 5, 1 << 30], sinks=2, recent=9, layers=2)
    c.run(va)
    c.check()


def test_two_calls_at_once(va):
    cases = [Case(91, [3000, 1200], [1500, 60], h=4, d=128, layers=3), Case(92, [20001], [5000], h=1, values="few", recent=5)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for c, s in zip(cases, streams):
        with torch.cuda.stream(s):
            c.run(va)
    for c in cases:
        c.check()


class Long(Case):
    """A case of long requests: the moves of a request, layer and head are made together."""

    def expect(self, skip=()):
        w5 = self.w if self.layers is not None else self.w[None]
        out = [x.copy() for x in (self.k, self.v, self.w)]
        for b in range(len(self.lens)):
            pages, slots = budget.slots_of(self.kvp, self.ids, self.last, self.page, b)
            for layer in range(w5.shape[0]):
                for h in range(w5.shape[3] if self.nhd else w5.shape[2]):
                    at = (lambda r: (layer, pages[r], slots[r], h)) if self.nhd else (lambda r: (layer, pages[r], h, slots[r]))  # noqa: E731
                    rows = np.array(budget.survivors(w5[at(slice(None))], int(self.keep[b]), self.sinks, self.recent), int)
                    for x, y in zip((self.k, self.v, self.w), out):
                        x5, y5 = (x, y) if self.layers is not None else (x[None], y[None])
                        y5[at(slice(0, len(rows)))] = x5[at(rows)]
        return out

    def run_on(self, va, num_sms, max_kv_len):
        """The call with a number of SMs of the caller's, which bounds the CTAs that share a request."""
        x, dims = self.dev, self.dev["k"].shape[-4:]
        page, h = (dims[1], dims[2]) if self.nhd else (dims[2], dims[1])
        p = lambda t: t.data_ptr()  # noqa: E731
        rc = va.lib().paged_kv_evict(
            p(x["w"]), p(x["keep"]), p(x["kvp"]), p(x["ids"]), p(x["last"]), p(x["k"]), p(x["v"]), self.layers or 1,
            len(self.lens), h, dims[3], x["v"].shape[-1], page, dims[0],
            va.KV_FP8_E4M3 if self.dt is torch.float8_e4m3fn else va.KV_BF16, 1 if self.nhd else 0, max_kv_len, self.sinks,
            self.recent, p(self.kv_len), p(self.status), num_sms, torch.cuda.current_stream().cuda_stream)
        assert rc == 0


# What a CTA holds of its weights: all of them, their upper halves, or none; by one
# CTA a unit, and by two, four and eight.  (case, SMs, max_kv_len: None the
# longest request's, CTAs a unit, mode)
HELD = [
    (dict(lens=[20000], keep=[7001], sinks=5, recent=77, h=1), 1, None, 1, "halves"),
    (dict(lens=[20000], keep=[7001], sinks=5, recent=77, h=1, values="close"), 1, None, 1, "halves"),
    (dict(lens=[16385], keep=[16000], sinks=1, h=1, values="equal", nhd=True, page=1, fp8=True), 1, None, 1, "halves"),
    (dict(lens=[17001, 300, 0, 16500], keep=[4003, 299, 0, 16499], sinks=33, recent=3, h=3, values="few", nhd=True, fp8=True), 12, None, 1, "halves"),
    (dict(lens=[16401], keep=[555], recent=50, h=1, values="special", page=256), 1, None, 1, "halves"),
    (dict(lens=[18000], keep=[60], sinks=9, recent=51, h=1, values="few"), 1, None, 1, "halves"),      # no key competes for a place
    (dict(lens=[18000], keep=[17990], sinks=9000, recent=8995, h=1, values="close"), 1, None, 1, "halves"),   # none between the ends
    (dict(lens=[40000, 33001], keep=[9999, 32990], sinks=3, recent=1001, h=1, d=128, values="close", page=64), 4, None, 2, "halves"),
    (dict(lens=[40001], keep=[20000], sinks=13, recent=100, h=1, values="few", fp8=True, nhd=True), 2, None, 2, "halves"),
    (dict(lens=[33333], keep=[11111], h=2, values="equal", recent=7), 4, None, 2, "halves"),
    (dict(lens=[35007], keep=[30000], h=1, values="special", sinks=17, nhd=True, page=32), 2, None, 2, "halves"),
    (dict(lens=[70001], keep=[33333], sinks=4, recent=37, h=1, d=128, values="close", page=128), 4, None, 4, "halves"),
    (dict(lens=[140003], keep=[70001], sinks=4, recent=37, h=1, d=128, values="few", page=128), 8, None, 8, "halves"),
    (dict(lens=[140003], keep=[139000], sinks=1, h=1, d=64, values="close", page=256), 8, None, 4, "halves"),
    # ranked whole by every CTA, from upper halves: short requests in a batch of long ones
    (dict(lens=[12001], keep=[6000], sinks=3, recent=40, h=1, values="close"), 1, 16500, 1, "halves"),
    (dict(lens=[15000, 9000], keep=[1000, 8999], sinks=3, recent=40, h=1, values="few"), 4, 33000, 2, "halves"),
    (dict(lens=[16384], keep=[9000], sinks=3, h=1, d=128, values="special", nhd=True), 8, 140000, 8, "halves"),
    # more room than keys: whole weights of more than a CTA of a cluster ranks by itself
    (dict(lens=[18000], keep=[6000], h=1, values="close", recent=5), 1, 1 << 19, 1, "whole"),
    (dict(lens=[30000], keep=[6000], h=1, values="special", recent=5, sinks=2), 2, 1 << 19, 2, "whole"),
    # more keys than room
    (dict(lens=[38001], keep=[16001], h=1, values="few", recent=5, sinks=2), 1, 1 << 19, 1, "reread"),
    (dict(lens=[38001], keep=[30000], h=1, values="close", nhd=True, fp8=True), 1, 1 << 19, 1, "reread"),
    (dict(lens=[75500], keep=[7000], h=1, values="special", sinks=40, d=128), 2, 1 << 19, 2, "reread"),
    (dict(lens=[75001], keep=[74000], h=1, values="equal", sinks=4, recent=99, page=64), 2, 1 << 19, 2, "reread"),
]


@pytest.mark.parametrize("n", range(len(HELD)))
def test_each_way_to_hold_the_weights(va, tmp_path, n):
    case, sms, most, cluster, mode = HELD[n]
    c = Long(200 + n, **case)
    most = most or max(c.lens)
    units = (c.layers or 1) * len(c.lens) * case["h"]
    chunks = (c.k.shape[-1] + c.v.shape[-1]) // 16
    got = shapes(tmp_path, [(units, chunks, sms, most, max(c.lens))])[0]
    assert (got[0], got[3]) == (cluster, mode)
    c.run_on(va, sms, most)
    c.check()


def test_upper_halves_of_many_units(va, tmp_path):
    """The binding's own call: more units than half the SMs, one CTA each."""
    sms = va.num_sms()
    layers = sms // 16 + 1
    c = Long(230, [17500, 16390], [9001, 16389], sinks=3, recent=45, h=8, d=64, fp8=True, nhd=True, layers=layers, values="close")
    got = shapes(tmp_path, [(layers * 2 * 8, 8, sms, 17500, n) for n in c.lens])
    assert [(g[0], g[3]) for g in got] == [(1, "halves")] * 2
    c.run(va, max_kv_len=17500)
    c.check()
