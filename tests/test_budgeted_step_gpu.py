"""A decoding loop over a cache with a budget: projection rows -> norm, rotation
and append -> attention over draft trees -> acceptance -> attention weights of
the accepted path -> compaction -> eviction -> next step.  The host follows every
key of every request and KV head through the moves and compares the cache's live
slots bit for bit, the weights within their bound and the attention with dense
attention over the keys that should be left."""
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


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


class Loop:
    B, P, SINKS, RECENT, KEEP = 3, 16, 2, 8, 60

    def __init__(self, va, fp8, nhd, d, seed):
        self.va, self.fp8, self.nhd, self.d = va, fp8, nhd, d
        self.hq, self.h = 8, 2
        self.rng = np.random.default_rng(seed)
        self.g = torch.Generator().manual_seed(seed)
        self.pages = 64
        mid = (self.P, self.h) if nhd else (self.h, self.P)
        dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
        raw = torch.full((self.pages,) + mid + (d * (1 if fp8 else 2),), 0xFF, dtype=torch.uint8, device="cuda")
        self.k, self.v = raw.clone().view(dt), raw.clone().view(dt)
        self.w = torch.full((self.pages,) + mid, float("nan"), device="cuda")
        self.scale = 0.02 if fp8 else 1.0
        self.free = list(self.rng.permutation(self.pages))
        self.table = [[] for _ in range(self.B)]
        self.len = [0] * self.B
        self.pos = [0] * self.B                       # positions go on counting
        self.qw, self.kw = ((torch.rand(d, generator=self.g) + 0.5).cuda() for _ in range(2))
        # what should be there: [request][head] -> raw K rows, raw V rows, weights
        self.have = [[(np.zeros((0, d * (1 if fp8 else 2)), np.uint8),) * 2 + (np.zeros(0),) for _ in range(self.h)]
                     for _ in range(self.B)]
        self.layout = "nhd" if nhd else "hnd"
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def tables(self):
        kvp = np.concatenate([[0], np.cumsum([len(t) for t in self.table])])
        ids = np.concatenate([np.asarray(t, np.int32) for t in self.table] + [np.zeros(1, np.int32)])
        last = [(n - 1) % self.P + 1 if n else 0 for n in self.len]
        return kvp.astype(np.int32), ids.astype(np.int32), np.asarray(last, np.int32)

    def rows(self, cache, b, n):
        """The first n rows of request b per head: [h, n, ...] (numpy)."""
        j = np.arange(n)
        page, slot = np.asarray(self.table[b], int)[j // self.P], j % self.P
        x = cache.cpu().numpy()
        return x[page, slot].swapaxes(0, 1) if self.nhd else x[page, :, slot].swapaxes(0, 1)

    def step(self, nodes, tree):
        va, B, d, rng = self.va, self.B, self.d, self.rng
        pre = list(self.len)
        for b in range(B):
            self.len[b] += nodes[b]
            while len(self.table[b]) * self.P < self.len[b]:
                self.table[b].append(self.free.pop())
        kvp, ids, last = self.tables()
        qo = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        total = int(qo[-1])
        rows = torch.randn((total, (self.hq + 2 * self.h) * d), generator=self.g).to(torch.bfloat16).cuda()
        q, k, v = rows.split([self.hq * d, self.h * d, self.h * d], 1)
        q, k, v = q.view(total, self.hq, d), k.view(total, self.h, d), v.view(total, self.h, d)
        parents, depth, bits = [], [], []
        for n in nodes:
            par = [-1] + [int(rng.integers(0, i)) if tree else i - 1 for i in range(1, n)]
            seen = np.zeros((n, n), bool)
            dep = []
            for i, p in enumerate(par):
                if p >= 0:
                    seen[i] = seen[p]
                seen[i, i] = True
                dep.append(dep[p] + 1 if p >= 0 else 0)
            parents += par
            depth.append(dep)
            bits.append(seen)
        flat = np.concatenate([s.reshape(-1) for s in bits])
        mask = torch.from_numpy(np.packbits(np.concatenate([flat, np.zeros(8, bool)]), bitorder="little")).cuda()
        mip = np.concatenate([[0], np.cumsum([n * n for n in nodes])]).astype(np.int32)
        positions = np.concatenate([self.pos[b] + np.asarray(depth[b]) for b in range(B)]).astype(np.int32)
        t = dict(kvp=_i32(kvp), ids=_i32(ids), last=_i32(last), qo=_i32(qo))
        scales = dict(k_scale=self.scale, v_scale=self.scale) if self.fp8 else {}
        qr = va.paged_qkv_append(q, k, v, t["qo"], t["kvp"], t["ids"], t["last"], self.k, self.v, q_weight=self.qw,
                                 k_weight=self.kw, positions=_i32(positions), kv_layout=self.layout, status=self.status,
                                 **scales)
        # the new rows against the definition; from here on their bits are what should be there
        freq = 10000.0 ** (-2.0 * np.arange(d // 2) / d)
        f = lambda x: x.double().cpu().numpy()  # noqa: E731
        want_k, size = budget.prepare_heads(f(k), f(self.kw), 0.0, float(np.float32(1e-6)), positions, freq, d, False)
        kc, vc = self.k.view(torch.uint8), self.v.view(torch.uint8)
        val = lambda raw: torch.from_numpy(np.ascontiguousarray(raw)).view(self.k.dtype).float().double().numpy()  # noqa: E731
        for b in range(B):
            kr, vr = self.rows(kc, b, self.len[b]), self.rows(vc, b, self.len[b])
            for h in range(self.h):
                new = val(kr[h, pre[b]:])
                y = want_k[qo[b]:qo[b + 1], h] / float(np.float32(self.scale))
                step = 2.0 ** -4 * np.abs(y) + 2.0 ** -10 if self.fp8 else 2.0 ** -8 * np.abs(y)
                assert np.all(np.abs(new - y) <= step + 40 * 2.0 ** -24 * size[qo[b]:qo[b + 1], h] / self.scale)
                ok, ov, ow = self.have[b][h]
                assert np.array_equal(kr[h, :pre[b]], ok) and np.array_equal(vr[h, :pre[b]], ov)
                self.have[b][h] = (kr[h], vr[h], ow)
        # attention over what is left
        plan = va.verify_attn_plan(kvp, qo, last, mip, self.hq, self.h, d, self.P,
                                   kv_dtype="fp8_e4m3" if self.fp8 else "bf16", kv_layout=self.layout)
        out, lse = va.verify_attn_run(qr, self.k, self.v, t["kvp"], t["ids"], t["last"], t["qo"], mask, _i32(mip), plan,
                                      k_scale=self.scale, v_scale=self.scale)
        G = self.hq // self.h
        seen_all = []
        for b in range(B):
            n, m = nodes[b], self.len[b]
            seen = np.ones((n, m), bool)
            seen[:, m - n:] = bits[b]
            seen_all.append(seen)
            for h in range(self.h):
                kk, vv = val(self.have[b][h][0]) * self.scale, val(self.have[b][h][1]) * self.scale
                s = np.einsum("ngd,md->ngm", f(qr)[qo[b]:qo[b + 1], h * G:(h + 1) * G], kk) / math.sqrt(d)
                s = np.where(seen[:, None], s, -np.inf)
                e = np.exp(s - s.max(-1, keepdims=True))
                o = np.einsum("ngm,md->ngd", e / e.sum(-1, keepdims=True), vv)
                err = np.abs(f(out)[qo[b]:qo[b + 1], h * G:(h + 1) * G] - o)
                assert np.all(err <= 1e-2 + 2.0 ** -8 * np.abs(o))
        # acceptance: the target's argmax follows a drawn root path
        vocab = 64
        draft = rng.integers(0, vocab, total)
        logits = torch.randn((total, vocab), generator=self.g)
        for b in range(B):
            v0 = int(rng.integers(0, nodes[b]))
            path = [i for i in range(nodes[b]) if bits[b][v0, i]]
            for a, c in zip(path, path[1:]):
                logits[qo[b] + a, draft[qo[b] + c]] = 100.0
        acc, path, _, _ = va.verify_accept_greedy(logits.cuda(), t["qo"], _i32(draft), _i32(parents))
        # weights of the accepted path, then its keys to the front
        va.verify_attn_key_weights(qr, self.k, t["kvp"], t["ids"], t["last"], t["qo"], lse, self.w, accept_len=acc,
                                   accepted_nodes=path, k_scale=self.scale, decay=0.9, kv_layout=self.layout,
                                   status=self.status)
        va.paged_kv_compact(acc, path, t["qo"], t["kvp"], t["ids"], t["last"], self.k, self.v, kv_layout=self.layout,
                            status=self.status)
        acc, path, lse = acc.tolist(), path.tolist(), lse.cpu().numpy()
        for b in range(B):
            nodes_b = path[qo[b]:qo[b] + acc[b]]
            self.len[b] = pre[b] + acc[b]
            self.pos[b] += acc[b]
            keys = list(range(pre[b])) + [pre[b] + i for i in nodes_b]
            got = self.rows(self.w, b, self.len[b])
            kk = np.stack([val(self.have[b][h][0]) for h in range(self.h)], 1)
            for h in range(self.h):
                ok, ov, ow = self.have[b][h]
                self.have[b][h] = (ok[keys], ov[keys], got[h])
            w, loss = budget.key_weights(f(qr)[qo[b]:qo[b + 1]], kk, lse[qo[b]:qo[b + 1]], seen_all[b],
                                         self.scale / math.sqrt(d), nodes_b)
            old = np.stack([np.concatenate([self.w_before[b][h][:pre[b]], np.zeros(acc[b])]) for h in range(self.h)], 1) \
                if self.w_before else np.zeros_like(w)
            want = w + old * float(np.float32(0.9))
            assert np.all(np.abs(got.T - want) <= loss + 2.0 ** -22 * want)
        self.check_live()
        # over the budget: pages behind the survivors are free again
        kvp, ids, last = self.tables_of(self.len)
        keep = _i32([self.KEEP] * B)
        kv_len = torch.empty(B, dtype=torch.int32, device="cuda")
        va.paged_kv_evict(self.w, keep, _i32(kvp), _i32(ids), _i32(last), self.k, self.v, sinks=self.SINKS,
                          recent=self.RECENT, kv_layout=self.layout, kv_len_out=kv_len, status=self.status)
        for b in range(B):
            for h in range(self.h):
                ok, ov, ow = self.have[b][h]
                stay = budget.survivors(ow, self.KEEP, self.SINKS, self.RECENT)
                self.have[b][h] = (ok[stay], ov[stay], ow[stay])
            self.len[b] = min(self.len[b], self.KEEP)
            used = -(-self.len[b] // self.P)
            self.free += self.table[b][used:]
            self.table[b] = self.table[b][:used]
        assert kv_len.tolist() == self.len
        self.check_live()
        self.w_before = [[self.have[b][h][2] for h in range(self.h)] for b in range(B)]
        assert int(self.status) == 0

    w_before = None

    def tables_of(self, lens):
        """Tables that list only the pages that `lens` keys fill."""
        used = [t[:-(-n // self.P)] for t, n in zip(self.table, lens)]
        for b, t in enumerate(used):
            self.free += self.table[b][len(t):]
            self.table[b] = t
        return self.tables()

    def check_live(self):
        kc, vc = self.k.view(torch.uint8), self.v.view(torch.uint8)
        for b in range(self.B):
            kr, vr, wr = (self.rows(x, b, self.len[b]) for x in (kc, vc, self.w))
            for h in range(self.h):
                ok, ov, ow = self.have[b][h]
                assert np.array_equal(kr[h], ok) and np.array_equal(vr[h], ov)
                assert np.array_equal(wr[h].view(np.uint32), np.asarray(ow, np.float32).view(np.uint32))


@pytest.mark.parametrize("fp8, nhd, d, tree", [(False, False, 128, True), (True, True, 128, True),
                                               (False, True, 64, False), (True, False, 64, True)])
def test_loop(va, fp8, nhd, d, tree):
    loop = Loop(va, fp8, nhd, d, seed=11 + d)
    loop.step([40, 55, 9], tree=False)      # the prompts, as chains that are accepted as far as the draw goes
    for n in range(7):
        loop.step([int(x) for x in loop.rng.integers(1, 18, 3)], tree)
    assert max(loop.len) <= loop.KEEP
