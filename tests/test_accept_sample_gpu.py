"""GPU parity of sampled acceptance (verify_accept_sample) with the 64-bit
oracle.  Lengths, paths and tokens are compared exactly: every case's
decisions lie further from their borders (the oracle's margin) than the
kernel's arithmetic can move them.

That arithmetic: a weight 2^((x - m) log2(e) / T) has a relative error below
2^-22 (the exponential instruction) + ln 2 * |exponent| * 2^-23 (its argument:
one subtraction, one product), under 3e-6 for exponents above -32, and weights
below 2^-32 carry less than 2^-32 * vocab <= 2^-14 of a sum at most where the
row's maximum is 1 -- their own relative error (at most 1.3e-5 at 2^-126) is
that share smaller.  A thread's fp32 sum of at most 2^8 weights adds 2^8 *
2^-24 = 1.6e-5 at worst; everything past it is fp64.  So probabilities, sums
and A, B are within 2.5e-5, and log-probabilities too.
"""
import numpy as np
import pytest
import torch

from oracle.accept_sample import accept_sampled

pytestmark = pytest.mark.gpu

MARGIN = 1e-4
LOGP_TOL = 2.5e-5


@pytest.fixture(scope="module")
def va():
    import __graft_entry__
    __graft_entry__.build()
    import speculative_decoding_verify_gqa_gb300 as m
    return m


def _parents(lens, kind, rng):
    out = []
    for n in lens:
        if n:
            out += [-1] + [i - 1 if kind == "chain" else 0 if kind == "star" else int(rng.integers(0, i))
                           for i in range(1, n)]
    return np.array(out, np.int32)


def _inputs(seed, lens, vocab, kind="tree", ldt=torch.bfloat16, qdt=None, temps=None, masked=0.0, spread=2.0,
            pad=0, u_min=0.0, u_max=1.0, near=0.5, greedy_drafts=False):
    """Peaked logits (a few hot tokens a row), drafts sampled from the draft
    distribution, or, without one, the likeliest tokens (repeats among them)."""
    rng = np.random.default_rng(seed)
    total, B = int(sum(lens)), len(lens)
    lg = rng.standard_normal((total, vocab + pad)) * spread
    for i in range(total):
        hot = rng.integers(0, vocab, 6)
        lg[i, hot] += np.log(vocab) + rng.standard_normal(6)
    if masked:
        keep = rng.random((total, vocab + pad)) >= masked
        keep[:, rng.integers(0, vocab, 3)] = True
        lg = np.where(keep, lg, -np.inf)
    lg = torch.from_numpy(lg).to(ldt)
    host = lg.double().numpy()[:, :vocab]
    indptr = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    par = _parents(lens, kind, rng)
    req = np.repeat(np.arange(B), lens)
    t = None if temps is None else np.array([temps[b % len(temps)] for b in range(B)], np.float32)
    x = host / np.maximum(np.ones(total) if t is None else t[req], 0.3)[:, None] + rng.standard_normal((total, vocab)) * near
    x = np.exp(x - x.max(1, keepdims=True))
    q = x / x.sum(1, keepdims=True)
    rows = np.array([indptr[req[i]] + max(int(par[i]), 0) for i in range(total)], np.int64)
    if qdt is None:
        top = np.argsort(-q, axis=1, kind="stable")[:, :4]
        toks = np.array([top[rows[i], int(rng.integers(0, top.shape[1]))] for i in range(total)], np.int32)
        dp = dp_host = None
    else:
        toks = (q[rows] / rng.exponential(size=(total, vocab))).argmax(1).astype(np.int32) if total else np.zeros(0, np.int32)
        dp = torch.from_numpy(np.concatenate([q, np.full((total, pad), np.nan)], 1)).to(qdt)
        dp_host = dp.double().numpy()[:, :vocab]
    if greedy_drafts:
        toks = host[rows].argmax(1).astype(np.int32)
    u = (u_min + (u_max - u_min) * rng.random(total)).astype(np.float32)
    u = np.minimum(u, np.float32(1 - 2.0 ** -24))
    noise = rng.exponential(size=(B, vocab + pad)).astype(np.float32)
    return dict(lg=lg, host=host, indptr=indptr, par=par, toks=toks, u=u, noise=noise, t=t, dp=dp, dp_host=dp_host,
                vocab=vocab)


def _ref(c):
    return accept_sampled(c["host"], c["indptr"], c["toks"], c["par"], c["u"], c["noise"][:, :c["vocab"]], c["t"],
                          c["dp_host"])


def _case(seed, *a, **kw):
    """The first of the seeds seed, seed + 1000, ... whose decisions are clear (by the oracle alone)."""
    for k in range(40):
        c = _inputs(seed + 1000 * k, *a, **kw)
        c["ref"] = _ref(c)
        if c["ref"][4] > MARGIN:
            return c
    raise AssertionError("no clear case")


def _dev(c):
    d = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    V = c["vocab"]
    dp = None if c["dp"] is None else c["dp"].cuda()[:, :V]
    return [c["lg"].cuda()[:, :V], d(c["indptr"]), d(c["toks"]), d(c["par"]), d(c["u"]), d(c["noise"])[:, :V], d(c["t"]),
            dp]


def _same(c, got, rows=None):
    acc, path, bonus, logp = [x.cpu().numpy() for x in got]
    r_acc, r_paths, r_bonus, r_logp, _ = c["ref"]
    assert np.array_equal(acc, r_acc)
    for b in range(len(r_acc)):
        o, n = int(c["indptr"][b]), int(c["indptr"][b + 1] - c["indptr"][b])
        want = np.full(n, -1)
        want[:r_acc[b]] = r_paths[b]
        assert np.array_equal(path[o:o + n], want)
    assert np.array_equal(bonus, r_bonus)
    err = np.abs(logp - r_logp) - 2.0 ** -24 * np.abs(r_logp)
    assert not err.size or err.max() <= LOGP_TOL, err.max()


def _run(va, c, **kw):
    args = _dev(c)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = va.verify_accept_sample(*args[:6], temperature=args[6], draft_probs=args[7], want_logprobs=True,
                                  status=status, **kw)
    torch.cuda.synchronize()
    assert int(status) == 0
    return got


F, H = torch.float32, torch.bfloat16
CASES = {
    "one_row": dict(lens=[1], vocab=32016),
    "chain_f32": dict(lens=[5], vocab=32016, kind="chain", qdt=F, temps=[0.8]),
    "chains_bf16_q": dict(lens=[1, 5, 8, 3, 2, 8, 7, 1] * 4, vocab=8192, kind="chain", qdt=H, temps=[0.0, 0.7, 1.3]),
    "tree_q": dict(lens=[17, 9, 30], vocab=4096, qdt=F),
    "tree_f32_logits": dict(lens=[17, 9], vocab=5003, ldt=F, qdt=H, temps=[1.1, 0.6]),
    "tree_no_q": dict(lens=[64, 33], vocab=20000, temps=[1.0, 0.0]),
    "star_no_q": dict(lens=[150], vocab=4000, kind="star"),      # five windows, more children than the list, repeats
    "star_no_q_late": dict(lens=[150, 90], vocab=300, kind="star", u_min=0.97),
    "star_q_late": dict(lens=[70, 40], vocab=500, kind="star", qdt=F, temps=[1.5], u_min=0.9),
    "star_bf16_q_late": dict(lens=[12, 20], vocab=8192, kind="star", qdt=H, u_min=0.95),
    "big_tree_q": dict(lens=[300, 2], vocab=600, qdt=F),                     # past what shared memory keeps of a tree
    "long_chain": dict(lens=[400, 140], vocab=40, kind="chain", qdt=F, near=0.0, u_max=0.4),   # hundreds accepted
    "long_chain_greedy": dict(lens=[200], vocab=300, kind="chain", temps=[0.0], greedy_drafts=True),
    "star_q": dict(lens=[70, 40], vocab=1000, kind="star", qdt=F, temps=[1.5]),
    "many_requests": dict(lens=[3] * 330, vocab=64, kind="chain", qdt=F),    # one CTA each
    "two_ctas": dict(lens=[2] * 120, vocab=9000, kind="chain", qdt=H),
    "vocab_1": dict(lens=[3, 1], vocab=1, kind="chain", qdt=F),
    "vocab_7": dict(lens=[4, 6, 2], vocab=7, qdt=F, temps=[0.9]),
    "odd_rows": dict(lens=[6, 0, 4], vocab=1001, ldt=F, qdt=F),
    "odd_bf16_rows": dict(lens=[6, 0, 4], vocab=4099),
    "padded_rows": dict(lens=[5, 6], vocab=4000, pad=24, qdt=F),
    "padded_odd_rows": dict(lens=[5, 6], vocab=4001, pad=2, qdt=H, ldt=F),
    "masked": dict(lens=[7, 5], vocab=6000, masked=0.995, qdt=F, temps=[0.7, 1.0]),
    "masked_no_q": dict(lens=[12, 5], vocab=6000, masked=0.999, ldt=F),
    "wide_range": dict(lens=[8, 8], vocab=3000, spread=30.0, qdt=F, ldt=F, temps=[2.0, 0.2]),
    "llama3_vocab": dict(lens=[8, 3], vocab=128256, kind="chain", qdt=F, temps=[0.7]),
    "empty": dict(lens=[0, 0], vocab=100),
}


@pytest.mark.parametrize("name", CASES)
def test_matches_oracle(va, name):
    c = _case(11, **CASES[name])
    _same(c, _run(va, c))


def test_repeated_calls_are_equal_and_outputs_are_reused(va):
    c = _case(3, lens=[9, 12], vocab=8192, qdt=F)
    a, b = _run(va, c), _run(va, c)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    out = tuple(torch.full_like(x, 77) for x in a)
    got = _run(va, c, out=out)
    assert all(x is y for x, y in zip(got, out)) and all(torch.equal(x, y) for x, y in zip(a, out))


def test_rows_behind_the_last_request_are_left(va):
    """A padded batch: logits rows past qo_indptr[B] are neither read (NaN) nor answered."""
    c = _case(4, lens=[4, 3], vocab=512, qdt=F)
    a = _dev(c)
    grow = lambda t, v: torch.cat([t, torch.full((3,) + t.shape[1:], v, dtype=t.dtype, device="cuda")])  # noqa: E731
    out = (torch.empty(2, dtype=torch.int32, device="cuda"), torch.full((10,), 55, dtype=torch.int32, device="cuda"),
           torch.empty(2, dtype=torch.int32, device="cuda"), torch.full((10,), 5.5, device="cuda"))
    got = va.verify_accept_sample(grow(a[0], float("nan")), a[1], grow(a[2], 1 << 30), grow(a[3], 9), grow(a[4], 2.0),
                                  a[5], draft_probs=grow(a[7], float("nan")), out=out)
    assert (got[1][7:] == 55).all() and (got[3][7:] == 5.5).all()
    _same(c, (got[0], got[1][:7], got[2], got[3][:7]))


def test_without_logprobs(va):
    c = _case(5, lens=[6, 6], vocab=700)
    a = _dev(c)
    got = va.verify_accept_sample(*a[:6])
    assert got[3] is None and np.array_equal(got[0].cpu().numpy(), c["ref"][0])
    assert np.array_equal(got[2].cpu().numpy(), c["ref"][2])


def test_equal_candidates_take_the_lowest_index(va):
    V = 5000
    z = torch.zeros
    got = va.verify_accept_sample(z(1, V, device="cuda", dtype=H), torch.tensor([0, 1], dtype=torch.int32).cuda(),
                                  z(1, dtype=torch.int32, device="cuda"),
                                  torch.tensor([-1], dtype=torch.int32).cuda(), z(1, device="cuda"),
                                  torch.ones(1, V, device="cuda"), want_logprobs=True)
    assert int(got[2]) == 0 and abs(float(got[3]) + np.log(V)) < LOGP_TOL


def test_zero_noise_wins_among_possible_tokens(va):
    V = 300
    lg = torch.zeros(1, V, device="cuda")
    lg[0, :100] = -float("inf")
    noise = torch.ones(1, V, device="cuda")
    noise[0, [50, 200]] = 0.0        # token 50 is impossible
    one = lambda v: torch.tensor([v], dtype=torch.int32).cuda()  # noqa: E731
    got = va.verify_accept_sample(lg, torch.tensor([0, 1], dtype=torch.int32).cuda(), one(0), one(-1),
                                  torch.zeros(1, device="cuda"), noise)
    assert int(got[2]) == 200


def test_a_residual_without_mass_draws_from_the_target(va):
    """q above p everywhere (a draft distribution that sums to more than 1):
    the rejected child leaves nothing, and the bonus token comes from p."""
    rng = np.random.default_rng(0)
    V = 400
    c = dict(lg=torch.from_numpy(rng.standard_normal((2, V))).to(F), indptr=np.array([0, 2], np.int32),
             par=np.array([-1, 0], np.int32), toks=np.array([0, 5], np.int32), u=np.array([0, 0.9], np.float32),
             noise=rng.exponential(size=(1, V)).astype(np.float32), t=None, vocab=V)
    c["host"] = c["lg"].double().numpy()
    p = np.exp(c["host"]) / np.exp(c["host"]).sum(1, keepdims=True)
    c["dp"] = torch.from_numpy(p * 1.5).to(F)
    c["dp_host"] = c["dp"].double().numpy()
    c["ref"] = _ref(c)
    assert c["ref"][0][0] == 1 and c["ref"][4] > MARGIN
    _same(c, _run(va, c))
    # and without q: the only possible token is rejected
    c["lg"] = torch.full((2, V), -float("inf"))
    c["lg"][:, 7] = 1.0
    c["host"], c["dp"], c["dp_host"] = c["lg"].double().numpy(), None, None
    c["toks"], c["u"] = np.array([0, 7], np.int32), np.array([0, 1.0], np.float32)   # u = 1: never accepted
    acc, path, bonus, logp = _run(va, c)
    assert int(acc) == 1 and int(bonus) == 7 and float(logp[0]) == 0.0


def test_rows_of_minus_infinity_end_the_path(va):
    lg = torch.zeros(3, 200, device="cuda")
    lg[0] = -float("inf")
    i = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    for t in (None, torch.zeros(1, device="cuda")):
        acc, path, bonus, logp = va.verify_accept_sample(lg, i(0, 3), i(0, 1, 2), i(-1, 0, 1),
                                                         torch.zeros(3, device="cuda"),
                                                         torch.ones(1, 200, device="cuda"), temperature=t,
                                                         want_logprobs=True)
        assert acc.tolist() == [1] and bonus.tolist() == [-1] and path.tolist() == [0, -1, -1]
        assert logp.tolist() == [0, 0, 0]


def test_tokens_outside_the_vocabulary_are_rejected(va):
    for qdt in (None, F):
        c = _inputs(6, [4, 4], 300, kind="star", qdt=qdt)
        c["toks"][[1, 2, 5]] = [300, -1, 1 << 30]
        c["ref"] = _ref(c)
        assert c["ref"][4] > MARGIN
        _same(c, _run(va, c))


def test_malformed_requests_are_flagged_and_the_others_answered(va):
    c = _case(8, lens=[5, 4, 3, 6], vocab=512, qdt=F, temps=[1.0, 0.8, 0.9, 1.2])
    a = _dev(c)
    a[3][5 + 2] = 3                 # request 1: a parent that comes later
    a[6][2] = float("nan")          # request 2: no temperature
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    acc, path, bonus, logp = va.verify_accept_sample(*a[:6], temperature=a[6], draft_probs=a[7], want_logprobs=True,
                                                     status=status)
    assert int(status) == 2
    for b in (1, 2):
        o, e = int(c["indptr"][b]), int(c["indptr"][b + 1])
        assert int(acc[b]) == 0 and int(bonus[b]) == -1
        assert (path[o:e] == -1).all() and (logp[o:e] == 0).all()
    for b in (0, 3):
        assert int(acc[b]) == c["ref"][0][b] and int(bonus[b]) == c["ref"][2][b]
    # a table that reaches past the rows: nothing is read for the request
    status.zero_()
    a = _dev(c)
    a[1][4] = 19
    acc, _, bonus, _ = va.verify_accept_sample(*a[:6], temperature=a[6], draft_probs=a[7], status=status)
    assert int(status) == 2 and int(acc[3]) == 0 and int(bonus[3]) == -1
    assert acc[:3].tolist() == c["ref"][0][:3].tolist()


@pytest.mark.parametrize("qdt", [None, F], ids=["no_q", "q"])
def test_a_batch_larger_than_the_gpu_is_answered_in_any_order(va, qdt):
    """200 ragged requests (more CTAs than SMs), empty, malformed and T = 0 ones among them: each as by itself."""
    rng = np.random.default_rng(11)
    lens = [int(n) for n in rng.integers(0, 10, 200)]
    lens[7] = lens[150] = 6
    c = _case(31, lens=lens, vocab=600, qdt=qdt, temps=[0.9, 0.0, 1.2])
    _same(c, _run(va, c))
    a = _dev(c)
    a[3][int(c["indptr"][7]) + 3] = 5          # a parent that comes later
    a[6][150] = -1.0                           # no temperature
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    acc, path, bonus, logp = va.verify_accept_sample(*a[:6], temperature=a[6], draft_probs=a[7], want_logprobs=True,
                                                     status=status)
    assert int(status) == 2
    want_acc, want_bonus = np.array(c["ref"][0]), np.array(c["ref"][2])
    want_acc[[7, 150]], want_bonus[[7, 150]] = 0, -1
    assert np.array_equal(acc.cpu().numpy(), want_acc) and np.array_equal(bonus.cpu().numpy(), want_bonus)
    for b in (7, 150):
        o, e = int(c["indptr"][b]), int(c["indptr"][b + 1])
        assert (path[o:e] == -1).all() and (logp[o:e] == 0).all()


def test_agrees_with_greedy_acceptance_at_temperature_zero(va):
    """Distinct siblings, T = 0: verify_accept_greedy's path and bonus token."""
    rng = np.random.default_rng(2)
    lens, V = [17, 9, 1, 30], 6001
    lg = torch.from_numpy(rng.integers(-6, 7, (sum(lens), V))).to(H).cuda()   # many equal maxima
    am = lg.argmax(1)
    host_am = np.array([int((lg[i] == lg[i].max()).nonzero()[0, 0]) for i in range(sum(lens))])
    par = _parents(lens, "tree", rng)
    indptr = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    toks, used = np.zeros(sum(lens), np.int32), {}
    for b, n in enumerate(lens):
        for i in range(1, n):
            o = int(indptr[b])
            v = o + int(par[o + i])
            first = v not in used
            used.setdefault(v, 1)
            toks[o + i] = host_am[v] if first and rng.random() < 0.8 else 6000 - i
    d = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    g = va.verify_accept_greedy(lg, d(indptr), d(toks), d(par))
    s = va.verify_accept_sample(lg, d(indptr), d(toks), d(par), torch.rand(sum(lens), device="cuda"),
                                torch.ones(len(lens), V, device="cuda"), temperature=torch.zeros(len(lens), device="cuda"))
    assert torch.equal(g[0], s[0]) and torch.equal(g[2], s[2]) and torch.equal(g[1], s[1])
    assert int(g[0].max()) > 2 and am.numel()


LONG = {   # 154 requests, a CTA or two each: long slices of the vocabulary, most drafts rejected
    "f32_q": dict(lens=[2] * 154, vocab=32768, kind="chain", qdt=F, u_min=0.8),
    "bf16_q_siblings": dict(lens=[3, 2] * 77, vocab=20000, kind="star", qdt=H, u_min=0.9, temps=[0.8, 0.0, 1.3]),
    "q_close_to_p": dict(lens=[2] * 154, vocab=16408, kind="chain", qdt=F, u_min=0.95, near=0.02),
    "f32_logits_masked": dict(lens=[2] * 154, vocab=24576, ldt=F, qdt=F, u_min=0.8, masked=0.98),
    "longest": dict(lens=[2] * 153, vocab=66000, kind="chain", qdt=H, u_min=0.8),
}


@pytest.mark.parametrize("name", LONG)
def test_long_slices_match_oracle(va, name):
    c = _case(21, **LONG[name])
    _same(c, _run(va, c))


def test_long_slices_noise_of_zero_and_residuals_without_mass(va):
    """p uniform, q twice p on the first half of the tokens: the residual lies on the second half alone."""
    B, V = 154, 32768
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    lg = torch.zeros(2 * B, V, dtype=H, device="cuda")
    q = torch.zeros(2 * B, V, device="cuda")
    q[:, :V // 2] = 2.0 / V
    noise = torch.ones(B, V, device="cuda")
    noise[:, 100] = 0.0                       # rejected with its half
    noise[1::3, 20000] = 0.0                  # the first possible one
    noise[2::3, [31000, 25001]] = 0.5
    args = (i32(range(0, 2 * B + 1, 2)), i32([0, 5] * B), i32([-1, 0] * B), torch.full((2 * B,), 0.9, device="cuda"))
    acc, path, bonus, logp = va.verify_accept_sample(lg, *args, noise, draft_probs=q, want_logprobs=True)
    assert acc.tolist() == [1] * B
    assert bonus.tolist() == [[V // 2, 20000, 25001][b % 3] for b in range(B)]
    assert (logp[::2] + np.log(V)).abs().max() < LOGP_TOL and (logp[1::2] == 0).all()
    # q above p everywhere: the bonus token comes from p
    acc, path, bonus, _ = va.verify_accept_sample(lg, *args, noise, draft_probs=torch.full_like(q, 1.5 / V))
    assert acc.tolist() == [1] * B and bonus.tolist() == [100] * B


@pytest.mark.parametrize("V", [1, 7, 1001, 40000])
@pytest.mark.parametrize("ldt", [H, F], ids=["bf16", "fp32"])
def test_greedy_bonus_is_the_first_of_equal_maxima(va, ldt, V):
    """T = 0 on rows with one to several equal maxima, +0 and -0 among them: the first index."""
    rng = np.random.default_rng(V)
    B = 24
    lg = np.full((B, V), -3.0, np.float32)
    for b in range(B):
        at = rng.integers(0, V, 1 + b % 5)
        lg[b, at] = [5.0, -0.0, 0.0][b % 3]
        if b % 3:
            lg[b, rng.choice(at)] *= -1
    x = torch.from_numpy(lg).to(ldt).cuda()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    acc, path, bonus, _ = va.verify_accept_sample(x, i32(range(B + 1)), i32([0] * B), i32([-1] * B),
                                                  torch.zeros(B, device="cuda"), torch.ones(B, V, device="cuda"),
                                                  temperature=torch.zeros(B, device="cuda"))
    assert acc.tolist() == [1] * B and path.tolist() == [0] * B
    assert bonus.tolist() == lg.argmax(1).tolist()


def test_graph_replay_and_side_stream(va):
    """Captured once, replayed over new inputs in the same buffers, on a stream of its own."""
    cs = [_case(s, lens=[5, 5, 5], vocab=4096, kind="chain", qdt=F, temps=[0.9]) for s in (21, 22)]
    bufs = _dev(cs[0])
    side = torch.cuda.Stream()
    out = tuple(torch.zeros(n, dtype=t, device="cuda") for n, t in ((3, torch.int32), (15, torch.int32), (3, torch.int32), (15, F)))
    torch.cuda.synchronize()
    call = lambda **kw: va.verify_accept_sample(*bufs[:6], temperature=bufs[6], draft_probs=bufs[7], out=out, **kw)  # noqa: E731
    call(stream=side)
    side.synchronize()
    _same(cs[0], out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call()
        call()
    for c in (cs[1], cs[0], cs[1]):
        for x, y in zip(bufs, _dev(c)):
            if x is not None:
                x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        _same(c, out)


def test_rows_far_apart(va):
    """Row and noise offsets past 2^32 bytes."""
    c = _case(31, lens=[2, 1], vocab=4096, kind="chain", qdt=F)
    a = _dev(c)
    far = 1 << 30
    big = torch.empty(2 * far + 4096, dtype=H, device="cuda")
    lg = big.as_strided((3, 4096), (far, 1))
    lg.copy_(a[0])
    nbig = torch.empty(far + 4096 + 4, dtype=F, device="cuda")
    noise = nbig[4:].as_strided((2, 4096), (far, 1))
    noise.copy_(a[5])
    _same(c, va.verify_accept_sample(lg, *a[1:5], noise, draft_probs=a[7], want_logprobs=True))


def test_refusals(va):
    c = _inputs(9, [3, 2], 64, kind="chain", qdt=F)
    a = _dev(c)

    def call(i, t, **kw):
        b = list(a)
        b[i] = t
        return va.verify_accept_sample(*b[:6], temperature=b[6], draft_probs=b[7], **kw)

    for i, t in ((0, a[0].half()), (0, a[0][:, ::2]), (0, a[0][0]), (1, a[1].long()), (1, a[1][:2]), (2, a[2][:4]),
                 (2, a[2].long()), (3, a[3].cpu()), (4, a[4].double()), (5, a[5][:1]), (5, a[5].bfloat16()),
                 (5, a[5].t().contiguous().t()), (6, torch.ones(3, device="cuda")), (7, a[7].half()), (7, a[7][:, :32]),
                 (0, a[0][:1].expand(5, 64))):
        with pytest.raises(ValueError):
            call(i, t)
    with pytest.raises(ValueError):
        call(0, a[0], out=(a[1], a[2], a[3], None))
