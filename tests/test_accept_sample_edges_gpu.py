"""Sampled acceptance at its borders: drafts that can not be emitted behind
siblings that take all the mass, and decisions one fp32 step from their
border."""
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

LAST = np.float32(1 - 2.0 ** -24)   # the largest uniform below 1


@pytest.fixture(scope="module")
def va():
    import __graft_entry__
    __graft_entry__.build()
    import speculative_decoding_verify_gqa_gb300 as m
    return m


def _cu(x, dt=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dt is None else t.to(dt)


@pytest.mark.parametrize("q", [False, True], ids=["no_q", "q"])
@pytest.mark.parametrize("possible", [1, 2, 3, 7, 31, 32, 40, 70])
def test_impossible_drafts_are_never_accepted(va, possible, q):
    """Every possible token is drafted, then a masked one, repeats and tokens
    outside the vocabulary, with the largest uniforms: what is accepted, and
    the bonus token, is a possible token at its first draft."""
    rng = np.random.default_rng(possible)
    B, V = 400, 96
    lg = np.full((B, V), -np.inf, np.float32)
    can = np.stack([rng.permutation(V)[:possible] for _ in range(B)])
    np.put_along_axis(lg, can, rng.standard_normal((B, possible)).astype(np.float32) * 3, 1)
    mask = np.isneginf(lg)
    masked = np.array([np.flatnonzero(r)[0] for r in mask])
    n = 1 + possible + 6
    toks = np.zeros((B, n), np.int32)
    toks[:, 1:1 + possible] = can
    toks[:, 1 + possible:] = np.stack([masked, can[:, 0], np.full(B, V), np.full(B, -1), can[:, -1], np.full(B, 1 << 30)], 1)
    par = np.tile(np.array([-1] + [0] * (n - 1), np.int32), (B, 1))
    u = np.full((B, n), LAST, np.float32)
    rows = np.repeat(lg[:, None], n, 1).reshape(B * n, V)
    probs = None
    if q:
        p = np.exp(lg.astype(np.float64))
        p /= p.sum(1, keepdims=True)
        probs = _cu(np.repeat((p * rng.uniform(0.9, 1.1, (B, 1)))[:, None], n, 1).reshape(B * n, V).astype(np.float32))
    noise = rng.exponential(size=(B, V)).astype(np.float32)
    acc, path, bonus, logp = va.verify_accept_sample(
        _cu(rows), _cu(np.arange(B + 1, dtype=np.int32) * n), _cu(toks.reshape(-1)), _cu(par.reshape(-1)),
        _cu(u.reshape(-1)), _cu(noise), draft_probs=probs, want_logprobs=True)
    acc, path, bonus = acc.cpu().numpy(), path.cpu().numpy().reshape(B, n), bonus.cpu().numpy()
    assert ((acc == 1) | (acc == 2)).all()
    taken = path[acc == 2, 1]
    assert ((taken >= 1) & (taken <= possible)).all(), "accepted %s" % np.unique(taken[taken > possible])
    assert not mask[np.arange(B), bonus].any()
    logp = logp.cpu().numpy().reshape(B, n)
    assert np.isfinite(logp).all() and (logp <= 0).all()


def _borders(x):
    """The fp32 numbers on either side of the fraction x, or x itself as the upper one."""
    f = np.float32(float(x))
    while Fraction(float(f)) >= x:
        f = np.nextafter(f, np.float32(0), dtype=np.float32)
    while Fraction(float(np.nextafter(f, np.float32(1), dtype=np.float32))) < x:
        f = np.nextafter(f, np.float32(1), dtype=np.float32)
    return f, np.nextafter(f, np.float32(1), dtype=np.float32)


@pytest.mark.parametrize("V", [64, 4096, 32768, 131072])
@pytest.mark.parametrize("ldt", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_one_step_from_the_border_without_draft_probs(va, V, ldt):
    """Equal logits: p = 1 / V, and after j rejections a token is accepted iff
    u < 1 / (V - j), in fp32 numbers on either side of it.  Weights, sums and
    what remains are exact here, so the decision is."""
    js = [0, 1, 2, 3, 5, 17, 31, 33, 40]
    lens, toks, us, want = [], [], [], []
    for j in js:
        for side in (0, 1):
            n = j + 2
            lens.append(n)
            toks += [0] + list(range(3, 3 + n - 1))
            us += [0.0] + [LAST] * j + [_borders(Fraction(1, V - j))[side]]
            want.append(2 - side)
    indptr = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    par = np.concatenate([[-1] + [0] * (n - 1) for n in lens]).astype(np.int32)
    total, B = int(indptr[-1]), len(lens)
    lg = torch.full((1, V), 1.5, device="cuda", dtype=ldt).expand(total, V).contiguous()
    for t in (None, torch.full((B,), 0.7, device="cuda")):
        acc, path, _, _ = va.verify_accept_sample(lg, _cu(indptr), _cu(np.array(toks, np.int32)), _cu(par),
                                                  _cu(np.array(us, np.float32)), torch.ones(B, V, device="cuda"),
                                                  temperature=t)
        assert acc.tolist() == want
        path = path.cpu().numpy()
        assert [int(path[indptr[b] + 1]) for b in range(B) if want[b] == 2] == [j + 1 for j in js]


@pytest.mark.parametrize("V", [64, 4096, 32768, 131072])
@pytest.mark.parametrize("qdt", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_one_step_from_the_border_with_draft_probs(va, V, qdt):
    """p = 1 / V throughout; q in units of 1 / V: 0 on the first quarter of the
    vocabulary, 7/8 on the next half, 9/4 on the last quarter.  A draft of the
    last quarter is accepted iff u 9/4 < 1; behind a rejected one, B = 1/4 +
    1/2 (1 - 7/8) = 5/16, a draft of the middle iff u 7/8 < (1/8) / (5/16)."""
    q = torch.zeros(V)
    q[V // 4:3 * V // 4], q[3 * V // 4:] = 7 / 8 / V, 9 / 4 / V
    lo, mid, hi = 1, V // 2, V - 3
    lens, toks, us, want = [], [], [], []
    for side in (0, 1):
        lens.append(2)
        toks += [0, hi]
        us += [0.0, _borders(Fraction(4, 9))[side]]
        want.append(2 - side)
        lens.append(3)
        toks += [0, hi, mid]
        us += [0.0, 0.9, _borders(Fraction(16, 35))[side]]
        want.append(2 - side)
        lens.append(4)   # and behind it a draft that q gives nothing: accepted while p leaves it anything
        toks += [0, hi, hi, lo]
        us += [0.0, 0.9, 0.0, LAST]
        want.append(2)
    indptr = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    par = np.concatenate([[-1] + [0] * (n - 1) for n in lens]).astype(np.int32)
    total, B = int(indptr[-1]), len(lens)
    acc, path, _, _ = va.verify_accept_sample(
        torch.full((total, V), -2.0, device="cuda", dtype=torch.bfloat16), _cu(indptr), _cu(np.array(toks, np.int32)),
        _cu(par), _cu(np.array(us, np.float32)), torch.ones(B, V, device="cuda"),
        draft_probs=q.to(qdt).cuda().expand(total, V).contiguous())
    assert acc.tolist() == want
    path = path.cpu().numpy()
    assert [int(path[indptr[b] + 1]) for b in range(B) if want[b] == 2] == [1, 2, 3, 3]
