"""Pins of the sampled-acceptance oracle (oracle/accept_sample.py): the emitted
token follows the target's distribution exactly (by enumeration, no
sampling), the residuals' closed form, and small worked cases; and the
argument checks of verify_accept_sample / paged_kv_compact that need no device."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

from oracle.accept_sample import accept_sampled, compact_rows, softmax64


@pytest.fixture(scope="module")
def va():
    from speculative_decoding_verify_gqa_gb300 import build as b
    b.build()
    import speculative_decoding_verify_gqa_gb300 as m
    m.lib()
    return m


def _law(p, q, m):
    """Law of the first emitted token with m siblings drawn i.i.d. from q,
    integrated over their uniforms, by the definition's residuals."""
    V = len(p)
    out = np.zeros(V)
    for toks in itertools.product(range(V), repeat=m):
        w, r = np.prod([q[x] for x in toks]), p.copy()
        for x in toks:
            a = min(1.0, r[x] / q[x]) if q[x] > 0 else 1.0
            out[x] += w * a
            w *= 1 - a
            left = np.maximum(r - q, 0)
            r = left / left.sum() if left.sum() > 0 else left
        out += w * r
    return out


@pytest.mark.parametrize("m", [1, 2, 3])
def test_definition_emits_the_target_distribution(m):
    rng = np.random.default_rng(m)
    p, q = rng.dirichlet(np.ones(4)), rng.dirichlet(np.ones(4))
    assert np.abs(_law(p, q, m) - p).max() < 1e-12


def test_residual_closed_form():
    rng = np.random.default_rng(5)
    p, q = rng.dirichlet(np.ones(50) * 0.3), rng.dirichlet(np.ones(50) * 0.3)
    r, A, B = p.copy(), 0.0, 1.0
    for _ in range(4):
        left = np.maximum(r - q, 0)
        r = left / left.sum()
        A, B = A + B, np.maximum(p - (A + B) * q, 0).sum()
        assert np.abs(r - np.maximum(p - A * q, 0) / B).max() < 1e-12


def test_oracle_acceptance_borders():
    """One child: accepted exactly while u q(x) < p(x); without q while u < p(x)."""
    p = np.array([0.5, 0.3, 0.2])
    lg, noise = np.log(np.stack([p, p])), np.ones((1, 3))
    for q, border in ((np.array([0.2, 0.6, 0.2]), 0.5), (None, 0.3)):
        dp = None if q is None else np.stack([q, q])
        for u, n in ((border - 1e-9, 2), (border + 1e-9, 1)):
            acc, paths, bonus, logp, _ = accept_sampled(lg, [0, 2], [0, 1], [-1, 0], [0.0, u], noise, None, dp)
            assert acc[0] == n and list(paths[0]) == list(range(n))
            if n == 1:
                # the residual: (p - q)+ = (.3, 0, 0), or p without token 1
                assert bonus[0] == 0 and logp[0] == pytest.approx(np.log(0.5))
            else:
                assert logp[0] == pytest.approx(np.log(0.3))


def test_oracle_race_prefers_small_noise_and_low_indices():
    lg = np.zeros((1, 4))
    one = lambda e: accept_sampled(lg, [0, 1], [0], [-1], [0.5], np.array([e]))[2][0]  # noqa: E731
    assert one([1.0, 0.5, 2.0, 0.25]) == 3
    assert one([1.0, 1.0, 1.0, 1.0]) == 0


def test_oracle_temperature_zero_is_the_first_argmax():
    lg = np.array([[0.0, 2.0, 2.0], [1.0, 0.0, 0.0]])
    acc, _, bonus, logp, _ = accept_sampled(lg, [0, 2], [0, 1], [-1, 0], [0, 0.999], np.ones((1, 3)), [0.0])
    assert acc[0] == 2 and bonus[0] == 0 and not logp.any()
    acc, _, bonus, _, _ = accept_sampled(lg, [0, 2], [0, 2], [-1, 0], [0, 0.0], np.ones((1, 3)), [0.0])
    assert acc[0] == 1 and bonus[0] == 1


def test_softmax64_masks_and_dead_rows():
    assert list(softmax64([-np.inf, 0.0, -np.inf], 0.7)) == [0, 1, 0]
    assert not softmax64([-np.inf, -np.inf], 1.0).any()


def test_compact_rows_closed_form():
    # 2 requests, pages of 4: prefix 5 + 4 drafts over pages 7, 3, 9; no prefix, 3 drafts on page 1
    moves, new = compact_rows([0, 4, 7], [0, 3, 4], [1, 3], 4, [7, 3, 9, 1], [3, 1], [0, 2, 3, -1, 0, -1, -1])
    assert moves == [((3, 3), (3, 2)), ((9, 0), (3, 3))]
    assert list(new) == [8, 1]


def test_accept_sample_validation_without_device(va):
    f = ctypes.c_void_p(4096)
    L = va.lib().verify_accept_sample

    def call(logits=f, dt=0, total=4, vocab=100, rs=100, indptr=f, batch=1, toks=f, par=f, u=f, noise=f, ns=100,
             temp=None, dp=None, dd=0, ds=0, acc=f, path=f, bonus=f, lp=None):
        return L(logits, dt, total, vocab, rs, indptr, batch, toks, par, u, noise, ns, temp, dp, dd, ds, acc, path,
                 bonus, lp, None, 152, None)

    assert call(batch=0) == 0
    for bad in (dict(rs=50), dict(ns=50), dict(vocab=0), dict(total=-1), dict(batch=-1), dict(dp=f, ds=50),
                dict(indptr=None), dict(noise=None), dict(logits=None), dict(u=None), dict(acc=None),
                dict(bonus=None), dict(path=None), dict(toks=None), dict(par=None),
                dict(logits=ctypes.c_void_p(4097)), dict(noise=ctypes.c_void_p(4098)),
                dict(dp=ctypes.c_void_p(4097), ds=100)):
        assert call(**bad) == -1, bad
    for bad in (dict(dt=1), dict(dp=f, dd=1, ds=100), dict(total=1 << 31), dict(rs=1 << 46),
                dict(vocab=0x7fffffff, rs=1 << 31, ns=1 << 31)):
        assert call(**bad) == -2, bad


def test_compact_validation_without_device(va):
    f = ctypes.c_void_p(4096)
    L = va.lib().paged_kv_compact

    def call(acc=f, path=f, qo=f, total=4, kvp=f, kvi=f, lpl=f, k=f, v=f, layers=1, batch=1, h=2, d=128, dv=0, ps=16,
             pages=10, dt=0, layout=0):
        return L(acc, path, qo, total, kvp, kvi, lpl, k, v, layers, batch, h, d, dv, ps, pages, dt, layout, None,
                 None, None)

    assert call(batch=0) == 0
    for bad in (dict(layers=0), dict(total=-1), dict(h=0), dict(dv=-1), dict(layout=2), dict(acc=None),
                dict(path=None), dict(qo=None), dict(kvp=None), dict(kvi=None), dict(lpl=None), dict(k=None),
                dict(v=None), dict(pages=0), dict(k=ctypes.c_void_p(4104)), dict(ps=0)):
        assert call(**bad) == -1, bad
    for bad in (dict(d=96), dict(dv=32), dict(ps=24), dict(dt=2), dict(batch=70000), dict(total=1 << 31)):
        assert call(**bad) == -2, bad


def test_compact_refuses_pools_that_overlap(va):
    """The same pool twice, or one that begins inside the other, either way round."""
    at = ctypes.c_void_p

    def call(k, v, d=128, dv=64):
        t = at(4096)
        return va.lib().paged_kv_compact(t, t, t, 4, t, t, t, at(k), at(v), 3, 1, 2, d, dv, 16, 10, 0, 0, None, None,
                                         None)

    k_bytes, v_bytes = 3 * 10 * 2 * 16 * 128 * 2, 3 * 10 * 2 * 16 * 64 * 2
    base = 1 << 20
    for k, v in ((base, base), (base, base + k_bytes - 16), (base + v_bytes - 16, base), (base, base + 16)):
        assert call(k, v) == -1


def test_binding_refuses_host_tensors(va):
    z = torch.zeros
    with pytest.raises(ValueError, match="current CUDA device"):
        va.verify_accept_sample(z(2, 8), z(2, dtype=torch.int32), None, None, None, None)
    with pytest.raises(ValueError, match="current CUDA device"):
        va.paged_kv_compact(None, None, None, None, None, None, z(1, 1, 16, 64), z(1, 1, 16, 64))
