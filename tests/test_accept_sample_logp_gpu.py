"""The digits of sampled acceptance's log-probabilities: relative to log p, also
where the model is sure and log p is small."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def va():
    import __graft_entry__
    __graft_entry__.build()
    import speculative_decoding_verify_gqa_gb300 as m
    return m


def _cu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


# log p = y ln 2 - log(1 + tail), tail the row's weights but the largest's own.
# Relative to log p, whatever its size, for |y| < 64 (half a step of the
# argument is 2^-19 there):
#   a weight 2^y: the instruction 2^-22, its argument ln 2 * 2^-19 = 1.33e-6;
#   on its way to the row's maximum a term is multiplied by up to five such
#   weights (a thread's maximum raised, warp, CTA, cluster), whose exponents add
#   up to |y|: together at most 5 * (2^-22 + 1.33e-6) = 7.9e-6;
#   a thread's sum: 32 additions in a row, then one a batch of 64 entries, four
#   batches at most here: 37 * 2^-24 = 2.2e-6;
#   three joins, 32 terms rounded to 2^-27 / 2 of the largest: 3 * 2^-23;
#   log(1 + tail) and the result: 2^-23.
LOGP_REL = 1.1e-5


@pytest.mark.parametrize("ldt", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("vocab", [5, 1001, 8192, 50257])
def test_log_p_of_sure_tokens_keeps_its_digits(va, vocab, ldt):
    """Rows whose likeliest token has p from 1 - 1e-9 to 0.5, tails of one token or of the whole vocabulary."""
    rng = np.random.default_rng(vocab)
    gaps = np.concatenate([np.linspace(0.5, 22, 40), np.linspace(0.5, 22, 40)])
    B = len(gaps)
    lg = rng.standard_normal((B, vocab)).astype(np.float32)
    lg[40:] = -np.inf
    hot = rng.integers(0, vocab, B)
    other = (hot + 1 + rng.integers(0, vocab - 1, B)) % vocab
    lg[np.arange(B), other] = 0.5
    top = np.where(np.isfinite(lg), np.exp(lg.astype(np.float64)), 0).sum(1)
    lg[np.arange(B), hot] = np.log(top) + gaps
    x = torch.from_numpy(lg).to(ldt)
    host = x.double().numpy()
    d = host - host[np.arange(B), hot][:, None]
    w = np.exp(d)
    w[np.arange(B), hot] = 0
    want = -np.log1p(w.sum(1))
    # the bonus token is the hot one: its noise is least
    noise = np.ones((B, vocab), np.float32)
    noise[np.arange(B), hot] = 1e-20
    one = np.zeros(B, np.int32)
    acc, _, bonus, logp = va.verify_accept_sample(x.cuda(), _cu(np.arange(B + 1, dtype=np.int32)), _cu(one), _cu(one - 1),
                                                  torch.zeros(B, device="cuda"), _cu(noise), want_logprobs=True)
    assert bonus.cpu().tolist() == hot.tolist()
    err = np.abs(logp.cpu().numpy() - want) / np.abs(want)
    print("log p of sure tokens: largest relative error %.3g, rms %.3g" % (err.max(), np.sqrt((err ** 2).mean())))
    assert err.max() <= LOGP_REL
    # the same as an accepted draft: a chain of two, u = 0
    rows = torch.repeat_interleave(x, 2, 0).cuda()
    toks, par = np.stack([one, hot.astype(np.int32)], 1).reshape(-1), np.tile(np.array([-1, 0], np.int32), B)
    acc, _, _, logp = va.verify_accept_sample(rows, _cu(np.arange(B + 1, dtype=np.int32) * 2), _cu(toks), _cu(par),
                                              torch.zeros(2 * B, device="cuda"), _cu(noise), want_logprobs=True)
    assert acc.tolist() == [2] * B
    err = np.abs(logp.cpu().numpy()[::2] - want) / np.abs(want)
    assert err.max() <= LOGP_REL


def test_log_p_of_equal_maxima(va):
    """n equal logits and nothing else near: log p = -log n, for tokens in one thread's reach and far apart."""
    V = 40000
    sets = [[7], [7, 8], [0, 39999], [5, 6, 7, 8, 9], list(range(1000)), list(range(0, 40000, 3))]
    lg = torch.full((len(sets), V), -40.0, dtype=torch.float32)
    for r, s in zip(lg, sets):
        r[s] = 4.0
    B = len(sets)
    z = torch.zeros(B, dtype=torch.int32, device="cuda")
    for dt in (torch.float32, torch.bfloat16):
        _, _, bonus, logp = va.verify_accept_sample(lg.to(dt).cuda(), torch.arange(B + 1, dtype=torch.int32, device="cuda"), z,
                                                    z - 1, torch.zeros(B, device="cuda"), torch.ones(B, V, device="cuda"),
                                                    want_logprobs=True)
        assert bonus.tolist() == [s[0] for s in sets]
        want = [-np.log(len(s)) if len(s) > 1 else -np.log1p((V - 1) * np.exp(-44.0)) for s in sets]
        err = [abs(float(x) - w) / abs(w) for x, w in zip(logp.cpu(), want)]
        assert max(err) <= LOGP_REL, err
