"""The eviction's rule for sharing a request and holding its weights, against
what the kernel relies on.  CPU only."""
import numpy as np

from evict_modes import shapes

ALONE, STATIC, SM = 1 << 14, 26 * 1024, 227 * 1024


def test_shapes(tmp_path):
    rng = np.random.default_rng(0)
    asked = []
    for _ in range(4000):
        most = int(np.exp(rng.uniform(0, np.log(1 << 19))))
        asked.append((int(np.exp(rng.uniform(0, np.log(3000)))), int(rng.choice([8, 12, 16, 24, 32])), int(rng.choice([1, 2, 4, 8, 40, 152])),
                      most, int(rng.integers(1, most + 1))))
    asked += [(80, 8, 152, 1 << 19, 1 << 19), (1, 8, 152, 1 << 19, 1 << 19), (1, 32, 152, 0, 0), (3, 32, 152, 1, 1)]
    seen = {}
    for (units, chunks, sms, most, n), (cluster, cap, slice_, mode) in zip(asked, shapes(tmp_path, asked)):
        assert cluster in (1, 2, 4, 8) and (cluster == 1 or (units * cluster <= sms and chunks // cluster >= 2))
        assert slice_ % 32 == 0 and slice_ * (1 if n <= ALONE else cluster) >= n
        # bits and counts of 64 keys' words, then the weights: within what the CTA's static arrays leave
        words = (most + 63) // 64 * 2
        assert words * 8 + cap * 2 <= SM - STATIC and cap >= 0
        assert {"whole": slice_ * 4 <= cap * 2, "halves": slice_ * 2 <= cap * 2, "reread": True}[mode]
        if n <= ALONE:
            assert mode != "reread"
        seen[mode] = seen.get(mode, 0) + 1
    assert set(seen) == {"whole", "halves", "reread"}
