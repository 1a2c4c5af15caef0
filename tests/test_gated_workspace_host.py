"""The partial sums' share of zero_gated_workspace (no GPU): a worker keeps less than 8 parts of either kind of tile, 256 KB
each on 76 pairs of SMs and 64 KB on 152 single ones; a part's sums have 16 tickets of 4 bytes."""
import random

import zero_sharded_mixed_03_gb300 as Z

KIND = 8 * 76 * ((256 << 10) + 64)


def up(n, to):
    return -(-n // to) * to


def sums_bytes(m, k, n, back, layout=0, dx=True, up_too=True):
    a = Z.zero_gated_t(rows=m, in_features=k, out_features=n, dtype16=Z.ZERO_BF16, layout=layout,
                       activation=Z.ZERO_ACT_SILU, ld_x=up(k, 8), ld_w_gate=up(max(k, n), 8), ld_w_up=up(max(k, n), 8), x=4096,
                       w_gate=8192, w_up=16384, h=32768, gate=65536, up=1 << 17, dh=1 << 18, dx=(1 << 19) if dx else None,
                       dw_gate=1 << 20, dw_up=(1 << 21) if up_too else None)
    return Z.zero_gated_workspace(a, back) - (2 * up(2 * m * up(n, 8), 256) if back else 0)


def test_partial_sums_are_bounded():
    r = random.Random(1)
    for i in range(4000):
        m, k, n = (int(2 ** r.uniform(2, 16)) for _ in range(3))
        assert 0 <= sums_bytes(m, k, n, False, i % 2) <= KIND
        both = sums_bytes(m, k, n, True, i % 2, r.random() < 0.8, r.random() < 0.8)
        assert 0 <= both <= 2 * KIND
    # sizes that have both kinds in parts
    most = 0
    for i in range(4000):
        m, k, n = 256 * r.randint(60, 260), 256 * r.choice([1, 1, 1, 2, 3]), 256 * r.randint(60, 260)
        both = sums_bytes(m, k, n, True, 0, True, r.random() < 0.3)
        assert 0 <= both <= 2 * KIND
        most = max(most, both)
    assert most > KIND and sums_bytes(50688, 256, 42752, True, 0, True, False) > KIND
