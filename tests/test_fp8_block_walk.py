"""The block-scaled decode's smaller splits against its workspace: a model of
the host's rule and of the kernel's share arithmetic.  A stream of n tokens
must fall to at most ceil(n / split) + 1 CTAs, in splits or in equal shares of
at least `split` tokens of stages."""
import random

import pytest

from paged_kv_cache_104_gb300 import binding as B

SMS, PER_SM, STAGE_HEADS, STAGE_TOKENS = 152, 3, 16, 64


def split_of(b, hkv, longest):
    streams = hkv // 4 if hkv % 4 == 0 else hkv
    s = 512
    while s > 64 and b * streams * longest < 4 * s * SMS * PER_SM:
        s //= 2
    return s


def slots(longest, s):
    n = -(-longest // s)
    return 1 if n <= 1 else n + 1


@pytest.mark.parametrize("seed", range(60))
def test_rule_and_shares_fit_the_partial_slots(seed):
    rng = random.Random(seed)
    hkv, b = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 7, 40, 200])
    longest = rng.choice([1, 64, 65, 777, 5000, 32768])
    lens = [rng.randint(0, longest) for _ in range(b)]
    lens[0] = longest
    s = split_of(b, hkv, longest)
    hq = hkv * rng.choice([1, 4])
    # the library's own size follows the same rule
    rows = b * hq * slots(longest, s)
    want = 0 if slots(longest, s) == 1 else rows * 130 * 4 + b * hq * 4
    assert 0 <= B.decode_fp8_block_workspace_bytes(b, hq, hkv, 128, longest) - want < 768
    grouped = hkv % 4 == 0
    streams, tok = (hkv // 4, STAGE_HEADS) if grouped else (hkv, STAGE_TOKENS)
    grid = min(b * streams * slots(longest, s), SMS * PER_SM)
    stages = [-(-n // tok) for n in lens for _ in range(streams)]
    total = sum(stages)
    if slots(longest, s) == 1 or total < s // tok * grid:
        assert all(-(-n // s) <= slots(longest, s) for n in lens)        # splits
        return
    cuts = [c * total // grid for c in range(grid + 1)]
    at = 0
    for i, st in enumerate(stages):
        pieces = sum(1 for c in range(grid) if max(cuts[c], at) < min(cuts[c + 1], at + st))
        assert pieces <= max(1, -(-lens[i // streams] // s) + 1) <= slots(longest, s) or st == 0
        at += st
    assert at == total
