"""CPU model of the ring of per-block scales that a decode kernel's producer
warp fills (decode_kernel.cuh, produce_pages).

The producer's lanes put the scales of up to 32 pages into slots k % 64 at once,
before the first of those pages is issued.  What a slot held, page k - 64, must
have been released by its consumers by then: a lane knows of the releases that
were waited for before its last convergence with the lanes that waited.  The
model walks a stream of segments and keeps, for a lane that runs ahead of lane
0 as far as the warp's convergence points let it, the pages whose release it
knows of; consumers release a page no sooner than somebody waits for it.
"""
import os
import random
import re

import pytest

RING = 64
SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "paged_kv_decode_fa_gb300", "csrc", "decode_kernel.cuh")


def sync_before_store():
    """Whether the source has the warp converge right before the scales' store."""
    with open(SOURCE) as f:
        text = f.read()
    store = text.index("(k + lane) % kBlockScaleRing")
    code = re.sub(r"//[^\n]*", "", text[text.rindex("id = next.id;", 0, store):store])
    return "__syncwarp();" in code


def violations(segments, S, PL, align, sync):
    """Pages whose scales a running-ahead lane overwrites unreleased; segments:
    (pages, from the pool) in order."""
    bad = []
    k = 0
    waited = -1  # every page up to this one was waited for by some lane
    known = -1   # the same, as the lane that runs ahead knows it
    for pages, pooled in segments:
        if pooled:
            known = waited            # the claimed index goes to all lanes
            pad = (align - k % align) % align
            waited = max(waited, k + pad - 1 - S)  # lane 0, for the empty stages
            k += pad
        for p0 in range(0, pages, 32):
            cnt = min(32, pages - p0)
            if sync:
                known = waited
            bad += [k + i - RING for i in range(cnt) if k + i >= RING and k + i - RING > known]
            known = waited            # the convergence after the store
            for i in range(0, cnt, PL):
                known = waited        # each step begins with a shuffle
                waited = k + min(i + PL, cnt) - 1 - S
                if PL > 1:
                    known = waited    # and ends with a convergence
            k += cnt
    return bad


# stages, issuing lanes, pages of a warp step over all warps: the page-split
# kernels at 4, 6 and 16 warps, the column splits, the cascade's prefix pass
CONFIGS = [(8, 4, 4), (16, 4, 4), (12, 4, 6), (32, 8, 16), (12, 4, 1), (8, 4, 1), (8, 1, 1)]


def streams(seed):
    rng = random.Random(seed)
    static = [(rng.randint(0, 90), False) for _ in range(rng.randint(0, 4))]
    return static + [(rng.randint(1, 90), True) for _ in range(rng.randint(0, 8))]


@pytest.mark.parametrize("S,PL,align", CONFIGS + [(32, 1, 1), (32, 1, 16)])
def test_no_scale_is_overwritten_before_its_release(S, PL, align):
    sync = sync_before_store()
    for seed in range(300):
        segs = streams(seed)
        assert not violations(segs, S, PL, align, sync), segs


def test_without_the_convergence_padding_lets_a_lane_ahead():
    """What the convergence is for: 32 stages and up to 15 empty ones before a
    pool segment, or 32 stages and one issuing lane."""
    assert any(violations(streams(s), 32, 8, 16, False) for s in range(300))
    assert any(violations(streams(s), 32, 1, 1, False) for s in range(300))
    assert not any(violations(streams(s), 12, 4, 6, False) for s in range(300))
