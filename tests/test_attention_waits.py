"""The attention kernel's pipeline waits end by themselves, in every order of
events, also once a wait of a CTA has run out.  CPU only: the protocols are
restated here, and the kernel's source is read for what it uses."""
import os
import random
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _kernel():
    """The partial kernel's source, without comments."""
    with open(os.path.join(ROOT, "paged_fp8_kv_attn_b200", "csrc", "attention.cu")) as f:
        text = f.read()
    body = text[text.index("attn_partial_kernel(const"):text.index("attn_merge_kernel(const")]
    return re.sub(r"//[^\n]*", "", body)


class NamedBarrier:
    """bar.arrive / bar.sync by warps: a phase is full after five arrivals, whoever they are."""

    def __init__(self):
        self.count = self.phase = 0

    def arrive(self):
        self.count += 1
        if self.count == 5:
            self.count, self.phase = 0, self.phase + 1

    def wait(self, use):
        self.arrive()
        self.until = self.phase + (self.count > 0)

    def done(self, use, failed):
        return self.phase >= self.until


class MBarrier:
    """Four arrivals a phase; a waiter sees the parity, and gives up at its limit."""

    def __init__(self):
        self.count = self.phase = 0

    def arrive(self):
        self.count += 1
        if self.count == 4:
            self.count, self.phase = 0, self.phase + 1

    def wait(self, use):
        pass

    def done(self, use, failed):
        return self.phase & 1 != (use + 1) & 1 or failed


def producer_ends(kind, uses, rng):
    """A stage used `uses` times by consumers that no longer wait; the producer waits
    before each use but the first.  rng: the order (None: consumers first)."""
    bar = kind()
    arrivals, at, waiting = 4 * uses, 1, False
    while at < uses:
        if arrivals and (rng is None or rng.random() < 0.7):
            bar.arrive()
            arrivals -= 1
            continue
        if not waiting:
            bar.wait(at)
            waiting = True
        if bar.done(at, True):
            at, waiting = at + 1, False
        elif not arrivals:
            return False
    return True


@pytest.mark.parametrize("uses", range(2, 30))
def test_expired_waits_do_not_stall_the_producer(uses):
    """An mbarrier whose waiter leaves once a wait of its CTA has expired lets the
    producer through in any order; a named barrier, whose phases a consumer that runs
    ahead fills by itself, does not (so the kernel has none between the two)."""
    assert producer_ends(MBarrier, uses, None)
    assert all(producer_ends(MBarrier, uses, random.Random(s)) for s in range(50))
    assert not producer_ends(NamedBarrier, uses, None)


def test_pipeline_waits_have_a_limit():
    src = _kernel()
    assert "named_barrier_arrive" not in src and "bar.arrive" not in src
    # barriers without a limit join the consumers only, which all walk the same segments
    syncs = re.findall(r"named_barrier_sync\(([^;]*)\);", src)
    assert syncs and set(syncs) == {"1, kConsumerThreads"}
    # stage barriers are waited for by the call that gives up (each role: full, empty)
    assert not re.findall(r"mbar_(?:try_)?wait\(", src)
    assert set(re.findall(r"wait_or_give_up\(&(\w+)\[", src)) == {"full_bar", "empty_bar"}
