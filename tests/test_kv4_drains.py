"""Copies under way when a wait of the cache's attention kernels gives up,
modelled on the CPU.

Every wait is bounded; a warp whose wait gives up takes no further step.  Bulk
copies that it (or another warp) has asked for still write into the CTA's
shared memory, which belongs to the next CTA once this one has left: before that
they have to be waited for, each on its slot's barrier and with the parity of its
phase.  No test can make a copy stay away without a GPU fault, so the rings'
bookkeeping is run here, with a wait given up at every place, and the waits that
the kernels then make are compared with the copies that are under way.  Ring
depths and the waits themselves are read from the kernel source.
"""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).resolve().parents[1] / "activation_sparse_moe_gb300" / "csrc"


def _squeeze(path):
    return re.sub(r"\s+", " ", re.sub(r"//[^\n]*", "", (CSRC / path).read_text()))


def few_row_waits(steps, give_up, slots, drains):
    """The ring of one warp of kv4_decode_kernel: `steps` steps, the wait of step
    `give_up` runs out (None: none does).  Returns the copies under way that are not
    waited for, and the waits that are made for nothing."""
    uses = [0] * slots                 # copies asked for, by slot
    done = [0] * slots                 # copies waited for
    in_slot = slot = asked = 0
    phase = 0

    def load():
        nonlocal in_slot, asked
        if asked < steps:
            uses[in_slot] += 1
            asked += 1
            in_slot = 0 if in_slot + 1 == slots else in_slot + 1
    for _ in range(slots):
        load()
    wrong = []

    def wait(s, parity):
        # the copy waited for is the slot's oldest: its phase's parity
        if done[s] == uses[s] or done[s] & 1 != parity:
            wrong.append((s, parity))
        else:
            done[s] += 1
    for step in range(steps):
        if phase < 2 and step == give_up:
            phase |= 2
        if phase >= 2:
            continue
        wait(slot, phase)
        slot += 1
        if slot == slots:
            slot, phase = 0, phase ^ 1
        load()
    if phase >= 2 and drains:
        while True:
            wait(slot, phase & 1)
            slot += 1
            if slot == slots:
                slot, phase = 0, phase ^ 1
            if slot == in_slot:
                break
    return [s for s in range(slots) if done[s] != uses[s]], wrong


def test_few_row_kernel_waits_for_its_copies():
    src = _squeeze("hs_kv4_attn.cu")
    slots = int(re.search(r"kSlots = (\d+);", src)[1])
    drains = ("if (phase >= 2) { do { mbar_wait(full + slot, phase & 1); if (++slot == C::kSlots) slot = 0, phase ^= 1; } "
              "while (slot != in_slot); }") in src
    for steps in range(1, 4 * slots + 2):
        for give_up in [None, *range(steps)]:
            left, wrong = few_row_waits(steps, give_up, slots, drains)
            assert not wrong
            assert not left, (steps, give_up, left)


def chunk_waits(fills, taken, slots, drains):
    """The loading warp of kv4_prefill_kernel: it has filled `fills` stages, of which the
    other warps have waited for the first `taken`.  The waits at its end."""
    under_way = {(i % slots, i // slots & 1) for i in range(taken, fills)}
    made = set()
    if drains:
        for i in range(fills - slots if fills > slots else 0, fills):
            made.add((i % slots, i // slots & 1))
    return under_way - made


def test_chunk_kernel_waits_for_its_copies_and_products():
    src = _squeeze("hs_kv4_prefill.cu")
    slots = int(re.search(r"kPfPacked = (\d+)", src)[1])
    drains = ("for (uint32_t i = f > kPfPacked ? f - kPfPacked : 0; i < f; ++i) "
              "mbar_wait(sh.packed_full + i % kPfPacked, (i / kPfPacked) & 1);") in src
    for fills in range(0, 5 * slots):
        # a stage is filled again only after its last copy has been taken
        for taken in range(max(0, fills - slots), fills + 1):
            assert not chunk_waits(fills, taken, slots, drains), (fills, taken)
    # products: all of them are committed and waited for before tensor memory is given back
    end = src.index("tmem_dealloc(tmem, 512)")
    assert re.search(r"umma_commit\(&sh\.products_done\); __syncwarp\(\); mbar_wait\(&sh\.products_done, 0\);", src[:end])
    assert "mbar_init(&sh.products_done, 1);" in src


def test_joins_in_shared_memory_wait_for_their_copies():
    src = _squeeze("hs_kv4_prefill.cu")
    assert "if (!mbar_wait(bar, 0)) { mbar_wait(bar, 0); return; }" in src


@pytest.mark.parametrize("name", ["hs_kv4_attn.cu", "hs_kv4_prefill.cu"])
def test_every_wait_is_bounded(name):
    src = _squeeze(name)
    assert "mbarrier.try_wait" not in src and "mbarrier.test_wait" not in src  # only through mbar_wait, which gives up
    assert not re.search(r"while \(!mbar_(try_wait|test)", src)


def test_a_warp_gives_up_as_one():
    """Lanes run out of patience one by one; a warp in which some have and some have
    not would meet its next vote or shuffle in parts and hang there.  So what a wait
    returns decides only by way of a vote; the ones at a warp's end decide nothing."""
    wait = _squeeze("hs_kv4.cuh").split("bool warp_wait(")[1].split("True in one lane")[0]
    assert wait.count("mbar_try_wait(") == wait.count("__all_sync(~0u, mbar_try_wait(bar, parity))") == 2
    assert "if (__any_sync(~0u, clock64() - t0 > kWaitLimitCycles)) { atomicOr(&g_status, 1u); return false; }" in wait
    for name, decided in (("hs_kv4_attn.cu", 0), ("hs_kv4_prefill.cu", 1)):
        src = _squeeze(name)
        uses = [m.start() for m in re.finditer(r"\bmbar_wait\(", src)]
        assert uses
        # a statement of its own, but for the one of add_pieces_at_end, which returns at once
        assert sum(1 for at in uses if not re.search(r"[;{})] $", src[:at])) == decided, name
