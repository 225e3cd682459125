"""Which copies the attention kernels wait for after a wait that ran out, checked
on the CPU.

A bulk copy in flight when its CTA returns would write into memory that is no longer
the CTA's.  So a kernel that gives up waits for its copies first, on their
barriers: a parity wait returns at once unless the barrier's phase is the one in
which the copy was issued, so a wait with the wrong parity protects nothing, and a
wait for a phase that no copy completes runs to its limit.  The models repeat the
index arithmetic of `kv_attn_few_kernel` and of `tile_copy_bulk` and
`tile_drain`; an edit to those must be made here too."""
import pytest


def protects(waits, copies, landed):
    """Whether the waits (barrier, parity), with no copy of `copies`
    (barrier, fill number) but those in `landed` complete, hold back until all
    others are, and would return once they are."""
    left = [c for c in copies if c not in landed]
    phase = {}  # a barrier's current phase: the fills of it that completed
    for bar, fill in copies:
        phase[bar] = min(phase.get(bar, fill), fill) if (bar, fill) in left else max(phase.get(bar, 0), fill + 1)
    for bar, fill in left:
        phase[bar] = fill
    held = {bar for bar, parity in waits if bar in phase and (phase[bar] & 1) == parity}
    return {bar for bar, _ in left} == held


def few_copies(total, stages, died):
    """Parts in flight at most when part `died` was waited for in vain."""
    return [(t % stages, t // stages) for t in range(died, min(died + stages, total))]


def few_drain(total, stages, died):
    return [(t % stages, (t // stages) & 1) for t in range(died, min(died + stages, total))]


def few_drain_by_the_running_stage(total, stages, died):
    """What does not do: parities from where the ring stands after the rest of the
    parts were passed over."""
    stage, phase = total % stages, (total // stages) & 1
    return [(i, phase ^ 1 if i < stage else phase) for i in range(stages)]


def every(total, stages):
    for died in range(total):
        copies = few_copies(total, stages, died)
        for bits in range(1 << len(copies)):
            yield died, copies, [c for i, c in enumerate(copies) if bits >> i & 1]


@pytest.mark.parametrize("stages", [2, 3])
def test_rows_of_16_wait_for_what_was_copied_ahead(stages):
    for total in range(1, 14):
        for died, copies, landed in every(total, stages):
            assert protects(few_drain(total, stages, died), copies, landed), (total, died, landed)


@pytest.mark.parametrize("stages", [2, 3])
def test_parities_of_the_running_stage_would_not_do(stages):
    wrong = [not protects(few_drain_by_the_running_stage(total, stages, died), copies, landed)
             for total in range(1, 14) for died, copies, landed in every(total, stages)]
    assert any(wrong) and not all(wrong)


def tile_drain(slots, copied, landing):
    waits = [(i % slots, (i // slots) & 1) for i in range(max(copied - slots, 0), copied)]
    return waits + ([("landed", landing)] if landing >= 0 else [])


@pytest.mark.parametrize("slots", [5, 8])
@pytest.mark.parametrize("positions", [1, 2, 3, 7, 8])
def test_tiles_wait_for_the_ring_and_a_tile_being_mended(slots, positions):
    # tile 2j holds keys and 2j + 1 values of position tile j; the first and last values are mended
    for mended in ({1}, {2 * positions - 1}, {1, 2 * positions - 1}, set()):
        for given_up in range(2 * positions + 1):  # at the wait before tile given_up, or after the last
            for in_mend in (False, True):
                if in_mend and given_up not in mended:
                    continue
                fills = [(i % slots, i // slots) for i in range(max(given_up - slots, 0), given_up)]
                done = [(i % slots, i // slots) for i in range(max(given_up - slots, 0), given_up) if i in mended]
                landing, copies = -1, list(fills)
                if in_mend:  # its slot's tile before it was read, so it has landed
                    before = len([i for i in mended if i < given_up])
                    landing, copies = before & 1, copies + [("landed", before)]
                    if given_up >= slots:
                        done.append((given_up % slots, given_up // slots - 1))
                waits = tile_drain(slots, given_up, landing)
                rest = [c for c in copies if c not in done]
                for bits in range(1 << len(rest)):
                    landed = done + [c for i, c in enumerate(rest) if bits >> i & 1]
                    assert protects(waits, copies, landed), (positions, given_up, in_mend, landed)
