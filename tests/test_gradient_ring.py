"""The ring of rows that the groups of the gradient rows' bulk kernel share
(csrc/w8a8_input_grad.cuh), as a model: every order in which copies can land
and groups can run is walked through.

Row i belongs to group i % groups and slot i % slots.  The group that is done
with row i asks for row i + slots in its slot.  A slot's barrier has completed
`landed` phases; a wait for phase p by parity is let through when the current
phase's parity differs from p's.
"""
from __future__ import annotations

import pytest


def early_row(slots, groups, rows, counted):
    """The first row found that a group can start on before its copy has
    landed, or None.  counted: a group first waits until its row's copy has
    been asked for."""
    start = (tuple((g, False) for g in range(groups)), tuple(int(s < rows) for s in range(slots)), (0,) * slots)
    seen, todo = {start}, [start]
    while todo:
        state = todo.pop()
        at, issued, landed = state
        after = []
        for s in range(slots):
            if landed[s] < issued[s]:
                after.append((at, issued, landed[:s] + (landed[s] + 1,) + landed[s + 1:]))
        for g in range(groups):
            row, working = at[g]
            if row >= rows:
                continue
            s, phase = row % slots, row // slots
            if working:
                more = issued[:s] + (issued[s] + (row + slots < rows),) + issued[s + 1:]
                after.append((at[:g] + ((row + groups, False),) + at[g + 1:], more, landed))
            elif not (counted and issued[s] <= phase) and landed[s] % 2 != phase % 2:
                if landed[s] != phase + 1:
                    return row
                after.append((at[:g] + ((row, True),) + at[g + 1:], issued, landed))
        for state in after:
            if state not in seen:
                seen.add(state)
                todo.append(state)
    return None


@pytest.mark.parametrize("slots,groups,rows", [(3, 2, 14), (4, 2, 12), (5, 4, 14), (7, 4, 16)])
def test_no_group_starts_on_a_row_that_has_not_landed(slots, groups, rows):
    assert early_row(slots, groups, rows, counted=True) is None


@pytest.mark.parametrize("slots,groups,rows", [(3, 2, 12), (7, 4, 16)])
def test_parity_alone_lets_a_group_through(slots, groups, rows):
    # why the kernel counts: slots that are no multiple of the groups
    assert early_row(slots, groups, rows, counted=False) is not None
