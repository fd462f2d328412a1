"""What a gathered decode's lanes note of a tile in shared memory is read by all lanes of the warp: between a note and the
next read, and between a read and the next note, the kernel's loop has a __syncwarp (CPU; the order in the source)."""

import os
import re

import pytest

from conftest import ROOT

TOKENS = re.compile(r"if constexpr \((?P<not>!?)F::kSteps\)|(?P<note>\bnote\()|(?P<keys>\bissue_keys\(\))|(?P<values>\bissue_values\(\))"
                    r"|(?P<sync>__syncwarp\(\))|lds\((?P<read>metas|steps)\b")


def block(text, at):
    """The text between the brace that opens at or behind `at` and its own."""
    at = text.index("{", at)
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at + 1:i]
    raise AssertionError("unbalanced braces")


def without_comments(text):
    return re.sub(r"//[^\n]*", "", text)


def events(text, parts, has_steps):
    """Notes, warp barriers and reads in a piece of the source in their order, calls of `parts` put in."""
    out, at = [], 0
    while m := TOKENS.search(text, at):
        at = m.end()
        if m.group("not") is not None:                      # a branch of the formats with steps, or of those without
            if (m.group("not") == "!") == has_steps:        # not taken: a block, or one statement
                rest = text[at:].lstrip()
                at = text.index("{", at) + len(block(text, at)) + 2 if rest.startswith("{") else text.index(";", at) + 1
            continue
        if m.group("keys"):
            out += events(parts["keys"], parts, has_steps)
        elif m.group("values"):
            out += events(parts["values"], parts, has_steps)
        else:
            out.append("note" if m.group("note") else "sync" if m.group("sync") else m.group("read"))
    return out


def faults(trace):
    """Pairs of a note and a read, either way round, with no barrier between."""
    found, noted, read = [], False, False
    for e in trace:
        if e == "sync":
            noted = read = False
        elif e == "note":
            if read:
                found.append("read, note")
            noted = True
        else:
            if noted:
                found.append(f"note, {e}")
            read = True
    return found


def traces(has_steps):
    path = os.path.join(ROOT, "paged_kv_cache_126_gb300", "csrc", "gather_kernel.cuh")
    text = without_comments(open(path).read())
    parts = {"keys": block(text, text.index("auto issue_keys = ")), "values": block(text, text.index("auto issue_values = "))}
    first = text.index("for (int k = 0; k < STAGES && issued < count; ++k)")
    loop = text.index("while (i < count && !stuck)")
    tile = block(text, text.index("for (; i < stop; ++i, ++got)"))
    start = events(text[first:loop], parts, has_steps)
    return start, events(tile, parts, has_steps)


@pytest.mark.parametrize("has_steps", [False, True])
def test_notes_are_seen_by_the_whole_warp(has_steps):
    start, tile = traces(has_steps)
    assert start.count("note") == 1 and tile.count("note") == 1 and "metas" in tile and ("steps" in tile) == has_steps
    assert not faults(start + 3 * tile)


def test_a_missing_barrier_is_found():
    assert faults(["note", "metas"]) == ["note, metas"] and faults(["steps", "note"]) == ["read, note"]
    assert not faults(["note", "sync", "metas", "sync", "note"])
