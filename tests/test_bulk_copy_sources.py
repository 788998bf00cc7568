"""The sources of the serving operators' kernels that copy to shared memory in the background: each bounds its waits, and
one that gives up waits for its own copies in flight (with a limit again) before its CTA and its shared memory go."""
import re

import pytest

from tests.test_paged_sources import FILES, code

COPY = r"\b(?:copy_in|bulk_load|tma_load_2d)\("


def kernels(name):
    """The bodies of a file's kernels that start bulk copies."""
    text = code(name)
    found = []
    for m in re.finditer(r"__global__", text):
        at = text.index("{", m.start())
        depth, end = 1, at + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
        if re.search(COPY, text[at:end]):
            found.append(text[at:end])
    return found


def test_the_kernels_are_found():
    assert {n for n in FILES if kernels(n)} == {"lq_attn_paged.cu", "lq_attn_paged_tiles.cu", "lq_attn_q4.cu", "lq_attn_q4_tiles.cu",
                                               "lq_logprobs.cu"}


@pytest.mark.parametrize("name", [n for n in FILES if kernels(n)])
def test_copies_in_flight_are_waited_for(name):
    for body in kernels(name):
        last = [m.start() for m in re.finditer(COPY, body)][-1]
        waits = re.findall(r"mbar_wait_bounded\((?:[^;]*?), kWaitCycles / 8\)", body[last:])
        assert len(waits) == 1, f"{name}: no wait for the copies in flight once a wait has run out"
