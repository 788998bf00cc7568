"""How lq_token_logprobs divides rows among CTAs (host code, no GPU)."""
import os
import subprocess

import pytest

from lattice_vq_weight_gb300 import build

SMS = 152
CLUSTERS = {1: SMS, 2: 76, 4: 36, 8: 16}       # at once, one CTA per SM
MOST = 208 * 1024 - 32                         # bytes of a share in shared memory at once

PROGRAM = r"""
#include <cstdio>
#include "lq_logprobs_plan.h"
int main() {
  long long rows, vocab;
  int esize;
  while (std::scanf("%lld %lld %d", &rows, &vocab, &esize) == 3) {
    lq::score::Plan p;
    if (!lq::score::make_plan(rows, vocab, esize, [](int c) { return c == 1 ? 152 : c == 2 ? 76 : c == 4 ? 36 : 16; }, &p))
      return 1;
    std::printf("%d %lld %d %d %d %lld\n", p.d.cluster, (long long)p.d.share, p.d.segment, p.d.per_piece, p.d.chunks,
                (long long)p.clusters);
  }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """plans([(rows, vocab, bytes of a logit), ...]): (CTAs per row, share, segment, chunks of a piece, chunks, clusters)."""
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", build.CSRC, str(at / "plan.cpp"), "-o",
                    str(at / "plan")], check=True)

    def ask(calls):
        text = "\n".join(" ".join(map(str, c)) for c in calls)
        out = subprocess.run([str(at / "plan")], input=text, capture_output=True, text=True, check=True).stdout
        got = [tuple(map(int, line.split())) for line in out.splitlines()]
        assert len(got) == len(calls)
        return list(zip(calls, got))
    return ask


def calls():
    """Vocabularies around those that fill the shared memory of 1, 2, 4 and 8 CTAs, and others, with few rows to many."""
    for esize in (2, 4):
        full = [c * (MOST // esize) + d for c in (1, 2, 4, 8) for d in range(-9, 18)]
        for vocab in [1, 2, 7, 1000, 2049, 32000, 50001, 128256, 262144, 1 << 20, 1 << 24] + full:
            for rows in (1, 2, 20, 76, 77, 96, 152, 153, 256, 304, 2047, 1 << 24):
                yield rows, vocab, esize


def test_a_row_is_divided_whole_and_fits(plans):
    for (rows, vocab, esize), (ctas, share, segment, per_piece, chunks, clusters) in plans(list(calls())):
        assert ctas in (1, 2, 4, 8) and (ctas - 1) * share < vocab <= ctas * share
        assert 0 < segment <= share and chunks * 16 >= segment * esize + 15 and 4 * per_piece >= chunks
        assert chunks * 16 <= 208 * 1024 and 1 <= clusters <= rows


def test_a_share_stays_in_shared_memory_where_a_cluster_can_hold_the_row(plans):
    """Only rows that eight CTAs cannot hold are read in segments, and so more than once."""
    for (rows, vocab, esize), (ctas, share, segment, *_) in plans(list(calls())):
        if segment < share:
            assert ctas == 8 and -(-vocab // 8) * esize > MOST, (rows, vocab, esize)


def test_no_more_clusters_than_the_device_holds(plans):
    """A CTA has 17 warps of 94 registers a thread and more: two do not fit an SM, however small their shares are.
    Those past the first round would start cold, where a resident one has its next row under way."""
    for (rows, *_), (ctas, *_, clusters) in plans(list(calls())):
        assert clusters == min(rows, CLUSTERS[ctas])
