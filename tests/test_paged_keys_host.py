"""The keys that a row tile of paged attention reads, against brute force over the
definition (no GPU): the function that every kernel takes them from, compiled by itself."""
import os
import random
import subprocess

import pytest

from attention_swa_forward_gb300 import build as B

SOURCE = """#include <cstdio>
#include "swa_paged.h"
using namespace swa;
int main() {
  int tree, pre, next, sinks, n, m, tok0, toks, shift;
  while (std::scanf("%d %d %d %d %d %d %d %d %d", &tree, &pre, &next, &sinks, &n, &m, &tok0, &toks, &shift) == 9) {
    static const uint32_t bits = 0;
    PagedArgs a{};
    a.sparse_mode = 4;
    a.pre = pre, a.next = next, a.sinks = sinks;
    a.tree = tree ? &bits : nullptr;
    const PagedKeys k = paged_keys<true>(a, n, m, tok0, toks);
    const PagedUnits u = paged_units<true>(k, shift);
    std::printf("%d %d %d %d", k.lo, k.hi, k.sinks, u.total);
    for (int x = 0; x < u.total; ++x) std::printf(" %d", u.at(x));
    std::printf("\\n");
  }
}
"""


@pytest.fixture(scope="module")
def keys_of(tmp_path_factory):
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(B._nvcc()))), "include")
    d = tmp_path_factory.mktemp("keys")
    (d / "keys.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", B.CSRC, "-I", B.INCLUDE, "-I", cuda, str(d / "keys.cpp"), "-o",
                    str(d / "keys")], check=True)

    def call(cases):
        text = "".join(" ".join(map(str, c)) + "\n" for c in cases)
        r = subprocess.run([str(d / "keys")], input=text, capture_output=True, text=True, check=True)
        return [list(map(int, line.split())) for line in r.stdout.splitlines()]

    return call


def needed(tree, pre, nxt, sinks, n, m, tok0, toks):
    """Keys that some token of the tile may see.  A tree: any bits and depths, and so all of the chunk."""
    before = n - m
    need = set()
    for i in (range(m) if tree else range(tok0, tok0 + toks)):
        p = before + i  # (of a tree: every depth that a token may have)
        for j in range(n):
            if tree and j >= before:
                need.add(j)
            elif j <= p + nxt and (j >= p - pre or j < sinks):
                need.add(j)
    return need


def draws(count, trees):
    r = random.Random(3)
    for x in range(count):
        n, m = r.randint(0, 90), r.randint(1, 40)
        pre = r.choice([r.randint(0, 100), r.randint(0, 6), r.randint(-60, -1)])
        nxt = max(-pre, r.choice([0, r.randint(0, 30), r.randint(-30, 0)]))
        tok0 = r.randint(0, m - 1)
        yield (int(trees), pre, max(nxt, 0) if trees else nxt, r.choice([0, 0, r.randint(1, 5), r.randint(1, 100)]), n, m,
               tok0, r.randint(1, m - tok0), r.choice([4, 7]))


@pytest.mark.parametrize("trees", [False, True])
def test_every_key_that_a_token_may_see_is_read(keys_of, trees):
    cases = list(draws(4000, trees))
    for case, (lo, hi, sinks, total, *units) in zip(cases, keys_of(cases)):
        need = needed(*case[:8])
        read = set(range(lo, hi + 1)) | set(range(sinks))
        assert need <= read, (case, lo, hi, sinks, sorted(need - read))
        assert read <= set(range(case[4])), case
        # runs of 2^shift keys: each that holds a key, once, in ascending order
        assert len(units) == total == len(set(units)) and units == sorted(units), case
        assert set(units) == {j >> case[8] for j in read}, case


def test_a_tree_reads_its_whole_chunk_whatever_the_window(keys_of):
    """A window that begins ahead of a token leaves the context out, not the chunk."""
    for pre in (-1, -5, -200):
        (lo, hi, sinks, _, *_), = keys_of([(1, pre, 300, 0, 100, 5, 0, 5, 4)])
        assert (lo, hi, sinks) == (95, 99, 0), pre
        (lo, hi, sinks, _, *_), = keys_of([(1, pre, 300, 7, 100, 5, 2, 1, 4)])
        assert (lo, hi, sinks) == (95, 99, 7), pre
