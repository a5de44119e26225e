"""Attention over the 8-bit cache: every case that is named for it, on a cache of
codes, against the 64-bit definition over the values that the codes stand for
(tests/paged_more_ref.py derives the tolerances)."""
import pytest

from tests.test_paged_more_gpu import CASES, check, geometry

pytestmark = pytest.mark.gpu


def on_codes(name):
    q_lens, kv_lens, page, tree, kw = CASES[name]
    geom = geometry(q_lens, kv_lens, page, cache_dtype="e4m3", **kw)
    assert geom.cache_dtype == "e4m3"
    return geom, kv_lens, tree


@pytest.mark.parametrize("name", [n for n in CASES if n.startswith("e4m3")])
def test_attention_over_codes_matches_the_definition(name):
    geom, kv_lens, tree = on_codes(name)
    check(geom, kv_lens, 11, tree)


@pytest.mark.parametrize("name", [n for n in CASES if not n.startswith("e4m3")])
def test_sinks_and_trees_over_codes_match_the_definition(name):
    geom, kv_lens, tree = on_codes(name)
    check(geom, kv_lens, 12, tree)
