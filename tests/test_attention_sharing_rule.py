"""Which calls look at their groups at all: those of up to 64 rows a KV head (entries x query heads of
a KV head), of which two fit an item, and prompts without a form whose entries are many beside
their cache; the others run as without groups.  Told by the workspace, which holds a list of items
where there is a form or groups are looked at."""

import os

import pytest

from speculative_decoding_verification_07_gb300 import binding
from tests.test_attention_form_checks import OK, attention_args, size_of


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from speculative_decoding_verification_07_gb300 import build
        build.build()
    return binding.load_library()


GROUPS = dict(shared_len=1 << 20, shared_members=1 << 20)


@pytest.mark.parametrize("Hq", [2, 8, 14])
@pytest.mark.parametrize("form", [{}, dict(softcap=30.0), dict(window=9)], ids=["plain", "cap", "window"])
def test_groups_of_calls_that_cannot_share(lib, Hq, form):
    group = Hq // 2
    for R in (1, 64 // group, 64 // group + 1, 128 // group + 1, 300, 2041):
        changed = dict(R=R, Hq=Hq, **form)
        without, with_groups = size_of(lib, attention_args(**changed)), size_of(lib, attention_args(**changed, **GROUPS))
        assert without[0] == with_groups[0] == OK
        looked_at = not form and (R * group <= 64 or R > 256)  # (16 blocks of 16 positions)
        assert (with_groups[1] == without[1]) == (not looked_at), (R, group)


def test_groups_of_prompts_over_long_caches(lib):
    """400 entries beside 2000 and 2016 positions."""
    for blocks, looked_at in ((125, True), (126, False)):
        changed = dict(R=400)
        a, b = attention_args(**changed), attention_args(**changed, **GROUPS)
        a.cache.max_blocks = b.cache.max_blocks = blocks
        assert (size_of(lib, a)[1] != size_of(lib, b)[1]) == looked_at


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("tree,Hq", [("binary:3", 10), ("chain:32", 4), ("chain:39", 8)])
@pytest.mark.parametrize("form", [None, "cap", "slopes"])
def test_results_of_calls_that_cannot_share(fmt, tree, Hq, form):
    """65 rows a KV head and more: the bits of the call without groups, whatever the groups hold."""
    from tests import test_gpu_attention_forms as F
    v = binding.Verifier(0)
    x = F.shared_batch(fmt, 128, Hq, 2, 16, tree, True, 20, [5, 60, 0, 9], [3, 1])
    kw = {} if form is None else F.forms_of(form, Hq)
    without = x.run(v, depth=F.ints(x.depth), **F.as_call(kw))
    x.check(without, **kw)
    bad = dict(length=F.ints([320, 16, 7, 320]), members=F.ints([4, 3, -2, 9]))
    for groups in (F.grouped(v, x), bad):
        assert (x.run(v, depth=F.ints(x.depth), groups=groups, **F.as_call(kw)) == without).all()
    assert v.error() == 0
    v.close()
