"""The waits of the decayed attention's tensor-core kernels, read from their source (CPU).  A warp leaves its role when a
bounded wait runs out, so no role may hold a barrier that counts on all of its warps: there the others would wait for
one that has left, without limit.  The barriers of the whole block stand outside the roles, where every thread comes."""
import os
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "video_diffusion_linear_b200", "csrc",
                   "tc_decay.cu")


def kernel_body(name):
    """The kernel's body without comments, from its opening brace to the matching one."""
    text = re.sub(r"//[^\n]*", "", open(SRC).read())
    start = text.index("{", re.search(r"\b" + name + r"\(const[^;{]*\)\s*\{", text).end() - 1)
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i + 1]
    raise AssertionError(name)


@pytest.mark.parametrize("name", ["k_decay_tc", "k_decay_segments_tc"])
def test_no_role_holds_a_barrier_of_several_warps(name):
    body = kernel_body(name)
    assert "named_bar" not in body and "bar.sync" not in body
    at = [m.start() for m in re.finditer(r"__syncthreads", body)]
    assert len(at) == 3                      # after the set-up, and before and after the teardown's drain
    for i in at:
        assert body[:i].count("{") - body[:i].count("}") == 1, body[i - 200:i]


@pytest.mark.parametrize("name", ["k_decay_tc", "k_decay_segments_tc"])
def test_every_wait_of_a_role_is_bounded(name):
    body = kernel_body(name)
    assert len(re.findall(r"mbar_wait\(", body)) > 3 and "try_wait" not in body
    # every one hands on the abort flag and the status word, and none is left unread
    for m in re.finditer(r"[^;{}]*\bmbar_wait\([^;{]*", body):
        call = m.group(0)
        assert "abort_flag, status)" in call and re.search(r"if \(|return|ok = |&&", call), call


@pytest.mark.parametrize("name", ["k_decay_tc", "k_decay_segments_tc"])
def test_teardown_after_a_timeout_waits_for_the_products(name):
    """Any warp can be the one that gives up, also after the issuing warp has left its role with products in flight:
    their drain stands where all have come together, before the tensor memory is freed."""
    body = kernel_body(name)
    together, freed = [m.start() for m in re.finditer(r"__syncthreads", body)][1:]
    drains = [m.start() for m in re.finditer(r"umma_commit\(&sm\.drain\)", body)]
    assert len(drains) == 1 and together < drains[0] < freed < body.index("tmem_dealloc")
