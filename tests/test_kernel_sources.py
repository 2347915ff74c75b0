"""Rules that the kernels' sources keep and that no run shows broken: what a kernel must have waited
for before it touches memory that is not its own."""
import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parents[1] / "q4_moe_speculative_gb300" / "csrc"


def code_of(name, kernel):
    """A kernel's body without comments."""
    text = re.sub(r"//[^\n]*", "", (CSRC / name).read_text())
    at = text.index("{", re.search(rf"\b{kernel}\(const __grid_constant__", text).end())
    depth, i = 0, at
    while True:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
        if depth == 0:
            return text[at:i]


def test_sampling_touches_other_ctas_only_when_they_have_started():
    # a CTA's shared memory may be accessed by the others of its cluster from a cluster barrier on
    body = code_of("sample.cu", "k_sample")
    first = body.index("map_shared_rank")
    arrive, wait = body.find("cluster_arrive()"), body.find("cluster_wait()")
    assert 0 <= arrive < wait < first
    # every thread of the cluster comes past both
    assert "return" not in re.sub(r"return l == l[^;]*;", "", body[:wait])


def test_no_warp_of_the_shared_prefix_kernel_is_left_in_a_barrier():
    # Softmax warps meet in pairs in barriers without a limit, so both of a pair have to come to each:
    # their runs come from one place, and how a wait ended is agreed on by the lanes and then by the pair.
    # No other role has such barriers.
    body = code_of("prefix_tc.cu", "k_prefix_tc")
    at = body.index("if (tid >= T::kFirst)")
    softmax, others = body[at:].split("} else if (warp > 0", 1)
    others = others[:others.rindex("__syncthreads()")]
    assert not re.search(r"barrier\.cta|bar\.sync|__syncthreads", others)
    assert softmax.count("walk.next") == 1
    assert re.search(r"if \(half == 0\) \{\s*if \(!alive \|\| !walk\.next\(a, &run\)\) run\.t1 = 0;", softmax)
    # a vote of the warp in the statement or right behind it, and a meeting before the result is used
    for found in re.finditer(r"(?<!= )\bwait\(&", softmax):
        start = softmax.rfind(";", 0, found.start())
        assert "__all_sync" in softmax[start:softmax.index(";", found.end()) + 60]
    assert not re.search(r"for \([^)]*&& alive", softmax)


def test_copies_in_flight_end_before_the_cta_of_a_shared_prefix():
    # a warp that brings tiles may be done before another gives up: it waits for its last copies always
    body = code_of("prefix_tc.cu", "k_prefix_tc")
    bring = body[body.index("} else if (warp > 0"):body.index("} else if (warp == 0)")]
    waits = [m.start() for m in re.finditer(r"for \(int j = (told|done) - kI?[nR]\w+ < 0", bring)]
    assert len(waits) == 2
    for at in waits:
        assert "abort" not in bring[bring.rindex(";", 0, at):at]


def test_copies_in_flight_end_before_the_cta_of_a_paged_cache():
    body = code_of("paged_tc.cu", "k_paged_tc")
    bring = body[body.index("bulk_copy("):body.index("} else if (warp == T::kMmaWarp)")]
    waits = [m.start() for m in re.finditer(r"for \(int j = done - (ring|kInfo) < 0", bring)]
    assert len(waits) == 2
    for at in waits:
        assert "abort" not in bring[bring.rindex(";", 0, at):at]


READS = r"lengths\[|prefix_len\(|prefix_page\(|__ldg\(|__ldcg\(|\bp\.[xu]\b|o\.q\b|table\[|logits"


@pytest.mark.parametrize("name,kernel", [("prefix_tc.cu", "k_prefix_tc"), ("prefix.cu", "k_prefix_join"),
                                         ("norm.cu", "k_block_norm"), ("sample.cu", "k_sample")])
def test_nothing_is_read_before_the_wait_for_earlier_kernels(name, kernel):
    # griddepcontrol.wait is what makes the results of the kernels before visible, to the grid that
    # executes it; that a grid in between has waited for them is not promised to be enough, unless what
    # that grid released behind its wait has been acquired
    body = code_of(name, kernel)
    before = body[:body.index("pdl_wait()")]
    assert not re.search(READS, before)


def test_the_shared_prefix_kernel_waits_unless_it_has_acquired():
    body = code_of("prefix_tc.cu", "k_prefix_tc")
    acquired = body.index("sh.given = given_is_there(o);")
    everyone = body.index("__syncthreads();", acquired)
    assert everyone < body.index("if (!sh.given) pdl_wait();\n  fence_async_global();")
    assert body.rindex("pdl_wait()") > body.rindex("mbar_wait")      # and for the join's sake at the end
    for name, kernel in (("paged_attn.cu", "k_paged"), ("paged_few.cu", "k_paged_few"),
                         ("paged_tc.cu", "k_paged_tc")):
        text = re.sub(r"//[^\n]*", "", (CSRC / name).read_text())
        assert text.count("pdl_trigger") == (1 if name == "paged_attn.cu" else 0)     # (its join's)
        assert re.search(r"pdl_wait\(\);\s*if \(blockIdx\.x == 0 && tid == 0\) \*a\.status = 0u;\s*"
                         r"if \(a\.pieces && tid == 0\) began\(a\);", text), kernel
