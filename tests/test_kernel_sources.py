"""Rules that the kernels' sources keep and that no run shows broken: what a kernel must have waited
for before it touches memory that is not its own."""
import re
from pathlib import Path

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
