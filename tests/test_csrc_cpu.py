"""What the kernels' sources have to keep to, where a run on a GPU would hardly ever show a fault."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_fp8_mixture_topk_gb300", "csrc")
# what reaches another CTA's shared memory, or is an address there
REMOTE = re.compile(r"\b(?:st|ld|red|atom)\.[\w.]*shared::cluster|\bcluster_map\(|\bmbar_arrive_cluster\(|\bmbar_arrive_release_cluster\(")
ALL_THERE = re.compile(r"\bcluster_barrier\(\)|\bcluster_wait\(\)")


def kernels():
    """(file, text of the body) of each __global__ function."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__\b[^;{]*?\)\s*\{", text):
            depth, i = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[i], 0)
                i += 1
            yield os.path.basename(path), text[m.end():i]


def test_clusters_wait_for_their_ctas():
    """No kernel reaches for another CTA's shared memory before a barrier of the cluster has completed: until then that CTA need
    not have started."""
    seen = 0
    for name, body in kernels():
        remote = REMOTE.search(body)
        if remote:
            seen += 1
            there = ALL_THERE.search(body)
            assert there and there.start() < remote.start(), f"{name}: {body[remote.start():remote.start() + 60]!r}"
    assert seen >= 4   # the 8-bit, the 16-bit and the 4-bit products, the router's sums


def test_cluster_barriers_are_whole():
    """Each early arrival at a cluster's barrier has its wait, and no kernel arrives twice without one."""
    for name, body in kernels():
        steps = re.findall(r"\bcluster_(arrive|wait)\(\)", body)
        assert steps == ["arrive", "wait"] * (len(steps) // 2), name


EXCHANGE = re.compile(r"\b(?:warp_max|warp_sum|lanes_max<\w+>|lanes_sum<\w+>|chosen_sum|__shfl\w*_sync|__any_sync|__all_sync|__ballot_sync|"
                      r"__reduce_\w+_sync|__syncwarp|__syncthreads\w*|half_ok)\(")


def test_no_exchange_behind_a_short_circuit():
    """What a whole warp or block has to enter does not stand behind &&, || or ?:, which lets some of its threads past it (a
    constant's, in capitals, is the same for all)."""
    def statements(text):
        """Pieces between braces and the semicolons outside of parentheses; headers of if, for and while by themselves."""
        depth, start = 0, 0
        for i, c in enumerate(text):
            depth += {"(": 1, ")": -1}.get(c, 0)
            header = c == ")" and depth == 0 and re.match(r"\s*(?:else\s+)?(?:if(?:\s+constexpr)?|for|while)\s*\(", text[start:i])
            if header or (c in ";{}" and depth == 0) or c in "{}":
                yield text[start:i + 1]
                start = i + 1
                depth = 0 if c in "{}" else depth

    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*|#[^\n]*", "", open(path).read())
        for part in statements(text):
            for m in EXCHANGE.finditer(part):
                seen += 1
                before = re.sub(r"\b[A-Z][A-Z0-9_]* (?:\?|&&)", "", part[:m.start()])
                assert not re.search(r"&&|\|\||\?", before), f"{os.path.basename(path)}: {' '.join(part.split())}"
    assert seen > 100


if __name__ == "__main__":
    pytest.main([__file__])
