"""What the paged forward's source has to keep and no run can show (no GPU)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def statements():
    """The kernels' source without comments, a statement to an entry."""
    with open(os.path.join(ROOT, "long_context_mask_gb300", "csrc", "bsa_paged_attn.cu"), encoding="utf-8") as f:
        src = f.read()
    src = re.sub(r"//[^\n]*", "", src)
    return [" ".join(x.split()) for x in re.split(r"[;{}]", src) if x.strip()]


def test_lanes_meet_before_instructions_of_a_whole_warp():
    """tcgen05.ld and tcgen05.alloc are executed by all lanes of a warp together: where
    lanes have gone ways of their own before, a __syncwarp() brings them back."""
    st = statements()
    found = 0
    for i, x in enumerate(st):
        if x.startswith(("tmem_ld32(t_row", "tmem_alloc(")):
            found += 1
            # (declarations may stand between)
            before = next(y for y in reversed(st[:i]) if not re.match(r"uint32_t \w+\[\d+\]$", y))
            assert before == "__syncwarp()", (before, x)
    assert found == 2
