"""What the sources of the calls on a cache in 4 bits have to keep and no run can show (no GPU)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def code(name):
    """A source without comments, white space as single blanks."""
    with open(os.path.join(ROOT, "long_context_mask_gb300", "csrc", name), encoding="utf-8") as f:
        return " ".join(re.sub(r"//[^\n]*", "", f.read()).split())


def test_a_descriptor_is_handed_back_after_the_last_wait_that_it_guards():
    """q_ready[k % kDesc] is waited for by its phase's parity, and goes on to the next phase with
    segment k + kDesc, which is told once every warp has handed segment k back: a warp that waits for it
    holds the descriptor until then (else it can miss the phase, and wait out its limit)."""
    src = code("bsa_fp4_prompt.cu")
    loops = src.split("next_segment(k, ok);")[1:]
    waits = 0
    for body in loops:
        at = body.find("paged_wait(smem_u32(&sh.q_ready"), body.find("wait_warp(smem_u32(&sh.q_ready")
        at = max(at)
        if at < 0:
            continue
        waits += 1
        # (what a segment without a key hands back on its way to the next one is no matter: nothing waits there)
        before = re.sub(r"if \(n == 0\) \{ hand_back\(k\); continue; \}", "", body[:at])
        assert "hand_back" not in before, before[-300:]
        assert "hand_back(k)" in body[at:]
    assert waits == 2  # (the warp that issues Q K^T, and the softmax)
