"""Every role of the tensor-memory kernel reports a wait that it gives up (by
reading its source: no input makes a wait run out)."""
import os
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "selective_state_space_51_b200", "csrc",
                   "kernel_linattn_tc.cuh")
# where each role's code starts, in order
ROLES = ["// ---- q, k, v in (stage it % 2), y out",
         "// ---- products, in a converged warp",
         "// ---- decays: every second chunk each",
         "// ---- scores: P -> P'",
         "// ---- the weighted values and the state; lane",
         "// ---- y; lane: a step"]
END = "if (warp == 13) tc::tmem_free"


def code_of(role):
    text = open(SRC).read()
    at = [text.index(r) for r in ROLES] + [text.index(END)]
    assert at == sorted(at)
    i = ROLES.index(role)
    return re.sub(r"//.*", "", text[at[i]:at[i + 1]])


@pytest.mark.parametrize("role", ROLES)
def test_a_role_that_gives_up_says_so(role):
    code = code_of(role)
    waits = [m.start() for m in re.finditer(r"\bwait\(|\bchunk_in\(|\bweigh\(",
                                            code)]
    said = [m.start() for m in re.finditer(r"gt\.dead = 1;", code)]
    assert waits and said
    # after the loop that waits, not somewhere in front of it
    assert max(said) > max(waits)


def test_the_last_products_are_reported():
    code = code_of(ROLES[1])
    assert "gt.dead = 1;" in code[code.index("tc::commit(e, bar(kFin))"):]


def test_the_block_passes_it_on():
    text = open(SRC).read()
    assert "if (threadIdx.x == 0 && gt.dead) *pp.status = 1;" in text
