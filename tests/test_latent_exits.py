"""Leaving a latent-attention kernel, read from its source: a CTA whose wait ran out in one role must not end while
another role's asynchronous work still writes its memory.  A run cannot show this without a fault on purpose, so the
conditions around the last waits are checked instead: none of them may depend on how the CTA got there."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "compressed_paged_kv_quant_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def conditions(text, at):
    """What stands before each brace that is open at `at`: its statement's head."""
    heads, start = [], 0
    for i in range(at):
        c = text[i]
        if c == "{":
            heads.append(" ".join(text[start:i].split()))
        elif c == "}":
            heads.pop()
        if c in "{};":
            start = i + 1
    return heads + [" ".join(text[start:at].split())]


def unconditional(text, pattern):
    found = [m.start() for m in re.finditer(pattern, text)]
    assert found, pattern
    return any(not re.search(r"timed_out|!ok|\bbad\b", h) for h in
               [" ".join(conditions(text, at)[1:]) for at in found])


@pytest.mark.parametrize("name,wait", [("latent_attn.cu", r"mbar_wait\(BAR\(C::B_FULL \+ i % 3"),
                                       ("latent_prefill.cu", r"mbar_wait\(BAR\(LPB_FULL \+ i % LP_RING"),
                                       ("latent_prefill.cu", r"mbar_wait\(BAR\(LPB_Q\), 0\);")])
def test_copies_land_before_the_cta_ends(name, wait):
    """A copy role that has issued its last copies leaves its loop in good order while they are under way; another role
    may give up on them."""
    assert unconditional(source(name), wait)


@pytest.mark.parametrize("name,wait", [("latent_attn.cu", r"mbar_wait\(BAR\(C::B_END\), 0\);"),
                                       ("latent_prefill.cu", r"mbar_wait\(BAR\(LPB_END\), 0\);")])
def test_mmas_complete_before_the_cta_ends(name, wait):
    """The issuing warp may have issued its last products in good order when the softmax gives up on them."""
    assert unconditional(source(name), wait)
