"""Limits of the loss that lie in two places of the source."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_linear_algebra_gb300", "csrc")


def test_rows_of_the_gradient_that_is_written_out():
    """The kernel's rows in shared memory are as many as any type's rule lets through, by the rules' own constants."""
    with open(os.path.join(CSRC, "loss.cu")) as f:
        source = f.read()
    assert "__shared__ Row rows[kSlopeRows];" in source
    rule = re.search(r"bool few_logits\(.*?\n}\n", source, re.S).group(0)
    assert "kFewLogitsGrad" in rule and "return few_rows(l.type, l.m, l.w_trans)" in rule
    most = re.search(r"kSlopeRows = std::max\(\{(.*?)\}\)", source).group(1)
    assert {c.strip() for c in most.split(",")} == {"kFewLogitsGrad", "kFewByRow", "kFewByColumn"}
