"""The sizes of tests/test_gpu_mx_forms.py reach every kernel of the MXFP4 products."""

import hashlib

import mx_forms


def test_rules_are_those_of_the_sources():
    """The text that tests/mx_forms.py follows.  After a change to it, bring
    dense_form, experts_form and the sizes in line, then this digest."""
    assert hashlib.sha256(mx_forms.rules().encode()).hexdigest()[:16] == "a84361fd0caa5ce8"


def test_every_kernel_has_a_size():
    reached = {mx_forms.dense_cases_form(*c) for c in mx_forms.DENSE}
    reached |= {mx_forms.experts_cases_form(*c) for c in mx_forms.EXPERTS}
    there = mx_forms.forms_in_sources()
    assert there - reached == set() and reached - there == set()
