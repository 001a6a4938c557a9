"""The launchers' rules that tests/product_forms.py repeats are those of the sources."""
import os

import pytest

from product_forms import CSRC, RULES


@pytest.mark.parametrize("name", sorted(RULES))
def test_rules_are_those_of_the_sources(name):
    with open(os.path.join(CSRC, name)) as f:
        text = " ".join(f.read().split())
    for rule in RULES[name]:
        assert " ".join(rule.split()) in text, rule
