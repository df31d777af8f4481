"""CPU test of the tests themselves: a second definition of a name replaces the
first, which then never runs."""
import ast
import glob
import os
from collections import Counter

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(HERE, "*.py"))), ids=os.path.basename)
def test_no_name_is_defined_twice(path):
    with open(path) as f:
        tree = ast.parse(f.read())
    for body in [tree.body] + [n.body for n in tree.body if isinstance(n, ast.ClassDef)]:
        names = Counter(n.name for n in body
                        if isinstance(n, (ast.FunctionDef, ast.AsyncFunctionDef, ast.ClassDef)))
        assert not [n for n, k in names.items() if k > 1]
