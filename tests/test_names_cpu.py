"""Every test is one that pytest finds: a second function of a name in a file
takes the first one's place, which then never runs."""
import ast
import glob
import os

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(HERE, "**", "*.py"), recursive=True)), ids=lambda p: os.path.relpath(p, HERE))
def test_names_are_used_once(path):
    with open(path) as f:
        tree = ast.parse(f.read())
    for scope in [tree, *(c for c in ast.walk(tree) if isinstance(c, ast.ClassDef))]:
        names = [d.name for d in scope.body if isinstance(d, (ast.FunctionDef, ast.AsyncFunctionDef, ast.ClassDef))]
        assert len(names) == len(set(names)), sorted(n for n in set(names) if names.count(n) > 1)
