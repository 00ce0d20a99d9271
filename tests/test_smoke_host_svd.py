"""CPU: smoke() takes no decomposition on the GPU (torch loads a library of its
own for those, which a profiled or trimmed-down process may not find)."""
import ast
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_smoke_decomposes_on_the_host():
    with open(os.path.join(ROOT, "__graft_entry__.py")) as f:
        tree = ast.parse(f.read())
    calls = [c for c in ast.walk(tree) if isinstance(c, ast.Call) and "torch.linalg." in ast.unparse(c.func)]
    assert calls
    for c in calls:
        assert ".cpu()" in ast.unparse(c.args[0]), ast.unparse(c)
