"""__graft_entry__.py run as a script: what it calls at its end is defined by then."""
import ast
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_script_part_comes_last():
    with open(os.path.join(ROOT, "__graft_entry__.py"), encoding="utf-8") as f:
        body = ast.parse(f.read()).body
    at = [i for i, x in enumerate(body) if isinstance(x, ast.If) and "__main__" in ast.dump(x.test)]
    assert at == [len(body) - 1]
