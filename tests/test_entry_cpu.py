"""The build-and-smoke entry as a program."""
import ast
import os
import sys


ENTRY = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "__graft_entry__.py")


def test_main_comes_last():
    """What `python __graft_entry__.py --smoke` calls is defined when it does."""
    body = ast.parse(open(ENTRY).read()).body
    mains = [i for i, n in enumerate(body) if isinstance(n, ast.If) and "__main__" in ast.unparse(n.test)]
    assert mains == [len(body) - 1]


def test_smoke_from_the_command_line_has_its_parts(monkeypatch):
    """Run as a program with a smoke that only looks its helpers up."""
    source = open(ENTRY).read()
    monkeypatch.setattr(sys, "argv", [ENTRY, "--smoke"])
    names = [n.name for n in ast.parse(source).body if isinstance(n, ast.FunctionDef)]
    assert {"build", "smoke", "_smoke_fp4", "_smoke_step"} <= set(names)
    called = []
    code = source.replace("def build() -> None:", "def build() -> None:\n    return\n\n\ndef _build() -> None:")
    code = code.replace("def smoke() -> None:", "def smoke() -> None:\n    _called.append((_smoke_fp4, _smoke_step))\n\n\ndef _smoke() -> None:")
    exec(compile(code, ENTRY, "exec"), {"__name__": "__main__", "__file__": ENTRY, "_called": called})
    assert len(called) == 1
