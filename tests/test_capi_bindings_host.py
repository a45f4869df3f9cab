"""The raw bindings of the operators around the layer: every checked wrapper
has a caller, so that no second copy of an entry point's argument order lies
untested beside the one in use (ops.py calls the library itself)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CAPI = os.path.join(ROOT, "fp4_weight_moe_gb300", "_capi.py")


def python_files():
    for folder in ("fp4_weight_moe_gb300", "tests", "examples"):
        for base, _, files in os.walk(os.path.join(ROOT, folder)):
            yield from (os.path.join(base, f) for f in files if f.endswith(".py"))


def test_every_wrapper_is_called():
    wrappers = re.findall(r"^def (moe_fp4_(?:fp8|block|route)_\w+)\(", open(CAPI).read(), re.M)
    # calls of the wrappers, not of the library's functions behind lib()
    callers = "\n".join(open(f).read() for f in python_files() if os.path.abspath(f) != CAPI)
    called = set(re.findall(r"(?<!lib\(\)\.)\b(moe_fp4_\w+)\(", callers))
    assert wrappers and not [w for w in wrappers if w not in called]
