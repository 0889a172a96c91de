"""The calls that the C++ binding marshals: the header's parameter names as
keywords, defaults for err and stream, and what it refuses."""
import re

import pytest

torch = pytest.importorskip("torch")

from _util import HEADER, ensure_library  # noqa: E402

ensure_library()
import decode_dsa_kv_gb300 as d  # noqa: E402
from decode_dsa_kv_gb300 import _abi  # noqa: E402

CALLS = [n for n in dir(_abi._binding) if not n.startswith("_")]


def parameters(name):
    """(name, is a pointer, is a float) of a function's parameters in the header."""
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"\b" + name + r"\s*\(([^)]*)\)\s*;", text, flags=re.S).group(1)
    out = []
    for p in body.split(","):
        p = " ".join(p.split())
        m = re.match(r"(.*?)(\*?\s*)(\w+)$", p)
        out.append((m.group(3), "*" in p, m.group(1).strip() in ("float", "double")))
    return out


def test_the_binding_has_the_paged_caches_calls():
    assert len(CALLS) == 13 and all(getattr(d, n) is getattr(_abi._binding, n) for n in CALLS)


@pytest.mark.parametrize("name", CALLS)
def test_every_parameter_is_a_keyword_of_the_headers_name(name):
    args = {}
    for p, pointer, number in parameters(name):
        args[p] = 0 if p == "stream" else None if pointer else 0.0 if number else 0
    f = getattr(d, name)
    status = f(**args)                       # nothing to do, or refused: nothing is enqueued
    assert status in (_abi.TS_OK, _abi.TS_ERR_INVALID_ARG)
    given = list(args.values())
    assert f(*given) == status
    if "err" in args:
        del args["err"]
        assert f(**args) == status
    with pytest.raises(TypeError, match="no argument"):
        f(**args, no_such=1)
    with pytest.raises(TypeError, match="at most"):
        f(*given, 0)
    first = next(iter(args))
    with pytest.raises(TypeError, match="two values"):
        f(given[0], **args)
    del args[first]
    with pytest.raises(TypeError, match="missing"):
        f(**args)


def test_arguments_of_the_wrong_kind():
    f = d.sfa_chunk_workspace_size
    with pytest.raises(OverflowError):
        f(1 << 40, 1, 1)
    with pytest.raises(TypeError):
        f("3", 1, 1)
    with pytest.raises(AttributeError):
        d.dsa_cache_write(1.5, 512, None, 64, None, 0, None, 0, 0, None, 0)
    assert f(True, 1, 1) == f(1, 1, 1)
