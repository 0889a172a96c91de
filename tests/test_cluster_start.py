"""Shared memory of another CTA may be touched only when that CTA is known to have
started: in every kernel of a cluster a cluster barrier's wait comes before the
first remote access. Read off the sources, since a kernel that breaks the rule
fails by a race at most."""
import glob
import os
import re

import pytest

from _util import ROOT

CSRC = os.path.join(ROOT, "decode_dsa_kv_gb300", "csrc")
REMOTE = re.compile(r"\b(?:ld|st)_dsmem_\w+\s*\(|\bdsmem_addr\s*\(")
WAIT = re.compile(r"\bcluster_(?:wait|sync_all)\s*\(\)")


def body_at(text, start):
    """The function body whose opening brace is the first one after `start`, outside
    of parentheses."""
    depth = 0
    for i in range(start, len(text)):
        depth += (text[i] == "(") - (text[i] == ")")
        if text[i] == "{" and depth == 0:
            break
    begin, braces = i, 0
    for i in range(begin, len(text)):
        braces += (text[i] == "{") - (text[i] == "}")
        if braces == 0:
            return text[begin:i + 1]
    raise AssertionError("no end")


def kernels():
    out = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
        for m in re.finditer(r"__global__", text):
            body = body_at(text, m.end())
            name = re.search(r"(\w+_kernel\w*)\s*\(", text[m.end():]).group(1)
            if REMOTE.search(body):
                out.append(pytest.param(body, id=f"{os.path.basename(path)}:{name}"))
    return out


def test_the_cluster_kernels_are_found():
    names = {p.id for p in kernels()}
    assert {"chunk.cu:chunk_kernel", "verify.cu:verify_kernel", "topk.cu:topk_cluster_kernel",
            "verify_tree.cu:verify_tree_kernel"} <= names


@pytest.mark.parametrize("body", kernels())
def test_a_cluster_barrier_precedes_the_first_remote_access(body):
    wait = WAIT.search(body)
    assert wait and wait.start() < REMOTE.search(body).start()
