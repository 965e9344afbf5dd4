"""What the sources of the token-by-token kernels promise, read as text (CPU)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_context_diffusion_b200", "csrc")
FILES = ("qk_norm_rope.cu", "decode_attn.cu", "evict.cu")


def _functions(src):
    """(name, body) of every function that waits for its predecessor grid."""
    src = re.sub(r"//[^\n]*|__launch_bounds__\([^\n]*", "", src)
    for m in re.finditer(r"\n[\w:<>,*& ]*?\b(\w+)\(([^;{}]*?)\)\s*\{", src):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(src[at], 0)
            at += 1
        body = src[m.end():at]
        if "pdl_wait()" in body:
            yield m.group(1), body


@pytest.mark.parametrize("name", FILES)
def test_nothing_on_the_device_is_read_before_the_wait(name):
    """Only the wait for the predecessor grid orders its writes before this
    grid's reads: lengths, tables, partials and tensors come after it."""
    found = list(_functions(open(os.path.join(CSRC, name)).read()))
    assert found, name
    for fn, body in found:
        before = body[:body.index("pdl_wait()")]
        for what in (r"\bseq_len\(", r"\bparts_of\(", r"\brow_norm\(", r"\bfind_(run|share)\(", r"\bcache_row\(",
                     r"\bturn\(", r"\ba\.\w+\[", r"\bws\.\w+\[", r"\bctx_len\b", r"\bsrc\["):
            assert not re.search(what, before), (fn, what)


def test_the_checked_kernels_are_found():
    names = {fn for f in FILES for fn, _ in _functions(open(os.path.join(CSRC, f)).read())}
    assert {"qk_norm_rope_kernel", "qk_norm_rope_wide_kernel", "decode_kernel", "decode_join_kernel", "add_masses",
            "evict_select_kernel", "cache_compact_kernel"} <= names, names
