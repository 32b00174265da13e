"""What a kernel may write of a row whose copy never came, and how its shared memory is laid out, by the text of the sources:
neither shows in a run that goes well."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_02_gb300", "csrc")


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def body(text, start):
    """From the first brace behind `start` to the one that closes it."""
    i = text.index("{", text.index(start))
    depth = 0
    for k in range(i, len(text)):
        depth += {"{": 1, "}": -1}.get(text[k], 0)
        if depth == 0:
            return text[i:k + 1]
    raise AssertionError(f"{start}: unbalanced")


def test_layer_norm_writes_no_row_that_never_came():
    """A row that a CTA shares is voted on in its meeting, and what is stored before that asks the thread's own wait: after a wait
    that gave up, the stage holds another row or half of one, and residual_out may be the input's own memory."""
    text = source("norm_forward.cuh")
    row = body(text, "void norm_row(")
    meeting = row.index("if (!meet())")  # of a CTA's row; a warp's meets as soon as it has read
    before = row[:meeting]
    stores = [m.start() for m in re.finditer(r"\bstore_chunk|\bstore_codes|\bscale\[", before)]
    assert stores
    guard = before.index("if (a.residual_out && there)")
    guarded = body(before[guard:], "if (a.residual_out && there)")
    assert all(guard < s < guard + len(guarded) + 40 for s in stores)
    assert "a.out" not in before and "a.codes" not in before and "a.scale" not in before
    ring = body(text, "norm_ring_kernel(")
    assert "came && row + w < a.rows, meet)" in ring
    walk = body(source("rmsnorm.cuh"), "void walk(")
    assert re.search(r"const bool ok = mbar_wait\(", walk) and "row_fn(data + st * stage_bytes(), row, ok, [&]" in walk


WORDS = {"float2": 8, "uint2": 8, "int2": 8, "float4": 16, "uint4": 16, "int4": 16, "uint64_t": 8, "double": 8}


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))))
def test_shared_arrays_read_as_words_are_aligned_to_them(name):
    """An array of floats is aligned to a float unless it says more: where it is read or written by wider words, it has to."""
    text = source(name)
    for m in re.finditer(r"__shared__\s+(?:__align__\((\d+)\)\s+)?(\w+)\s+([^;]*);", text):
        align = int(m.group(1) or WORDS.get(m.group(2), 4))
        for array in re.findall(r"(\w+)\s*\[\]", re.sub(r"\[[^\]]*\]", "[]", m.group(3)) + " "):
            for word in re.findall(r"reinterpret_cast<(?:const\s+)?(\w+)\s*\*>\(\s*&?\s*" + array + r"\b", text):
                assert WORDS.get(word, 4) <= align, f"{name}: {array} is aligned to {align} bytes and read as {word}"
