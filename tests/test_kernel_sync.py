"""What orders the kernels' copies and arrivals, by the text of the sources: mistakes here show as wrong rows in one call of
many, or in none on a quiet GPU, so they are looked for on the CPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_02_gb300", "csrc")
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


def asm_strings(name):
    """The inline PTX of a source: each asm statement's string literals put together."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    out = []
    for m in re.finditer(r"\basm\s*(?:volatile)?\s*\(", text):
        lits, rest = [], text[m.end():]
        while (lit := re.match(r'\s*"((?:[^"\\]|\\.)*)"', rest)):
            lits.append(lit.group(1))
            rest = rest[lit.end():]
        out.append("".join(lits))
    return out


def test_the_reader_sees_the_sources():
    assert any("tcgen05.mma" in a for a in asm_strings("common.cuh"))
    assert any("cp.async.bulk.shared::cluster.shared::cta" in a for a in asm_strings("sparse_mla.cu"))


@pytest.mark.parametrize("name", SOURCES)
def test_bulk_groups_wait_for_copies_that_join_them(name):
    """A bulk async-group takes the copies that complete on groups (.bulk_group).  Those that count bytes on an mbarrier
    join none, and waiting for a group does not wait for them."""
    asm = asm_strings(name) + asm_strings("common.cuh")
    if any(re.search(r"cp\.async\.bulk\.(commit_group|wait_group)", a) for a in asm):
        copies = [a for a in asm if re.search(r"cp\.(reduce\.)?async\.bulk\.(tensor|shared|global)", a)]
        assert any(".bulk_group" in a for a in copies) and all(".bulk_group" in a or ".global" in a for a in copies)


@pytest.mark.parametrize("name", SOURCES)
def test_no_relaxed_arrivals(name):
    """An arrival tells another thread that reads or writes are done: it releases them."""
    assert not [a for a in asm_strings(name) if re.search(r"mbarrier\.arrive[a-z_.]*\.relaxed", a)]


@pytest.mark.parametrize("name", SOURCES)
def test_arrivals_in_another_cta_release_at_cluster_scope(name):
    """Scope says which threads synchronise, not where the data lies: an arrival that another CTA's threads act on releases
    at cluster scope (so do the counts of asynchronous copies and stores), whatever it announces."""
    remote = [a for a in asm_strings(name) if re.search(r"mbarrier\.arrive[a-z_.:]*shared::cluster", a)]
    assert all(".release.cluster" in a for a in remote)
