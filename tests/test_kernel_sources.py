"""Rules of the kernels that no run can show without letting a wait run out on the GPU: their source is read instead (CPU)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "chunked_gated_delta_05_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


@pytest.mark.parametrize("name,roles", [("k_attn_fwd.cu", 2), ("k_attn_bwd.cu", 4)])
def test_warps_that_use_tensor_memory_vote_on_their_waits(name, roles):
    """Reads and writes of tensor memory, and the products, are instructions of a whole warp: its lanes come to them together, and where a wait
    ran out for one of them none goes on. So these roles wait by functions in which all lanes vote."""
    seen = 0
    for section in source(name).split("// ---------------- ")[1:]:
        if not re.search(r"\b(tmem_(ld|st)\w*|product_\w+)[<(]", section):
            continue
        seen += 1
        section = re.sub(r"__all_sync\(0xffffffffu, wait\(", "", section.split("\ntemplate <int D>")[0])
        alone = re.findall(r"^.*(?<!\w)(?:wait|attn_wait|mbar_wait|get)\(.*$", section, re.M)
        assert not alone, alone
    assert seen == roles


def test_step_warps_vote_on_their_waits():
    lines = [x for x in source("k_attn_step.cu").splitlines() if re.search(r"\b(attn|mbar)_wait\(", x)]
    assert lines and all("__all_sync(0xffffffffu, attn_wait(" in x for x in lines), lines


def test_the_join_trusts_no_piece_that_was_not_written():
    """A step whose wait ran out leaves its rows' places in the workspace as they were. The join's addresses come from those, so it holds them
    against the number of shares first."""
    join = source("k_attn_step.cu").split("k_attn_join(", 1)[1].split("template <int D, int kRows>", 1)[0]
    read, first = join.index("p.span["), join.index("p.part +")
    between = join[read:first]
    for condition in (r"span\.x < 0", r"span\.x >= span\.y", r"span\.y >= p\.shares"):
        assert re.search(condition + r".*return;", between), condition


@pytest.mark.parametrize("name", ["k_prep.cu", "k_prep_kda.cu", "k_chain.cu", "k_chain_bwd.cu", "k_bwd_feat.cu", "k_bwd_tok.cu", "k_bwd_tok_kda.cu"])
def test_the_recurrences_warps_vote_on_their_waits(name):
    """In these kernels a wait of whole warps is one whose result goes on to all of their threads: a named result, or a chain warp's loop. Waits of a
    single thread (issuing and copying) and those whose result is not used stay as they are."""
    voted = 0
    chain = name.startswith("k_chain")
    text = source(name)
    if chain:       # behind the single threads' branches
        text = text[text.index("} else if (warp < kChainThreads / 32) {"):]
    for line in text.splitlines():
        if "mbar_wait(" not in line or (not chain and not re.search(r"\bok\d?\b|\btma_ok\b", line)) or "tid == 0" in line:
            continue
        assert "warp_all(" in line, line
        voted += 1
    assert voted


def test_the_shared_header_lists_no_attention_kinds():
    """bench.py's traffic figures hold while a kernel's file and the shared header are those of their capture: other operators' kinds stay out of it."""
    shared = set(re.findall(r"\bkK[A-Z]\w*", source("common.cuh")))
    used = set(re.findall(r"TimedScope \w+\((kK\w+)", source("attn_api.cu")))
    assert used and not used & shared, used & shared
