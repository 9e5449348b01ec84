"""What the sources of the feed-forward part and the losses have to keep to, without a GPU."""
import os
import re

import pytest

import update_merged_table_gb300 as mt

CSRC = os.path.join(os.path.dirname(mt.__file__), "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", ["mt_tiles.cuh", "mt_vocab.cu", "mt_vocab_fused.cu", "mt_vocab_logits.cu", "mt_vocab_rows.cuh", "mt_vocab_sums.cu",
                                  "mt_gated.cu"])
def test_kernels_beside_their_predecessors_load_coherently(name):
    """A kernel that is resident while the one before it still writes must not read through the read-only path, which wants
    memory that nothing writes during the kernel's life."""
    text = source(name)
    assert "__ldg" not in text and "ld.global.nc" not in text
    assert "__restrict__" not in text  # with it the compiler may choose that path by itself


def test_offsets_are_loaded_coherently():
    """The gated part's kernels read them right behind the caller's kernels."""
    text = source("mt_block.cuh")
    body = text[text.index("void load_offsets("):]
    body = body[:body.index("\n}")]
    assert "offsets[i]" in body and "__ldg" not in body
