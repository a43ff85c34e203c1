"""What the sources of the kernels that may start before the kernel in front of
them has ended (programmatic launches) must not say."""

import glob
import os
import re

import pytest

from greedy_speculative_decoding_gb300 import build as B

OPERATORS = sorted(os.path.basename(f) for p in ("paged_*", "chunk_*", "token_*") for f in glob.glob(os.path.join(B.CSRC, p)))


@pytest.mark.parametrize("name", OPERATORS)
def test_no_load_through_the_read_only_path(name):
    """Such loads are defined for data that nobody writes while the kernel lives,
    which begins beside the kernel that writes the operators' inputs."""
    with open(os.path.join(B.CSRC, name)) as f:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    assert not re.findall(r"__ldg\b|ld\.global\.nc|__restrict__", code)


def test_the_operators_sources_are_there():
    assert {"token_logprobs.cu", "paged_share.cu", "paged_copy.cu", "chunk_attn.cuh", "paged_attn.cuh"} <= set(OPERATORS)
