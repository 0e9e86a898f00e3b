"""Kernels that start while the stream's last one still writes (programmatic
dependent launch) must not read through the read-only path: its loads are for
data that nothing writes while the kernel lives, and may be moved above the
wait.  No run can show that it is right, so the sources are held to the rule:
they read inputs by load_input, and only it knows the read-only path."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "wavelet_guided_sparse_gb300", "csrc")
READ_ONLY = re.compile(r"__ldg\w*\(|ld\.global\.nc|\bldg16\w*\(")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", [
    "wf_pages.cu", "wf_paged_umma.cuh", "wf_paged_kernel.cuh", "wf_attn_umma.cuh",
    "wf_paged_tree.cu", "wf_paged_window.cu", "wf_prefill.cu", "wf_attn_fma.cu"])
def test_no_read_only_loads(name):
    assert READ_ONLY.findall(source(name)) == []


def test_the_one_helper():
    text = source("wf_attn.cuh")
    assert READ_ONLY.findall(text) == ["__ldg("]
    assert "if constexpr (READ == kReadConst) return __ldg(p);" in text


def test_every_early_kernel_is_among_them():
    early = {n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh"))
             and re.search(r"launch_early\(|ProgrammaticStreamSerialization", source(n))}
    assert early <= {"wf_attn.cuh", "wf_pages.cu", "wf_paged_umma.cuh", "wf_paged_kernel.cuh",
                     "wf_prefill.cu", "wf_attn_fma.cu"}
