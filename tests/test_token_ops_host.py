"""CPU checks of the token operators' host side: what needs no GPU to be seen."""

import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ENTRIES = ("dmuon_embedding", "dmuon_embedding_grad", "dmuon_add_rmsnorm", "dmuon_add_rmsnorm_grad", "dmuon_policy_loss",
           "dmuon_token_logprobs")


def entry_body(name):
    with open(os.path.join(ROOT, "newton_schulz_momentum_gb300", "csrc", "api.cu")) as f:
        src = f.read()
    found = re.search(r"^int %s\([^{]*\{\n(.*?)^\}" % name, src, re.S | re.M)
    assert found, name
    return found.group(1)


@pytest.mark.parametrize("name", ENTRIES)
def test_entries_let_no_exception_out(name):
    """A host allocation that fails (the list of timed launches, of workspace blocks) becomes a status: an exception that
    leaves a C function ends the process."""
    body = entry_body(name).strip()
    assert body.startswith("try {") and "catch (const std::exception" in body
