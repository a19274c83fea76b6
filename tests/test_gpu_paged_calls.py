"""Calls of the paged 4-bit cache and of beam search in orders that no other test makes: a process's first call at sizes of
its own, steps captured before any ran, selections whose vocabulary changes, prompts without tokens."""
import subprocess
import sys
from pathlib import Path

import pytest
import torch

from gated_deltanet_recurrence_delta_gb300 import gdn

pytestmark = pytest.mark.gpu
PAGE = 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gated_deltanet_recurrence_delta_gb300 import build
    build.build()
    gdn.load_library()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_a_first_fork_at_any_number_of_pages():
    """The fork of 60000 pages as the only one of a process: its shared memory passes the default limit."""
    code = """
import torch
from gated_deltanet_recurrence_delta_gb300 import gdn
ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
out, new, src, dst, index = ints([[-1, -1]]), ints([0]), ints([0]), ints([0]), ints([[0]])
pinned = torch.ones(60000, dtype=torch.uint8, device="cuda")
pinned[59999] = 0
gdn.cache_fork(ints([[7, -1]]), ints([64]), out, new, index, src, dst, 60000, pinned=pinned)
gdn.check_status()
assert (out.tolist(), new.tolist(), index.tolist()) == ([[7, 59999]], [65], [[59999 * 64]]), (out, new, index)
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=Path(__file__).resolve().parents[1], timeout=300)
