"""CPU checks around the gated delta rule's calls that need no GPU: what the binding copies, and how the
kernels map packed offsets to rows."""
import os
import subprocess

import pytest
import torch

import gated_delta_rule_31_amd as kda
from gated_delta_rule_31_amd.build import HIPCC
from gated_delta_rule_31_amd.gdr import _input
from tests.test_gdr import _bwd, _fwd


@pytest.mark.parametrize("first", range(1, 8))
def test_only_wide_loads_need_a_border_of_16(first):
    """A tensor on the border that its reader needs is taken as it is, any other copied to one."""
    base = torch.arange(16, dtype=torch.float32)
    assert base.data_ptr() % 16 == 0
    x = base[first : first + 5]
    assert _input(x, "x", base, torch.float32, 4).data_ptr() == x.data_ptr()
    wide = _input(x, "x", base, torch.float32)
    assert wide.data_ptr() % 16 == 0 and torch.equal(wide, x) and (wide.data_ptr() == x.data_ptr()) == (first % 4 == 0)


def test_packed_offsets_stay_in_range(tmp_path):
    """The device's own mapping of offsets to rows and chunk slots, compiled for the host: in range for any offsets,
    one slot a chunk and one chunk a token for offsets in order."""
    exe = str(tmp_path / "rows")
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run([HIPCC, "--offload-host-only", "-O1", "-std=c++17", os.path.join(here, "gdr_rows_check.hip"), "-o", exe], check=True,
                   capture_output=True, timeout=300)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


@pytest.mark.parametrize("B,T", [(1 << 10, 1 << 60), (1 << 10, (1 << 60) + 64), (1 << 12, (1 << 57) + 1), (2, (1 << 63) - 1), (1, (1 << 28) + 1)])
def test_counts_of_chunks_do_not_wrap(B, T):
    """Rows whose chunks would pass 64 bits are refused, and have no workspace size, as any that are too long."""
    lib = kda._load()
    assert _fwd(lib, B=B, T=T, HK=1, HV=1) == 4 and _bwd(lib, B=B, T=T, HK=1, HV=1) == 4
    assert kda.gdr_chunk_fwd_workspace_size(torch.bfloat16, B, T, 1, 1, 16, 16) == 0
    assert kda.gdr_chunk_bwd_workspace_size(torch.bfloat16, B, T, 1, 1, 16, 16) == 0
