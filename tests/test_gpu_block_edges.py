"""The operators of ar_block.h where a plain binary32 computation of the same
formula is exact or the range of a type ends: ties of the 8-bit rounding, rows
and gates far from 1, and the kernels that only large calls take."""
import pytest
import torch

import all_reduce_amd as ar
import block_ref as ref
from gpu_util import note
from test_gpu_block import DT, E4M3, Planes, comm, draw  # noqa: F401  (comm is a fixture)

pytestmark = pytest.mark.gpu


# ---- quantisation --------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(2000, 1024), (1, 8192), (9000, 2056)])
def test_quantisation_is_the_quotient(comm, rows, cols, dtype):
    """Without an activation nothing is rounded before the scale: both it and the
    8-bit values are those of binary32 divisions, to the bit.  (The quotient is
    off by one bit of binary32 where it lies within 2^-46 of a tie between two of
    them: of these sizes none is expected to, and of 18 million none that is also
    next to a tie between two 8-bit values.)"""
    x = draw((rows, cols), rows + cols, DT[dtype], 3.0)
    note(f"quotient {rows}x{cols} {dtype}")
    src = Planes(1, rows, cols, DT[dtype]).fill([x])
    out, scales = Planes(1, rows, cols, E4M3), Planes(1, ref.blocks(cols), rows, torch.float32)
    comm.gate_quant(src.ranks, out.ranks, scales.ranks, act="none")
    torch.cuda.synchronize()
    assert src.untouched() and out.untouched() and scales.untouched()
    y = torch.nn.functional.pad(x.float(), (0, -cols % 128)).unflatten(1, (-1, 128))
    s = (y.abs().amax(-1) / 448).clamp_min(2.0 ** -126)
    assert torch.equal(scales.ranks[0].cpu(), s.t())
    q = (y / s.unsqueeze(-1)).flatten(1)[:, :cols].to(E4M3)
    off = out.ranks[0].cpu().float() != q.float()
    assert not off.any(), f"{int(off.sum())} of {off.numel()} values"
