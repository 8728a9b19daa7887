"""What the binding refuses before the library is asked, on the host."""
import pytest
import torch

from mamba_ssd_scan_02_b200 import ssd

CFG = dict(nheads=2, ngroups=1)


def tensors(rows=(1, 4)):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)
    f = torch.float32
    return dict(q=z(*rows, 128), k=z(*rows, 128), v=z(*rows, 128), dt=z(*rows, 2), b=z(*rows, 2), A=z(2, dtype=f), dt_bias=z(2, dtype=f))


@pytest.mark.parametrize("workspace", [
    torch.empty(1 << 20, dtype=torch.uint8, device="meta"),            # another device
    torch.empty(1, dtype=torch.uint8).expand(1 << 20),                 # one byte that looks like a megabyte
    torch.empty(1 << 21, dtype=torch.uint8)[::2],
], ids=["device", "expanded", "strided"])
def test_workspace(workspace):
    with pytest.raises(ValueError, match="workspace"):
        ssd.delta_prefill(CFG, **tensors(), workspace=workspace)
    with pytest.raises(ValueError, match="workspace"):
        ssd.delta_prefill_varlen(CFG, [0, 4], **tensors((4,)), workspace=workspace)


@pytest.mark.parametrize("cu", [[0, (1 << 32) + 2, 4], [1 << 32, 4], [0, (1 << 32) + 4], [0, 2 - (1 << 32), 4], [0, -1, 4]], ids=str)
def test_offsets_beyond_32_bits(cu):
    """Not taken as their low 32 bits, which here would make a valid batch."""
    with pytest.raises(ValueError, match="offsets"):
        ssd.delta_prefill_varlen(CFG, cu, **tensors((4,)))
    with pytest.raises(ValueError, match="offsets"):
        ssd.delta_varlen_workspace_size(CFG, cu)
