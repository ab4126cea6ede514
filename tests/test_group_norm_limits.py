"""What the group norm's entry points refuse by size, the function refuses by name
(ValueError) before any device work; CPU."""
import pytest
import torch

import recurrent_networks_gb300 as rn
from recurrent_networks_gb300 import _lib


class OnGpu(torch.Tensor):
    """A stand-in for a tensor on the GPU."""
    is_cuda = True


def test_groups_and_channels():
    size = _lib.rnn_group_norm_workspace_size
    most, width = _lib.NORM_MAX_GROUPS, _lib.NORM_MAX_CHANNELS // 32768
    assert size(1, most, 8, torch.bfloat16) > 0 and size(1, most + 1, 8, torch.bfloat16) == 0
    assert size(1, 32768, width, torch.bfloat16) > 0 and size(1, 32768, width + 1, torch.bfloat16) == 0
    for groups, channels in ((most + 1, 8 * (most + 1)), (32768, 32768 * (width + 1))):
        x = torch.zeros(1, 1).expand(2, channels).as_subclass(OnGpu)
        with pytest.raises(ValueError, match="groups"):
            rn.group_norm(x, groups)
