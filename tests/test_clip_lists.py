"""Host side of the clipping's tensor lists (no GPU)."""
import pytest
import torch

import backward_token_expert_amd as bte
from backward_token_expert_amd import lrm


def test_a_list_in_place_may_come_from_an_iterator():
    # as `(p.grad for p in parameters)`: read once, for sources and destinations alike.  Host tensors
    # are turned down for where they are, not for a destination that is missing.
    with pytest.raises(lrm.LrmError, match="on cpu"):
        bte.make_tensor_list(t for t in [torch.zeros(4), torch.zeros(5)])
    with pytest.raises(lrm.LrmError, match="2 sources, 1 destinations"):
        bte.make_tensor_list((torch.zeros(4) for _ in range(2)), iter([torch.zeros(4)]))
