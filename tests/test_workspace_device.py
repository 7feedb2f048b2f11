"""A workspace is made on a GPU only.  No GPU here."""
import pytest
import torch

import rank_markov_draft_amd as rmd


@pytest.mark.parametrize("device", ["cpu", "meta", torch.device("cpu")])
def test_workspace_off_the_gpu_is_refused(device):
    """Before its memory is handed to a kernel."""
    with pytest.raises(ValueError, match="runs on a GPU"):
        rmd.Workspace(2, 3, 64, 16, sample=True, device=device)
