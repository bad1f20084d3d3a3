"""Wrong arguments of the decode-step bindings raise TypeError or ValueError, whatever they are (CPU)."""
import pytest

import speculative_decoding_draft_rmsnorm_gb300 as D


@pytest.mark.parametrize("scores", [[1.0, 2.0], None, 3.0, "flat"])
def test_beam_scores_that_are_no_table(scores):
    import torch
    x = torch.zeros(2, 3, 10)
    with pytest.raises((TypeError, ValueError)):
        D.beam_select(x, torch.zeros(6) if scores == "flat" else scores)
