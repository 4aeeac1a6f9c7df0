"""The example of whole layers: serving continues a prompt, gradients agree with differences."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_hybrid_layers():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import hybrid_layers
    serving, training = hybrid_layers.main(["--lengths", "130,1,65", "--more", "9"])
    # four mixers of about five bf16 roundings each (2^-9 at most, 1.7e-3 in the mean) add up to
    # sqrt(20) 1.7e-3 = 7.6e-3 on either side; twice that bounds their difference
    assert serving <= 1.5e-2
    # noise of a difference of two losses: five bf16 roundings an output on either side, 1.7e-3
    # sqrt(10) = 5.4e-3 of |out| |dout|, over a signal of 2 eps |out| |dout| about (eps 0.25 or
    # 0.5 along a unit gradient): 1.1e-2 as a standard deviation at most; twice that
    assert all(v <= 2.2e-2 for v in training.values()), training
