"""GPU: gradients of rows whose logits are large as a whole, in every type, with the
bounds of test_gpu_token_loss.py: the softmax depends on differences alone."""

import numpy as np
import pytest
import torch

from test_gpu_token_loss import Batch, check_policy, check_preference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,offset", [(torch.float32, 4000.0), (torch.float16, 4096.0), (torch.float16, 60000.0),
                                          (torch.bfloat16, 4096.0), (torch.bfloat16, 2.0 ** 20)])
@pytest.mark.parametrize("vocab", [300, 50_257])
def test_gradients_of_large_logits(vocab, dtype, offset):
    for sign in (1.0, -1.0):
        def edit(z, y, w, rng):
            z += sign * offset
            z[0] = sign * offset                # every token alike
            z[1, ::2] = sign * offset
            z[1, 1::2] = sign * offset - 32.0
        b = Batch(4, vocab, dtype, masked=0.0, edit=edit)
        for temperature in (1.0, 0.7, 3.0):
            check_policy(b, temperature=float(np.float32(temperature)))
        check_preference(b, np.array([0, 2, 4], np.int32))
