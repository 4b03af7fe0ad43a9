"""The example attention layer: single-token steps through the cache agree with prompt attention over the whole sequences."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

# Of the result's norm.  Both sides round their weights and their result to the type (unit roundoff u): at most 4 u, as
# averages of values that are no larger than a few times the result.  The projection of one token may sum its products in
# another order than that of a prompt, which moves its rounded outputs by a unit here and there: 2 u more.  The codes of
# a quantised cache are off by half a step of their scale at the most, 1/254 and 1/14 of a row's largest value; rows of
# normal values have their largest near 3 times the root mean square and errors of a third of a step, evenly spread, in
# keys (through scores of about unit size) and values alike.
UNIT = {"bf16": 2.0**-8, "f16": 2.0**-11, "int8": 2.0**-8, "int4": 2.0**-8}
STEP = {"bf16": 0.0, "f16": 0.0, "int8": 3.0 / 127, "int4": 3.0 / 7}


@pytest.mark.parametrize("fmt", ["bf16", "f16", "int8", "int4"])
def test_steps_agree_with_prompts(fmt):
    import attention_layer

    got, want, _ = attention_layer.run(fmt, steps=5, seqs=4, prompt=200, hidden=512, heads=8, kv_heads=2)
    torch.cuda.synchronize()
    assert got.shape == want.shape == (4, 8, 128)
    got, want = got.double().cpu().numpy(), want.double().cpu().numpy()
    assert np.isfinite(got).all()
    off = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert off <= 6 * UNIT[fmt] + 2 * STEP[fmt] / 3
