"""The example over a matrix in 4 bits and with clipped gradients: it runs, and its
gradients are those that the norms say.  A clipped adapter's norm is the limit but for
the factor's 1e-6 / norm and the gradients' rounding to bfloat16, at most 2^-8 of every
value and so of the norm; one that is not clipped keeps its norm (a double, rounded
to float32 once)."""
import importlib.util
import os

import pytest
import torch

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "adapter_step.py")


@pytest.mark.gpu
@pytest.mark.parametrize("matrix", ["bf16", "mxfp4"])
def test_norms_and_gradients(matrix):
    spec = importlib.util.spec_from_file_location("adapter_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    trace = []
    losses = module.train(steps=3, matrix=matrix, trace=trace)
    assert len(losses) == len(trace) == 3 and all(torch.isfinite(torch.tensor(losses)))
    limit = float(trace[0][0].median())
    clipped = []
    module.train(steps=3, matrix=matrix, limit=limit, trace=clipped)
    assert torch.equal(clipped[0][0], trace[0][0])          # the first step's norms know no limit
    for norms, da, db in clipped:
        after = (da.double().square().sum((1, 2)) + db.double().square().sum((1, 2))).sqrt().cpu()
        norms = norms.double().cpu()
        want = torch.where(norms > limit, limit * norms / (norms + 1e-6), norms)
        assert ((after - want).abs() <= want * (2.0 ** -8 + 2.0 ** -20) + 1e-6 * limit).all()
