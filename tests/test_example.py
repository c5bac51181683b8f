"""The example runs lora_linear, lora_cross_entropy and their backward passes as a
training step uses them."""
import importlib.util
import os

import pytest

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "adapter_step.py")


@pytest.mark.gpu
def test_adapters_learn():
    spec = importlib.util.spec_from_file_location("adapter_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    losses = module.train(steps=12)
    assert all(later < earlier for earlier, later in zip(losses, losses[1:])), losses
