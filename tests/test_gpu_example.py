"""The example of a decoder layer served in 8 bits: its graph replays give the eager outputs."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "decoder_layer.py")
    spec = importlib.util.spec_from_file_location("decoder_layer_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("fmt", ["fp8", "fp8_block", "mxfp8"])
def test_graph_and_eager_steps_agree(example, fmt):
    print("example", fmt, flush=True)
    layer = example.DecoderLayer(fmt, 512, 8, 2, 64, 1024)
    runs = [example.serve(layer, 512, [70, 5, 1], 4, block_size=16, graph=g) for g in (False, True)]
    for out, steps, _ in runs:
        assert out.shape == (76, 512) and len(steps) == 4 and bool(torch.isfinite(out).all())
        assert torch.equal(out, runs[0][0])
    for a, b in zip(*(r[1] for r in runs)):
        assert a.shape == (3, 512) and torch.equal(a, b)


def test_main_prints_its_times(example, capsys):
    print("example main", flush=True)
    assert example.main(["--prompts", "40,3", "--tokens", "2", "--hidden", "256", "--heads", "4,2,64", "--ff",
                         "512"]) == 0
    assert "HIP graph" in capsys.readouterr().out
