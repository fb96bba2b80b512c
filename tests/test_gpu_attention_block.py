"""The example that runs projection, rotary cache write, prompt attention and
paged attention together: the attention of the prompts' last rows comes out the
same over whole prompts and over the cache."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("attention_block", os.path.join(ROOT, "examples", "attention_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("lengths", [(700, 33, 1, 258), (64,), (5, 129, 127, 128, 64, 63, 65, 2)])
def test_prompt_and_paged_attention_agree(example, lengths):
    # the same bf16 keys and values: both round the weights and the output once (2^-8 each, of the weighted values)
    worst, most = example.run(lengths, steps=3, seed=len(lengths))
    assert worst <= 4 * 2.0 ** -8 * max(most, 1.0)


def test_8_bit_cache(example):
    # keys and values off by 2^-4 of themselves move an output of unit-size values by no more than a few of that
    worst, most = example.run((300, 77), steps=2, e4m3=True, seed=9)
    assert worst <= 8 * 2.0 ** -4 * max(most, 1.0)
