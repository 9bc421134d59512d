"""bf16 queries over codes in the calls whose operands never carry scales (few new
tokens, heads above 128 dims): the bounds without that rounding hold."""

import pytest

import test_gpu_attention as attention

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def nothing_folded(monkeypatch):
    monkeypatch.setattr(attention, "FOLDED", None)


@pytest.mark.parametrize("length", [1, 15, 64, 129, 300, 5000])
@pytest.mark.parametrize("new", [1, 5, 32])
@pytest.mark.parametrize("d", [40, 64, 128])
def test_few_new_tokens(q4lib, length, new, d):
    attention.run(q4lib, "bf16", "i8", 4, 2, d, 16, [length + new, new], [new, min(new, 3)])


@pytest.mark.parametrize("window", [1, 100])
@pytest.mark.parametrize("new", [1, 16])
def test_windows(q4lib, window, new):
    attention.run(q4lib, "bf16", "i8", 8, 2, 128, 64, [new + 130, 900], [new, new], window=window)


@pytest.mark.parametrize("d", [136, 192, 256])
@pytest.mark.parametrize("new", [1, 40, 200])
def test_large_heads(q4lib, d, new):
    attention.run(q4lib, "bf16", "i8", 4, 2, d, 32, [new + 300, 90 + new], [new, new])


@pytest.mark.parametrize("sharp", [1e-3, 8.0])
def test_flat_and_sharp(q4lib, sharp):
    attention.run(q4lib, "bf16", "i8", 4, 1, 128, 16, [700, 20], [5, 5], sharp=sharp)
