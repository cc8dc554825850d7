"""examples/serve_steps.py over either cache with samples of a prompt: what a row
computes does not depend on whose pages it shares, where they stand or who has ended."""
import os
import sys

import pytest
import torch

from activation_sparse_moe_gb300 import hs

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from activation_sparse_moe_gb300 import build
    build.build()
    hs.lib()


@pytest.mark.parametrize("bits", [4, 8])
def test_example_runs(bits):
    import serve_steps
    serve_steps.main(bits)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("prompt,sample", [(37, 37), (48, 48), (53, 32), (53, 40)])
def test_a_sample_computes_what_its_own_request_would(bits, prompt, sample):
    """A row forked off a prompt at `sample` tokens, and one that was given those
    tokens itself: the same next hidden state up to the roundings to bf16 of matrix
    products over other numbers of rows, within the 2^4 * 2^-8 = 0.06 in norm that
    tests/test_gpu_serve_example.py derives.  (A block of the 8-bit cache keeps the scale of
    tokens that a fork left behind; of 53 tokens cut at 40 the five last ones are such, and a scale
    that is a power of two larger only moves values below 2^-6 of it.)  Then the
    rows decode on, the prompt ends, pages move, and all come back."""
    import serve_steps as e
    a, b = e.Server(bits=bits), e.Server(bits=bits)
    x, other = e.hidden(prompt, 1), e.hidden(61, 2)
    a.step([prompt, 61, 0, 0], torch.cat((x, other)))
    b.step([61, 0, sample, 0], torch.cat((other, x[:sample])))
    free = a.free_pages()
    a.fork([0, 0], [2, 3], [sample, prompt])
    assert a.free_pages() == free - (sample % 16 > 0) - (prompt % 16 > 0) and a.length.tolist() == [prompt, 61, sample, prompt]
    new = e.hidden(1, 3)
    ya = a.step([0, 1, 1, 0], torch.cat((e.hidden(1, 4), new)))
    yb = b.step([1, 0, 1, 0], torch.cat((e.hidden(1, 4), new)))
    diff = (ya[-1].float() - yb[-1].float()).norm() / yb[-1].float().norm()
    assert float(diff) < 0.06, float(diff)
    for i in range(20):                     # past the end of the shared page and of the next one
        if i == 7:
            a.keep([0, 1 << 30, 1 << 30, 1 << 30])   # the prompt itself ends
            a.compact()
        rows = [0 if i >= 7 else 1, 1, 1, 1]
        y = a.step(rows, e.hidden(sum(rows), 100 + i))
        assert int(a.short) == 0 and bool(y.isfinite().all())
    assert a.length.tolist() == [0, 82, sample + 21, prompt + 20] and hs.hs_device_status() == hs.HS_OK
    a.keep([0] * 4)
    assert a.free_pages() == a.n_pages and not a.shared.any()
