"""The serving example: steps over the 4-bit cache and the MoE layers together."""
import os
import sys

import pytest
import torch

from activation_sparse_moe_gb300 import hs

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def serve():
    from activation_sparse_moe_gb300 import build
    build.build()
    import serve_steps
    return serve_steps


def test_example_runs_and_gives_its_pages_back(serve):
    s = serve.Server()
    all_pages = s.free_pages()
    s.step([37, 5, 130, 0], serve.hidden(172, 0))
    assert s.length.tolist() == [37, 5, 130, 0] and s.free_pages() == all_pages - 3 - 1 - 9
    s.step([1, -1, 20, 60], serve.hidden(81, 1))
    assert s.length.tolist() == [38, 0, 150, 60] and s.free_pages() == all_pages - 3 - 10 - 4
    serve.main()


def test_prompt_in_one_chunk_equals_token_by_token(serve):
    """A chunk of 60 tokens (240 query rows a kv head: the tensor-core kernel; the
    MoE layer's batch kernels) and the same tokens one by one (the few-row
    kernel, batch-1 MoE) leave the same hidden state of the last token, up to the
    roundings to bf16 between the layers.  Each of the two layers adds two bf16
    roundings to a state of about unit size in the attention branch and two in the
    MoE branch (2^-8 of a value at most, in the mean over channels 2^-8 / sqrt(3)),
    and each branch passes the differences of the ones before on with about unit
    gain: 4 branches, doubled by each branch at worst, 2^4 * 2^-8 = 0.06 in norm.  A
    routed expert chosen differently at a near tie would show as a difference of
    order 1."""
    x = serve.hidden(60, 5)
    a, b = serve.Server(), serve.Server()
    chunk = a.step([60, 0, 0, 0], x)[-1].float()
    for i in range(60):
        last = b.step([1, 0, 0, 0], x[i:i + 1])
    torch.cuda.synchronize()
    assert hs.hs_device_status() == hs.HS_OK
    diff = (chunk - last[0].float()).norm() / chunk.norm()
    assert float(diff) < 0.06, float(diff)
