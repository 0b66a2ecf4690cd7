"""More of the calls over a paged latent cache: workspaces on other streams."""
import pytest
import torch

import _paged as P
from sparse_attention_kv_echo_gb300 import _lib as L

pytestmark = pytest.mark.gpu
dev = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    L.load(build_if_missing=True)


def _weigh(bt, lse, mass, stream=None, ws=None):
    row_off, q, tok_off, tok_end, pages = bt.on(dev, L)
    out = torch.zeros_like(mass)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    torch.cuda.synchronize()

    def call():
        L.mla_mass(row_off, q, lse, tok_off, bt.n_tokens, pages, bt.scale, mass, out, st, decay=0.5, tok_end=tok_end,
                   stream=stream, ws=ws)
    return call, out, st


def test_weights_on_another_stream_take_a_workspace_of_that_stream():
    # a block of the workspace's size is freed on the current stream while the kernel that fills it is still pending
    # there: the call on the other stream does not get it
    bt = P.Batch([900, 300], [1, 40], 128, 64, seed=3)
    lse = bt.attend()[1].float().to(dev)
    mass = torch.rand(bt.n_tokens, device=dev)
    size = L.mla_mass_workspace_size(bt.n_tokens, 2)
    call, want, st = _weigh(bt, lse, mass, ws=torch.zeros(size, dtype=torch.uint8, device=dev))
    call()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    call, got, st2 = _weigh(bt, lse, mass, stream=other)
    for cycles in (0, 20_000, 100_000):
        block = torch.empty(size, dtype=torch.uint8, device=dev)
        torch.cuda._sleep(cycles)
        block.zero_()
        del block
        call()
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and int(st2.item()) == 0
        assert torch.equal(got, want)
