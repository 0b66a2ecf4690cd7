"""Wrappers name the tensor that has another number of dimensions (on the CPU: the library and the device replaced)."""
import pytest
import torch

from sparse_attention_kv_echo_gb300 import _lib as L
from test_paged_calls import host  # noqa: F401


def _zeros(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("shape", [(576,), (4, 576), (4, 2, 576, 1)])
def test_queries_of_another_rank(host, shape):  # noqa: F811
    off, st, kv = torch.tensor([0, 4]), _zeros(1), torch.zeros((16, 576), dtype=torch.bfloat16)
    pages, q = L.KVPages(_zeros(4), kv, 4), _zeros(*shape, dtype=torch.bfloat16)
    out, lse, ws = torch.zeros((4, 2, 512), dtype=torch.bfloat16), torch.zeros(4, 2), _zeros(64, dtype=torch.uint8)
    mass = torch.zeros(16)
    for call in (lambda: L.mla_chunk(off, q, torch.tensor([0, 16]), 16, pages, 0.1, out, lse, ws, st),
                 lambda: L.mla_tree(off, q, _zeros(4, 1), torch.tensor([0, 16]), 16, pages, 0.1, out, lse, ws, st),
                 lambda: L.mla_mass(off, q, lse, torch.tensor([0, 16]), 16, pages, 0.1, mass, mass.clone(), st, ws=ws)):
        with pytest.raises(ValueError, match=r"mla_\w+: q must be"):
            call()
    assert not host.calls


@pytest.mark.parametrize("shape", [(40,), (4, 10, 1)])
def test_probabilities_of_another_rank(host, shape):  # noqa: F811
    with pytest.raises(ValueError, match="draft_verify: target must be"):
        L.draft_verify(torch.tensor([0, 4]), _zeros(4), _zeros(4), torch.zeros(shape), _zeros(4), _zeros(1), _zeros(1), _zeros(1))
    assert not host.calls
