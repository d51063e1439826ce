"""Sampling: outputs in the place of an input, where the call takes that."""
import pytest
import torch

from _util import status_ok
from test_gpu_paged import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sdv():
    from speculative_decoding_verify_gb300 import build as b
    b.build()
    import speculative_decoding_verify_gb300 as m
    m.lib()
    return m


@pytest.mark.parametrize("N", [1, 7, 400])
def test_probabilities_in_the_random_numbers_place(sdv, N):
    """The same tokens and probabilities whether prob is a buffer of its own, u or min_p (400 rows are more than run at a time, and are put
    in order first)."""
    torch.manual_seed(N)
    V = 5000
    l, u = torch.randn(N, V, device="cuda") * 3, torch.rand(N, device="cuda") * 0.999
    T, p, low = torch.rand(N, device="cuda") + 0.5, torch.rand(N, device="cuda") * 0.5 + 0.5, torch.rand(N, device="cuda") * 0.1
    k = i32([(7 * i) % 300 for i in range(N)])
    own, token = torch.zeros(N, device="cuda"), i32([0] * N)
    sdv.sample(l, u, token, temperature=T, top_k=k, top_p=p, min_p=low, prob=own)
    for place in (u, low):
        was, again = place.clone(), i32([0] * N)
        sdv.sample(l, u, again, temperature=T, top_k=k, top_p=p, min_p=low, prob=place)
        status_ok()
        assert torch.equal(again, token) and torch.equal(place, own)
        place.copy_(was)


def test_the_smallest_temperatures(sdv):
    """Temperatures above 0 and below 1.4e-36 count as that: logits of their size are weighed alike, others give the likeliest token."""
    torch.manual_seed(3)
    N, V = 6, 700
    u, T = torch.rand(N, device="cuda") * 0.999, torch.tensor([1.4e-36, 1e-36, 1e-38, 1e-40, 1e-44, 1e-45], device="cuda")
    token, prob = i32([0] * N), torch.zeros(N, device="cuda")
    near = (torch.randn(1, V, device="cuda") * 1e-36).expand(N, V).contiguous()
    u[:] = u[0]
    sdv.sample(near, u, token, temperature=T, prob=prob)
    status_ok()
    assert torch.all(token == token[0]) and torch.all(prob == prob[0])
    w = torch.softmax(near[0].double() / (1.4426950408889634e-36), 0)
    assert abs(float(prob[0]) - float(w[int(token[0])])) <= 1e-5 * float(prob[0])
    far = torch.randn(N, V, device="cuda")
    sdv.sample(far, u, token, temperature=T, prob=prob)
    status_ok()
    assert torch.equal(token.long(), far.argmax(1)) and torch.all(prob == 1.0)
