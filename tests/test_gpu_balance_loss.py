"""The balance loss where it is small: selections of experts with tiny scores,
a few selections among many sequences.  It has the relative accuracy of the
means and counts that it is formed from."""
import pytest
import torch

import test_gpu_balance as base
from oracle import expert_oracle as XO

pytestmark = pytest.mark.gpu
DEV = base.DEV


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def unlikely(T, E, K, seed=0):
    """Logits whose first K experts are 30 below, and a choice of those."""
    l, _ = base.make(T, E, K, seed=seed)
    l[:, :K] -= 30.0
    return l, torch.arange(K).repeat(T, 1)


@pytest.mark.parametrize("T,E,K", [(1, 8, 2), (40, 64, 4), (700, 257, 3), (300, 1024, 8), (2500, 33, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_loss_of_unlikely_experts(T, E, K, score):
    """Every token chooses the same experts of tiny scores.  `check` holds the
    loss to the relative error of its exponentials and sums."""
    l, idx = unlikely(T, E, K)
    base.check(l, idx, score, coef=1.0)
    assert 2.0**-100 < XO.balance(l.double().numpy(), idx.numpy(), score, 1.0)[0] < 2.0**-36


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_loss_of_one_selection_among_many_sequences(score):
    """700 sequences, one of which has one selection of an unlikely expert: more
    items than blocks join them."""
    T, E = 2100, 24
    l, _ = base.make(T, E, 2, spread=7.0)
    idx = torch.full((T, 2), -1)
    idx[1234, 0] = int(l[1234].argmin())
    base.check(l, idx, score, coef=1e-6, seq=list(range(0, T + 1, 3)))


def test_loss_of_empty_and_one_token_sequences_between():
    """Empty sequences at the start of, within and at the end of a chunk, and
    past the last token."""
    l, idx = unlikely(150, 40, 2)
    base.check(l, idx, "softmax", seq=[0, 0, 0, 16, 16, 17, 17, 17, 47, 48, 48, 112, 150, 150, 150])


def test_small_loss_captured_and_replayed():
    m = base.ep()
    l, idx = unlikely(900, 130, 4)
    dl, idx = l.to(DEV), idx.to(DEV)
    m.ep_balance_loss(dl, idx)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = m.ep_balance_loss(dl, idx)
    for k in range(4):
        dl.copy_(unlikely(900, 130, 4, seed=k)[0])
        want = m.ep_balance_loss(dl, idx)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and float(got[0]) > 0
