"""The operators around the 4-bit cache run together, as the example does."""
import importlib.util
import os

import pytest

from tests.gpu_helpers import cuda_or_skip

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_kv4.py")


@pytest.fixture(scope="module")
def example():
    cuda_or_skip()
    spec = importlib.util.spec_from_file_location("decode_kv4", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.fixture(scope="module")
def model(example):
    return example.Model(2, 512, 4, 2, 128, 5000, 512)


def _prompts(torch, n, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(0, 5000, (int(k),), generator=g).tolist() for k in torch.randint(1, 90, (n,), generator=g)]


@pytest.mark.parametrize("requests", [1, 3, 7])
def test_replays_give_the_tokens_of_separate_calls(example, model, requests):
    torch, w4 = cuda_or_skip()
    prompts = _prompts(torch, requests, requests)
    u = torch.rand(21, requests, generator=torch.Generator().manual_seed(5)).cuda()
    draw = dict(temperature=torch.full((requests,), 0.9, device="cuda"))
    a, b = (example.generate(model, prompts, 20, draw, u, graph=graph) for graph in (True, False))
    assert torch.equal(a, b)
    assert int(a.min()) >= 0 and int(a.max()) < 5000 and len(set(a[:, 0].tolist())) > 3
    assert w4.w4a16_check_device_error() == 0


def test_a_request_alone_gives_the_tokens_it_gives_in_a_batch(example, model):
    # and in two pieces as in one, up to BF16 roundings of hidden states (2^-8
    # each, a dozen in a row, independent: 5% of the logits' spread is ample,
    # and a wrong mask, page or position moves them by their whole spread)
    torch, w4 = cuda_or_skip()
    prompts = _prompts(torch, 4, 9)
    lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
    u = torch.zeros(4, device="cuda")
    s = example.Server(model, 4, 128)
    together, _ = s.step(torch.tensor(sum(prompts, []), device="cuda"), lens, max(map(len, prompts)), dict(u=u))
    for b, p in enumerate(prompts):
        one = example.Server(model, 1, 128)
        cut = len(p) // 2     # in two pieces
        for piece in (p[:cut], p[cut:]):
            if piece:
                alone, _ = one.step(torch.tensor(piece, device="cuda"),
                                    torch.tensor([len(piece)], dtype=torch.int32, device="cuda"), len(piece), dict(u=u[:1]))
        near = (alone[0].float() - together[b].float()).square().mean().sqrt()
        assert float(near) < 0.05 * float(together[b].float().std())
    assert w4.w4a16_check_device_error() == 0


def test_main(example, capsys):
    torch, _ = cuda_or_skip()
    tokens = example.main(["--layers", "1", "--requests", "2", "--steps", "3", "--hidden", "256", "--vocab", "2000"])
    assert tokens.shape == (4, 2) and "request 1" in capsys.readouterr().out
