"""The hybrid example (GDN layers and 4-bit KV attention in one stack) end to
end: a prompt's rows equal the same tokens decoded one by one, a fork continues
as its parent would, freed and compacted pages change nothing."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture()
def stack():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import hybrid_stack
    return hybrid_stack


def rel(a, b):
    a, b = a.double(), b.double()
    return ((a - b).norm() / b.norm()).item()


def test_prompt_equals_decode(stack):
    """Decoding a prompt's tokens one by one goes through other kernels and other
    roundings (BF16 rows, FP32 sums in other orders, NVFP4 codes that can move by
    a step where a value lies on a border): the rows agree to a few percent."""
    net = stack.HybridStack()
    x = torch.randn(40, net.shape.hidden, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    _, y = net.prompt([x])
    seq, first = net.prompt([x[:1]])
    assert rel(first[0], y[0]) <= 5e-2
    for t in range(1, 40):
        row = net.decode(seq, x[t:t + 1])
        assert rel(row[0], y[t]) <= 5e-2, t
    assert net.check() == 0


def test_fork_free_and_compact(stack):
    net = stack.HybridStack()
    gen = torch.Generator(device="cuda").manual_seed(2)
    H = net.shape.hidden
    seqs, _ = net.prompt([torch.randn(n, H, generator=gen, device="cuda").bfloat16() for n in (50, 21)])
    child = net.fork(seqs[0])
    x = torch.randn(3, H, generator=gen, device="cuda").bfloat16()
    x[2] = x[0]
    y = net.decode(seqs + [child], x)
    assert torch.equal(y[0], y[2])
    step = torch.randn(1, H, generator=gen, device="cuda").bfloat16()
    before = net.decode([seqs[0]], step)             # the parent goes on alone
    net.free(seqs.pop(0))
    assert net.cache.compact() == len(set(net.cache.book.pages(seqs[0]) + net.cache.book.pages(child)))
    assert torch.equal(net.decode([child], step), before)
    assert net.check() == 0


def test_main(stack, capsys):
    stack.main()
    assert "equals its parent's: True" in capsys.readouterr().out
