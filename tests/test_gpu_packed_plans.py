"""Plans of as many tokens as 32 bits can count."""
import pytest
import torch

from sparse_long_context_cca_gb300 import api
from test_gpu_packed import device

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("cu", [[0, MOST], [0, 700, MOST - 3], [5, 5, 6]], ids=["one", "two", "short"])
@pytest.mark.parametrize("g", [1, 16])
def test_the_largest_number_of_tokens(cu, g):
    # positions and first tokens are counted past the last stripe of a block without leaving 32 bits
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = api.cca_pack(device(cu), MOST, g, None, dev_status=status)
    assert int(status) == 0
    lists = p.plan[:64].view(torch.int32)[8:10].cpu().sum().item()
    assert lists == sum(-(-(b - a) // n) for a, b in zip(cu, cu[1:]) for n in (256, 128))
    size = api.load_library().cca_pack_size(len(cu) - 1, MOST, g)
    first = p.plan[size - (4 * (MOST // g) + 15) // 16 * 16:][:4 * (MOST // g)].view(torch.int32)

    def expect(tensor, a, b, want):     # in pieces: 2^31 of anything else would not fit next to it
        for x in range(a, b, 1 << 28):
            y = min(x + (1 << 28), b)
            assert torch.equal(tensor[x:y], want(torch.arange(x, y, dtype=torch.int64, device="cuda")).to(torch.int32))
    zero, none = lambda i: 0 * i, lambda c: 0 * c - 1   # noqa: E731
    expect(p.positions, 0, cu[0], zero)
    expect(first, 0, cu[0] // g, none)
    for a, b in zip(cu, cu[1:]):
        expect(p.positions, a, b, lambda i: i - a)
        whole = a // g + (b - a) // g
        expect(first, a // g, whole, lambda c: a + (c - a // g) * g)
        expect(first, whole, b // g, none)
    expect(p.positions, cu[-1], MOST, zero)
    expect(first, cu[-1] // g, MOST // g, none)
