"""One status word for the calls of a step: which error the host finds in it."""
import pytest
import torch

from sparse_long_context_cca_gb300 import api

pytestmark = pytest.mark.gpu

OK, BAD, NO_PAGES, TIMEOUT = 0, api.CCA_ERR_INVALID_ARG, api.CCA_ERR_NO_PAGES, api.CCA_ERR_TIMEOUT


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Step:
    """Two sequences over a pool of n pages, and the calls of a serving step, all with one status word."""

    def __init__(self, n, dtype=torch.bfloat16, d=128):
        self.K, self.V = (torch.zeros(n, 1, 16, d, dtype=dtype, device="cuda") for _ in range(2))
        self.Kc, self.Vc = (torch.zeros(4, 1, 8, d, dtype=dtype, device="cuda") for _ in range(2))
        self.refs, self.table = i32(*[0] * n), i32(*[-1] * 8).view(2, 4)
        self.ctable, self.lens = i32(0, 1, 2, 3).view(2, 2), i32(0, 0)
        self.q, self.k = (torch.randn(2, h, 4, d, device="cuda").to(dtype) for h in (2, 1))
        self.status = i32(0)

    def reserve(self, *extra):
        return api.cca_pages_reserve(self.refs, self.table, self.lens, i32(*extra), 16, dev_status=self.status)

    def append(self):
        return api.cca_rope_append(self.q, self.k, self.k, self.K, self.V, self.table, self.lens, dev_status=self.status)

    def tree(self, lens=None):
        return api.cca_tree_fwd(self.q, self.K, self.V, self.table, self.Kc, self.Vc, self.ctable,
                                self.lens if lens is None else lens, 8, 16, dev_status=self.status)

    def pool(self):
        return api.cca_pool_pages(self.q, self.K, self.V, self.table, self.Kc, self.Vc, self.ctable, i32(6, 6), i32(4, 4), 8,
                                  dev_status=self.status)


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 64)])
def test_too_few_pages_is_not_forgotten(dtype, d):
    """The calls behind a reserve that found too few pages find none for their tokens; the word keeps what
    tells the host to make room and try again."""
    s = Step(1, dtype, d)
    s.reserve(20, 20)
    assert s.status.item() == NO_PAGES
    s.append(), s.tree(), s.pool()
    pairs = i32(0, 9).view(1, 2)
    api.cca_pages_copy(s.K, s.V, pairs, dev_status=s.status)
    api.cca_pages_free(s.refs, i32(*[0] * 8).view(2, 4), i32(0, 0), i32(4, 4), dev_status=s.status)
    api.cca_pages_fork(s.refs, s.table, i32(0), i32(0), s.lens, 16, dev_status=s.status)
    api.cca_pages_compact(s.K, s.V, s.table, s.lens, i32(1, 0, 1, 0).view(2, 2), i32(2, 2), dev_status=s.status)
    assert s.status.item() == NO_PAGES


def test_too_few_pages_counts_for_more_than_a_bad_argument():
    s = Step(1)
    s.tree(i32(-1, -1))
    assert s.status.item() == BAD
    s.reserve(20, 20)
    assert s.status.item() == NO_PAGES
    s = Step(1)
    s.reserve(1000, 20)          # in one call: a range that leaves the table, and too few pages for the other
    assert s.status.item() == NO_PAGES


def test_what_is_in_the_word_stays():
    for held in (TIMEOUT, NO_PAGES):
        for call in ("reserve", "append", "tree", "pool"):
            s = Step(1)
            s.status.fill_(held)
            getattr(s, call)(*((20, 20) if call == "reserve" else ()))
            assert s.status.item() == held, call


@pytest.mark.parametrize("heads", [2, 256], ids=["one half", "two halves"])
def test_a_time_out_counts_for_more_than_a_bad_argument(heads):
    """A bad length is reported at once, the waits run out later: the output is not complete."""
    s = Step(8)
    s.q = torch.zeros(2, heads, 4, 128, dtype=torch.bfloat16, device="cuda")[:, :heads]
    s.reserve(8, 8)
    lib = api.load_library()
    s.tree()
    assert s.status.item() == OK
    lib.cca_test_set_wait_limit_ns(2_000_000)
    lib.cca_test_skip_q_load(1)
    try:
        s.tree(i32(-1, 0))
        torch.cuda.synchronize()
    finally:
        lib.cca_test_skip_q_load(0)
        lib.cca_test_set_wait_limit_ns(1_000_000_000)
    assert s.status.item() == TIMEOUT
