"""pages_resize on sequences of many pages, whose entries take every warp of a CTA."""
from __future__ import annotations

import random

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_gqa_02_gb300 import build, ops
import serving_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ops.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Books:
    def __init__(self, seqs, pages, blocks, page=16):
        self.p = ops.make_params(num_seqs=seqs, num_q_heads=1, num_kv_heads=1, head_dim=64, page_size=page, num_pages=pages,
                                 max_blocks_per_seq=blocks, max_context_len=blocks * page, dtype="bf16")
        self.ref = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.tables = torch.full((seqs, blocks), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.pairs = torch.zeros(seqs, 2, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = torch.empty(ops.pages_workspace_size(self.p), dtype=torch.uint8, device="cuda")

    def resize(self, new):
        self.status.zero_()
        ops.pages_resize(self.p, self.ref, self.tables, self.lens, i32(new), self.pairs, self.ws, dev_status=self.status)
        return int(self.status.item())

    def model(self):
        return ref.PageModel(self.ref.tolist(), self.tables.tolist(), self.lens.tolist(), self.p.page_size)


def test_long_sequences_freed_and_shrunk_release_every_page():
    seqs, blocks = 60, 900
    b = Books(seqs, seqs * blocks, blocks)
    rng = random.Random(3)
    for _ in range(8):
        lens = [rng.randint(300, blocks) * 16 - rng.randint(0, 15) for _ in range(seqs)]
        for new in (lens, [rng.choice([-1, 0, rng.randint(0, n), n]) for n in lens], [0] * seqs):
            m = b.model()
            want, _ = m.resize(new)
            assert b.resize(new) == 0
            assert b.ref.tolist() == m.ref and b.lens.tolist() == m.lens and b.pairs.tolist() == want
            assert b.tables.tolist() == m.tables
        assert int(b.ref.abs().sum()) == 0 and (b.tables == -1).all()


@pytest.mark.parametrize("last", (1, 5999))
def test_an_entry_that_names_a_free_page_takes_no_hold_from_its_new_owner(last):
    """Sequence 0 is handed page 0 while the last one gives back an entry that names it without a hold:
    whichever comes first, the page is sequence 0's and the entry is flagged."""
    b = Books(last + 1, 40, 3)
    b.tables[last, 0], b.tables[last, 1] = 0, 7
    b.lens[last], b.ref[7] = 32, 1
    for _ in range(3):
        tables, lens, counts = b.tables.clone(), b.lens.clone(), b.ref.clone()
        assert b.resize([20] + [-1] * (last - 1) + [0]) == ops.PA_DEV_BAD_PAGE
        assert b.ref.tolist() == [1, 1] + [0] * 38
        assert b.tables[0].tolist() == [0, 1, -1] and (b.tables[last] == -1).all()
        b.tables.copy_(tables), b.lens.copy_(lens), b.ref.copy_(counts)


def test_more_sharers_than_a_page_counts_leave_no_negative_count():
    """Three entries name a page of refcount 2: each sequence that grows gets its own page, the third hold is flagged."""
    b = Books(3, 10, 2)
    b.tables[:, 0], b.lens[:] = 4, 5
    b.ref[4] = 2
    assert b.resize([6, 7, 8]) == ops.PA_DEV_BAD_PAGE
    assert b.ref.tolist() == [1, 1, 1] + [0] * 7
    assert b.pairs.tolist() == [[4, 0], [4, 1], [4, 2]] and b.tables[:, 0].tolist() == [0, 1, 2]
