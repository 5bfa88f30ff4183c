"""kv_append and kv_append_q8 on ragged batches of many sequences: what is out of range is flagged
wherever it stands, and the other sequences are appended as if it were not there."""
import numpy as np
import pytest
import torch

from serve_util import f64, i32
from test_gpu_append import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from position_invariant_kv_gb300.build import build
    build()


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("rows", [1, 2])
@pytest.mark.parametrize("bad", [3, 256, 300, 599])
def test_a_bad_length_anywhere_in_the_batch_is_flagged(q8, rows, bad):
    b = Batch(ctx=[int(5 * i % 40) for i in range(600)], rows=[rows] * 600, hq=2, hkv=1, d=64)
    lens = list(b.lens)
    lens[bad] = 16 * b.table.shape[1] + 1          # more tokens than its table has pages for
    lens[7] = 0                                    # an idle place: not an error
    seqs = b.kvrp.Seqs(seq_lens=i32(lens), block_tables=i32(b.table), num_pages=b.pages, n_rows=600 * rows, row_start=i32(b.starts))
    kind = torch.uint8 if q8 else torch.bfloat16
    pool = [torch.full((b.pages, 16, b.hkv, b.d), 7, dtype=kind, device="cuda") for _ in range(2)]
    extra = {}
    if q8:
        extra = {n: torch.full((b.pages, b.hkv), 2.0 ** -126, device="cuda") for n in ("k_scale", "v_scale")}
    call = b.kvrp.kv_append_q8 if q8 else b.kvrp.kv_append
    call(*b.inputs, seqs, k_pool=pool[0], v_pool=pool[1], **extra, **b.args)
    torch.cuda.synchronize()
    assert int(b.status) == 4
    q, stale = f64(b.q_out), (pool[1].cpu() == 7).all(-1).all(-1).numpy()
    left = [stale[page, slot] for page, slot in b.places()]
    for s in range(600):
        mine = slice(b.starts[s], b.starts[s + 1])
        assert np.isnan(q[mine]).all() == (s in (bad, 7)) and all(left[mine]) == (s in (bad, 7)), s
        if s not in (bad, 7):
            assert np.all(np.abs(q[mine] - b.q[mine]) <= 2.0 ** -8 * np.abs(b.q[mine]) + 2.0 ** -16 * b.q_mag[mine])
