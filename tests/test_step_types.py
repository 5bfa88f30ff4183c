"""Tensors of the wrong type are refused by the step's calls before anything reaches the library (no GPU needed)."""
import pytest
import torch

from test_serve_abi import kvrp  # noqa: F401

N, ROWS, VOCAB = 3, 7, 11


def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def _seqs(kvrp):  # noqa: F811
    return kvrp.Seqs(seq_lens=_i32(N), block_tables=_i32(N, 4), num_pages=8, n_rows=ROWS, row_start=_i32(N + 1))


def _tables(kvrp, **over):  # noqa: F811
    a = dict(kept_lens=_i32(N), new_rows=_i32(N), held_pages=_i32(N), held_out=_i32(N), free_pages=_i32(8), free_state=_i32(2),
             free_state_out=_i32(2), positions=_i32(ROWS), slots=torch.zeros(ROWS, dtype=torch.int64), stream=0)
    a.update(over)
    kvrp.kv_step_tables(a.pop("kept_lens"), a.pop("new_rows"), _seqs(kvrp), **a)


def _verify(kvrp, **over):  # noqa: F811
    a = dict(target=torch.zeros(ROWS, VOCAB), draft=torch.zeros(ROWS, VOCAB), vocab=VOCAB, tokens=_i32(ROWS),
             u_accept=torch.zeros(ROWS), u_sample=torch.zeros(N), out_tokens=_i32(ROWS), accepted=_i32(N), kept_lens=_i32(N), stream=0)
    a.update(over)
    kvrp.kv_verify_drafts(a.pop("target"), _seqs(kvrp), **a)


@pytest.mark.parametrize("name", ["kept_lens", "new_rows", "held_pages", "held_out", "free_pages", "free_state", "free_state_out",
                                  "positions"])
@pytest.mark.parametrize("dtype", [torch.int64, torch.int16, torch.float32])
def test_tables_take_int32(kvrp, name, dtype):  # noqa: F811
    with pytest.raises(ValueError, match=name):
        _tables(kvrp, **{name: torch.zeros(8, dtype=dtype)})


@pytest.mark.parametrize("dtype", [torch.int32, torch.float64])
def test_tables_take_int64_slots(kvrp, dtype):  # noqa: F811
    with pytest.raises(ValueError, match="slots"):
        _tables(kvrp, slots=torch.zeros(ROWS, dtype=dtype))


@pytest.mark.parametrize("name", ["tokens", "out_tokens", "accepted", "kept_lens"])
@pytest.mark.parametrize("dtype", [torch.int64, torch.float32])
def test_verification_takes_int32(kvrp, name, dtype):  # noqa: F811
    with pytest.raises(ValueError, match=name):
        _verify(kvrp, **{name: torch.zeros(ROWS, dtype=dtype)})


@pytest.mark.parametrize("name", ["u_accept", "u_sample"])
@pytest.mark.parametrize("dtype", [torch.float64, torch.bfloat16, torch.int32])
def test_verification_takes_float32_numbers(kvrp, name, dtype):  # noqa: F811
    with pytest.raises(ValueError, match=name):
        _verify(kvrp, **{name: torch.zeros(ROWS, dtype=dtype)})


def test_verification_takes_one_type_of_probabilities(kvrp):  # noqa: F811
    wide, narrow = torch.zeros(ROWS, VOCAB), torch.zeros(ROWS, VOCAB, dtype=torch.bfloat16)
    for over in (dict(target=narrow), dict(draft=narrow), dict(target=narrow, prob_type=kvrp.KVRP_BF16),
                 dict(target=narrow, draft=narrow, prob_type=kvrp.KVRP_F32), dict(target=narrow, draft=None, prob_type=kvrp.KVRP_F32),
                 dict(target=wide, draft=None, prob_type=kvrp.KVRP_BF16), dict(target=0x10000, draft=narrow, prob_type=kvrp.KVRP_F32),
                 dict(target=wide.half(), draft=wide.half()), dict(target=wide.double(), draft=None), dict(draft=wide.half())):
        with pytest.raises(ValueError, match="target|draft"):
            _verify(kvrp, **over)


@pytest.mark.skipif(torch.cuda.is_available(), reason="host tensors: not for a call that would be launched")
def test_right_types_reach_the_library(kvrp):  # noqa: F811
    narrow = torch.zeros(ROWS, VOCAB, dtype=torch.bfloat16)
    for call, over in ((_tables, {}), (_tables, dict(held_out=None, free_state_out=None, positions=None, slots=None)),
                       (_tables, dict(free_pages=0x13000, positions=0x15000)), (_verify, {}), (_verify, dict(draft=None)),
                       (_verify, dict(target=narrow, draft=narrow)), (_verify, dict(target=narrow, draft=narrow, prob_type=kvrp.KVRP_BF16)),
                       (_verify, dict(accepted=None, kept_lens=None, tokens=0x30000))):
        with pytest.raises(kvrp.KvrpError) as e:
            call(kvrp, **over)
        assert e.value.status == kvrp.KVRP_ERR_CUDA
