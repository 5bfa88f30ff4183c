"""Refusals of the serving calls, on the host before any CUDA call (no GPU needed)."""
import ctypes as C
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def kvrp():
    from position_invariant_kv_gb300.build import build
    build()
    import position_invariant_kv_gb300 as m
    m.lib()
    return m


class _Seqs:
    """A kvrp_seqs of made-up addresses (nothing is read before the checks are through)."""

    def __init__(self, kvrp, **over):
        f = dict(row_start=0x1000, seq_lens=0x2000, block_tables=0x3000, n_seqs=2, n_rows=10, table_stride=8, num_pages=16,
                 max_rows=0)
        f.update(over)
        self.c = kvrp._abi.kvrp_seqs(*[f[n] for n, _ in kvrp._abi.kvrp_seqs._fields_])
        self.ref = C.byref(self.c)


BAD_SEQS = [
    (dict(seq_lens=None), "INVALID_ARG"), (dict(block_tables=None), "INVALID_ARG"), (dict(n_seqs=0), "INVALID_ARG"),
    (dict(n_seqs=65536), "INVALID_ARG"), (dict(n_rows=-1), "INVALID_ARG"), (dict(max_rows=11), "INVALID_ARG"),
    (dict(row_start=None), "INVALID_ARG"), (dict(table_stride=0), "INVALID_ARG"), (dict(num_pages=0), "INVALID_ARG"),
    (dict(num_pages=1 << 28), "INVALID_ARG"), (dict(seq_lens=0x2002), "ALIGNMENT"), (dict(row_start=0x1001), "ALIGNMENT"),
    (dict(block_tables=0x3002), "ALIGNMENT"),
]


def _append(kvrp, q8, seqs=None, **over):
    args = dict(q=0x10000, k=0x20000, v=0x30000, n_q_heads=8, n_kv_heads=2, head_dim=128, rope_theta=1e4, q_out=0x40000,
                k_pool=0x50000, v_pool=0x60000, q_norm=0x70000, k_norm=0x70100, stream=0)
    if q8:
        args.update(k_scale=0x80000, v_scale=0x90000)
    args.update(over)
    q, k, v = args.pop("q"), args.pop("k"), args.pop("v")
    with pytest.raises(kvrp.KvrpError) as e:
        (kvrp.kv_append_q8 if q8 else kvrp.kv_append)(q, k, v, seqs or _Seqs(kvrp), **args)
    assert kvrp.kvrp_last_launch_count() == 0
    return e.value.status


@pytest.mark.parametrize("q8", [False, True])
def test_append_refusals(kvrp, q8):
    inv, ali, uns = kvrp.KVRP_ERR_INVALID_ARG, kvrp.KVRP_ERR_ALIGNMENT, kvrp.KVRP_ERR_UNSUPPORTED
    st = lambda **o: _append(kvrp, q8, **o)  # noqa: E731
    for over, code in BAD_SEQS:
        assert st(seqs=_Seqs(kvrp, **over)) == getattr(kvrp, "KVRP_ERR_" + code), over
    assert st(k=None) == inv and st(v_pool=None) == inv
    assert st(q=None) == inv and st(q_out=None) == inv              # q and q_out go together
    assert st(q_norm=None) == inv                                    # and so do the two norms
    assert st(norm_eps=-1.0) == inv and st(norm_eps=float("nan")) == inv
    assert st(rope_theta=0.0) == inv and st(rope_theta=float("inf")) == inv
    assert st(mrope_section=(16, 24, 23)) == inv and st(mrope_section=(-1, 33, 32)) == inv
    assert st(head_dim=96) == uns and st(n_q_heads=7) == uns and st(n_q_heads=34) == uns and st(n_kv_heads=0) == uns
    assert st(q_stride=1016) == inv and st(k_stride=255) == inv     # shorter than the row
    assert st(v_stride=260) == ali and st(k=0x20008) == ali and st(q_out=0x40004) == ali and st(k_norm=0x70102) == ali
    assert st(positions=0x1002) == ali
    assert st(q_out=0x10000, q_stride=2048) == inv                   # in place needs dense rows
    if q8:
        assert st(k_scale=None) == inv and st(v_scale=0x90002) == ali
    import torch
    if not torch.cuda.is_available():                                # well-formed: no GPU, no fallback
        assert st() == kvrp.KVRP_ERR_CUDA
        assert st(q=None, q_out=None, q_norm=None, k_norm=None, mrope_section=(16, 24, 24)) == kvrp.KVRP_ERR_CUDA


def test_no_rows_is_no_work(kvrp):
    kvrp.kv_append(0x10000, 0x20000, 0x30000, _Seqs(kvrp, n_rows=0), n_q_heads=8, n_kv_heads=2, head_dim=128, rope_theta=1e4,
                   q_out=0x40000, k_pool=0x50000, v_pool=0x60000, stream=0)
    assert kvrp.kvrp_last_launch_count() == 0


def test_pack_refusals(kvrp):
    inv, ali, uns = kvrp.KVRP_ERR_INVALID_ARG, kvrp.KVRP_ERR_ALIGNMENT, kvrp.KVRP_ERR_UNSUPPORTED

    def st(**over):
        args = dict(k=0x10000, v=0x20000, n_layers=2, n_tokens=100, n_kv_heads=2, head_dim=64, k_pool=0x30000, v_pool=0x40000,
                    k_scale=0x50000, v_scale=0x60000, num_pages=16, block_table=0x70000, src_table=0x80000, src_pages=7, stream=0)
        args.update(over)
        k, v = args.pop("k"), args.pop("v")
        with pytest.raises(kvrp.KvrpError) as e:
            kvrp.kv_pack_q8(k, v, **args)
        return e.value.status

    assert st(k=None) == inv and st(v_pool=None) == inv and st(k_scale=None) == inv
    assert st(n_layers=0) == inv and st(n_tokens=-1) == inv and st(num_pages=0) == inv and st(src_pages=0) == inv
    assert st(block_table=None, num_pages=6) == inv                  # 7 pages do not fit
    assert st(num_pages=1 << 28) == inv and st(src_pages=1 << 28) == inv
    assert st(head_dim=32) == uns and st(n_kv_heads=0) == uns
    assert st(pool_layer_stride=16) == inv and st(scale_layer_stride=31) == inv and st(src_layer_stride=8) == inv
    assert st(src_layer_stride=7 * 16 * 128 + 4) == ali and st(pool_layer_stride=16 * 16 * 128 + 8) == ali
    assert st(k=0x10008) == ali and st(v_pool=0x40001) == ali and st(block_table=0x70002) == ali and st(v_scale=0x60001) == ali
    import torch
    if not torch.cuda.is_available():
        assert st() == kvrp.KVRP_ERR_CUDA


def test_attend_q8_refusals(kvrp):
    inv, ali, uns = kvrp.KVRP_ERR_INVALID_ARG, kvrp.KVRP_ERR_ALIGNMENT, kvrp.KVRP_ERR_UNSUPPORTED

    def st(seqs=None, **over):
        args = dict(q=0x10000, n_q_heads=8, n_kv_heads=2, head_dim=128, softmax_scale=0.1, k_pool=0x20000, v_pool=0x30000,
                    k_scale=0x40000, v_scale=0x50000, out=0x60000, lse=0x70000, workspace=0x100000, workspace_bytes=1 << 40,
                    stream=0)
        args.update(over)
        q = args.pop("q")
        with pytest.raises(kvrp.KvrpError) as e:
            kvrp.kv_attend_q8(q, seqs or _Seqs(kvrp, max_rows=2), **args)
        assert kvrp.kvrp_last_launch_count() == 0
        return e.value.status

    for over, code in BAD_SEQS:
        assert st(seqs=_Seqs(kvrp, **over)) == getattr(kvrp, "KVRP_ERR_" + code), over
    assert st(q=None) == inv and st(out=None) == inv and st(k_scale=None) == inv and st(v_pool=None) == inv
    assert st(softmax_scale=0.0) == inv and st(softmax_scale=-1.0) == inv and st(softmax_scale=float("nan")) == inv
    assert st(head_dim=256) == uns and st(n_q_heads=7) == uns and st(n_q_heads=34) == uns
    assert st(q_stride=1016) == inv and st(q_stride=1028) == ali
    assert st(q=0x10008) == ali and st(k_pool=0x20008) == ali and st(out=0x60004) == ali and st(lse=0x70002) == ali
    assert st(v_scale=0x50001) == ali
    assert st(workspace=None) == kvrp.KVRP_ERR_WORKSPACE and st(workspace_bytes=1024) == kvrp.KVRP_ERR_WORKSPACE
    assert kvrp.kv_attend_q8_workspace_size(8, 3, 128, 1) == 0 and kvrp.kv_attend_q8_workspace_size(8, 2, 96, 1) == 0
    assert kvrp.kv_attend_q8_workspace_size(8, 2, 128, 0) == 0
    assert st(seqs=_Seqs(kvrp, n_rows=1 << 27, max_rows=2)) == uns                # n_rows x group reaches 2^28
    need = kvrp.kv_attend_q8_workspace_size(8, 2, 128, 2)
    assert need > 0
    import torch
    if not torch.cuda.is_available():
        assert st(workspace_bytes=need) == kvrp.KVRP_ERR_CUDA


def test_seqs_object_checks(kvrp):
    import torch
    lens, table = torch.zeros(3, dtype=torch.int32), torch.zeros((3, 4), dtype=torch.int32)
    s = kvrp.Seqs(seq_lens=lens, block_tables=table, num_pages=9)
    assert (s.c.n_seqs, s.c.n_rows, s.c.table_stride, s.c.num_pages, s.c.row_start) == (3, 3, 4, 9, None)
    for bad in (dict(seq_lens=lens.long()), dict(seq_lens=lens[:2]), dict(block_tables=table[:, :2]),
                dict(row_start=lens), dict(row_start=torch.zeros(4, dtype=torch.int32)), dict(seq_lens=lens.float())):
        with pytest.raises(ValueError):
            kvrp.Seqs(**{**dict(seq_lens=lens, block_tables=table, num_pages=9), **bad})


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs a host C compiler")
def test_seqs_struct_layout(kvrp, tmp_path):
    cls = kvrp._abi.kvrp_seqs
    body = "".join(f'printf("%zu ", offsetof(kvrp_seqs, {f}));' for f, _ in cls._fields_)
    src = tmp_path / "seqs.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kvrp.h"\n'
                   f'int main(void) {{ {body} printf("%zu", sizeof(kvrp_seqs)); return 0; }}\n')
    exe = tmp_path / "seqs"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [getattr(cls, f).offset for f, _ in cls._fields_] + [C.sizeof(cls)]
