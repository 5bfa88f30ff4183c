"""Refusals of the step's calls, on the host before any CUDA call (no GPU needed)."""
import ctypes as C
import os
import shutil
import subprocess

import pytest

from test_serve_abi import BAD_SEQS, ROOT, _Seqs, kvrp  # noqa: F401


class _Prefix:
    def __init__(self, kvrp, **over):  # noqa: F811
        f = dict(block_table=0x4000, length=0x5000, n_pages=4)
        f.update(over)
        self.c = kvrp._abi.kvrp_prefix(*[f[n] for n, _ in kvrp._abi.kvrp_prefix._fields_])
        self.ref = C.byref(self.c)


BAD_PREFIX = [(dict(block_table=None), "INVALID_ARG"), (dict(length=None), "INVALID_ARG"), (dict(n_pages=-1), "INVALID_ARG"),
              (dict(n_pages=1 << 28), "INVALID_ARG"), (dict(block_table=0x4002), "ALIGNMENT"), (dict(length=0x5001), "ALIGNMENT")]


def test_step_tables_refusals(kvrp):  # noqa: F811
    inv, ali, uns = kvrp.KVRP_ERR_INVALID_ARG, kvrp.KVRP_ERR_ALIGNMENT, kvrp.KVRP_ERR_UNSUPPORTED

    def st(seqs=None, **over):
        args = dict(kept_lens=0x10000, new_rows=0x11000, held_pages=0x12000, free_pages=0x13000, free_state=0x14000,
                    positions=0x15000, slots=0x16000, stream=0)
        args.update(over)
        kept, new = args.pop("kept_lens"), args.pop("new_rows")
        with pytest.raises(kvrp.KvrpError) as e:
            kvrp.kv_step_tables(kept, new, seqs or _Seqs(kvrp), **args)
        assert kvrp.kvrp_last_launch_count() == 0
        return e.value.status

    for over, code in BAD_SEQS:
        assert st(seqs=_Seqs(kvrp, **over)) == getattr(kvrp, "KVRP_ERR_" + code), over
    for over, code in BAD_PREFIX:
        assert st(prefix=_Prefix(kvrp, **over)) == getattr(kvrp, "KVRP_ERR_" + code), over
    assert st(seqs=_Seqs(kvrp, row_start=None, n_rows=2)) == inv
    for name in ("kept_lens", "new_rows", "held_pages", "free_pages", "free_state"):
        assert st(**{name: None}) == inv and st(**{name: 0x10002}) == ali, name
    assert st(positions=0x15001) == ali and st(slots=0x16004) == ali and st(held_out=0x17003) == ali
    assert st(seqs=_Seqs(kvrp, n_seqs=65535, table_stride=1 << 16)) == uns
    import torch
    if not torch.cuda.is_available():
        assert st() == kvrp.KVRP_ERR_CUDA and st(positions=None, slots=None) == kvrp.KVRP_ERR_CUDA


def test_verify_refusals(kvrp):  # noqa: F811
    inv, ali, uns = kvrp.KVRP_ERR_INVALID_ARG, kvrp.KVRP_ERR_ALIGNMENT, kvrp.KVRP_ERR_UNSUPPORTED

    def st(seqs=None, **over):
        args = dict(target=0x10000, draft=0x20000, vocab=100, tokens=0x30000, u_accept=0x31000, u_sample=0x32000,
                    out_tokens=0x33000, accepted=0x34000, kept_lens=0x35000, stream=0)
        args.update(over)
        target = args.pop("target")
        with pytest.raises(kvrp.KvrpError) as e:
            kvrp.kv_verify_drafts(target, seqs or _Seqs(kvrp), **args)
        assert kvrp.kvrp_last_launch_count() == 0
        return e.value.status

    for over, code in BAD_SEQS:
        assert st(seqs=_Seqs(kvrp, **over)) == getattr(kvrp, "KVRP_ERR_" + code), over
    for name in ("target", "tokens", "u_accept", "u_sample", "out_tokens"):
        assert st(**{name: None}) == inv, name
    assert st(prob_type=2) == uns and st(vocab=0) == uns and st(vocab=(1 << 22) + 1) == uns
    assert st(target_stride=99) == inv and st(draft_stride=99) == inv and st(out_tokens=0x30000) == inv
    assert st(target=0x10002) == ali and st(draft=0x20001) == ali and st(target=0x10001, prob_type=kvrp.KVRP_BF16) == ali
    for name in ("tokens", "u_accept", "u_sample", "out_tokens", "accepted", "kept_lens"):
        assert st(**{name: 0x36002}) == ali, name
    import torch
    if not torch.cuda.is_available():
        assert st() == kvrp.KVRP_ERR_CUDA and st(draft=None, accepted=None, kept_lens=None) == kvrp.KVRP_ERR_CUDA


def test_attend_shared_refusals(kvrp):  # noqa: F811
    inv, ali, uns = kvrp.KVRP_ERR_INVALID_ARG, kvrp.KVRP_ERR_ALIGNMENT, kvrp.KVRP_ERR_UNSUPPORTED

    def st(seqs=None, prefix=0, **over):
        args = dict(q=0x10000, n_q_heads=8, n_kv_heads=2, head_dim=128, softmax_scale=0.1, k_pool=0x20000, v_pool=0x30000,
                    k_scale=0x40000, v_scale=0x50000, out=0x60000, lse=0x70000, workspace=0x100000, workspace_bytes=1 << 40,
                    stream=0)
        args.update(over)
        q = args.pop("q")
        with pytest.raises(kvrp.KvrpError) as e:
            kvrp.kv_attend_shared_q8(q, seqs or _Seqs(kvrp, max_rows=2), _Prefix(kvrp) if prefix == 0 else prefix, **args)
        assert kvrp.kvrp_last_launch_count() == 0
        return e.value.status

    for over, code in BAD_SEQS:
        assert st(seqs=_Seqs(kvrp, **over)) == getattr(kvrp, "KVRP_ERR_" + code), over
    for over, code in BAD_PREFIX:
        assert st(prefix=_Prefix(kvrp, **over)) == getattr(kvrp, "KVRP_ERR_" + code), over
    assert st(prefix=None) == inv
    for name in ("q", "out", "k_pool", "v_pool", "k_scale", "v_scale"):
        assert st(**{name: None}) == inv, name
    assert st(softmax_scale=0.0) == inv and st(softmax_scale=float("inf")) == inv and st(q_stride=1016) == inv
    assert st(head_dim=96) == uns and st(n_q_heads=7) == uns and st(n_q_heads=34) == uns
    assert st(q=0x10008) == ali and st(v_pool=0x30008) == ali and st(out=0x60004) == ali and st(lse=0x70002) == ali
    assert st(q_stride=1028) == ali and st(d_status=0x70001) == ali
    size = kvrp.kv_attend_shared_q8_workspace_size
    for rows in (2, 10):
        need = size(8, 2, 128, rows, 10)
        assert need > 0 and st(seqs=_Seqs(kvrp, max_rows=rows), workspace_bytes=need - 1) == kvrp.KVRP_ERR_WORKSPACE
    assert st(workspace=None) == kvrp.KVRP_ERR_WORKSPACE
    assert size(8, 3, 128, 1, 1) == 0 and size(8, 2, 96, 1, 1) == 0 and size(8, 2, 128, 0, 1) == 0 and size(8, 2, 128, 3, 2) == 0
    assert st(seqs=_Seqs(kvrp, n_rows=1 << 27, max_rows=2), workspace_bytes=1 << 50) == uns
    import torch
    if not torch.cuda.is_available():
        assert st(seqs=_Seqs(kvrp, max_rows=2), workspace_bytes=size(8, 2, 128, 2, 10)) == kvrp.KVRP_ERR_CUDA


def test_prefix_object_checks(kvrp):  # noqa: F811
    import torch
    table, length = torch.zeros(5, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    assert kvrp.Prefix(table, length).c.n_pages == 5 and kvrp.Prefix(table[:0], length).c.block_table is None
    for bad in (dict(block_table=table.long()), dict(block_table=table[::2]), dict(length=table), dict(length=length.float())):
        with pytest.raises(ValueError):
            kvrp.Prefix(**{**dict(block_table=table, length=length), **bad})


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs a host C compiler")
def test_prefix_struct_layout(kvrp, tmp_path):  # noqa: F811
    cls = kvrp._abi.kvrp_prefix
    body = "".join(f'printf("%zu ", offsetof(kvrp_prefix, {f}));' for f, _ in cls._fields_)
    src = tmp_path / "prefix.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kvrp.h"\n'
                   f'int main(void) {{ {body} printf("%zu", sizeof(kvrp_prefix)); return 0; }}\n')
    exe = tmp_path / "prefix"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [getattr(cls, f).offset for f, _ in cls._fields_] + [C.sizeof(cls)]
