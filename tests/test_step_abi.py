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
