"""Host-side checks of the serving step's later entry points: refusals before any
launch.  No GPU needed."""
import ctypes

import pytest
import torch

import long_context_chunked_gb300 as cp
from long_context_chunked_gb300 import build as cpbuild
from test_paged_host import A, _pages


@pytest.fixture(scope="module")
def lib():
    cpbuild.build()
    return cp.load()


def _write(ctx, pages, seqs=2, rows=5, have=A, lens=A, starts=A, k=A, v=A):
    p = None if pages is None else ctypes.byref(pages)
    return ctx.lib.cpattn_paged_write_planned_kv(ctx._h, p, seqs, rows, have, lens, starts, k, v, None)


def test_write_after_a_plan_refusals(lib):
    ctx, ok = cp.Context(8, 2, 128, 2, 64, 32), _pages()
    assert lib.cpattn_paged_write_planned_kv(None, ctypes.byref(ok), 1, 1, *[A] * 5, None) == cp.E_INVALID
    assert _write(ctx, None) == cp.E_INVALID
    for seqs, want in ((0, cp.E_INVALID), (cp.MAX_PAGED_SEQS + 1, cp.E_UNSUPPORTED)):
        assert _write(ctx, ok, seqs=seqs) == want
    for kw in (dict(lens=0), dict(lens=A + 2), dict(have=0), dict(have=A + 1), dict(starts=A + 2), dict(k=0), dict(v=A + 8),
               dict(rows=-1), dict(starts=0, rows=3)):
        assert _write(ctx, ok, **kw) == cp.E_INVALID, kw
        assert ctx.last_error()
    assert _write(ctx, ok, rows=0) == cp.OK               # nothing to do: no launch
    if not torch.cuda.is_available():                     # past every check: no device to launch on
        assert _write(ctx, ok) == cp.E_CUDA
        assert _write(ctx, ok, rows=2, starts=0) == cp.E_CUDA
