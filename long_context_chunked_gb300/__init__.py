"""cpattn: fused chunked-prefill GQA attention on GB300 (sm_103a).

The compute path is the CUDA library ``libcpattn.so`` (C ABI, include/cpattn.h):
the striped KV-cache write and the fused cache+current prefill kernel, the
attention of packed prompts, the paged KV cache (bf16, e4m3 or e2m1) with its
write, read and decode attention, and a serving step around it: page plans, and
norms and rotations of heads that append to the pages.  This package only loads
it and marshals arguments (``binding.Context``, ``binding.PagedKV``,
``binding.NormRope``).
"""
from .binding import (E_CUDA, E_INVALID, E_NOMEM, E_PAGE, E_RANGE, E_TIMEOUT, E_UNSUPPORTED,
                      EXPORTS, LIB_PATH, MAX_PAGED_SEQS, MAX_ROW_BLOCKS, MAX_SEQS, OK, PAGE_SIZES,
                      Context, CpattnError, NormRope, PagedKV, load)

__all__ = ["Context", "CpattnError", "NormRope", "PagedKV", "load", "LIB_PATH", "EXPORTS", "OK", "E_INVALID",
           "E_UNSUPPORTED", "E_CUDA", "E_NOMEM", "E_TIMEOUT", "E_RANGE", "MAX_SEQS",
           "MAX_ROW_BLOCKS", "E_PAGE", "MAX_PAGED_SEQS", "PAGE_SIZES"]
