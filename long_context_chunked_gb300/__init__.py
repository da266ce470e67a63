"""cpattn: fused chunked-prefill GQA attention on GB300 (sm_103a).

The compute path is the CUDA library ``libcpattn.so`` (C ABI, include/cpattn.h):
the striped KV-cache write and the fused cache+current prefill kernel, the
attention of packed prompts, and the paged KV cache with its write, read and
decode attention.  This package only loads it and marshals arguments
(``binding.Context``, ``binding.PagedKV``).
"""
from .binding import (E_CUDA, E_INVALID, E_NOMEM, E_PAGE, E_RANGE, E_TIMEOUT, E_UNSUPPORTED,
                      EXPORTS, LIB_PATH, MAX_PAGED_SEQS, MAX_ROW_BLOCKS, MAX_SEQS, OK, PAGE_SIZES,
                      Context, CpattnError, PagedKV, load)

__all__ = ["Context", "CpattnError", "PagedKV", "load", "LIB_PATH", "EXPORTS", "OK", "E_INVALID",
           "E_UNSUPPORTED", "E_CUDA", "E_NOMEM", "E_TIMEOUT", "E_RANGE", "MAX_SEQS",
           "MAX_ROW_BLOCKS", "E_PAGE", "MAX_PAGED_SEQS", "PAGE_SIZES"]
