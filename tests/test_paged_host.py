"""Host-side checks of the paged cache and the packed prompts: every refusal
of the C entry points (before any launch), the binding's checks, and pins of
the oracle's e4m3 rounding and paged addressing.  No GPU needed."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import long_context_chunked_gb300 as cp
from long_context_chunked_gb300 import binding
from long_context_chunked_gb300 import build as cpbuild

A = 256  # an aligned stand-in for a device pointer: nothing is launched


@pytest.fixture(scope="module")
def lib():
    cpbuild.build()
    return cp.load()


def _pages(**kw):
    c = dict(format=1, page_size=16, num_pages=8, max_pages=4, table_stride=4, k_pages=A,
             v_pages=A, k_scales=A, v_scales=A, block_table=A)
    c.update(kw)
    return binding.Pages(*[c[n] for n, _ in binding.Pages._fields_])


def _write(ctx, pages=None, seqs=2, rows=2, lens=A, starts=A, k=A, v=A):
    p = None if pages is None else ctypes.byref(pages)
    return ctx.lib.cpattn_paged_write_kv(ctx._h, p, seqs, rows, lens, starts, k, v, None)


def _read(ctx, pages=None, seqs=2, first=None, lens=A, k=A, v=A):
    p = None if pages is None else ctypes.byref(pages)
    return ctx.lib.cpattn_paged_read_kv(ctx._h, p, seqs, first, lens, k, v, None)


def _decode(ctx, pages=None, seqs=2, lens=A, q=A, out=A, lse=None, ws=A, nbytes=1 << 30):
    p = None if pages is None else ctypes.byref(pages)
    return ctx.lib.cpattn_paged_decode(ctx._h, p, seqs, lens, q, out, lse, ws, nbytes, None)


BAD_PAGES = [
    (dict(format=2), cp.E_INVALID), (dict(format=-1), cp.E_INVALID),
    (dict(page_size=0), cp.E_UNSUPPORTED), (dict(page_size=8), cp.E_UNSUPPORTED),
    (dict(page_size=48), cp.E_UNSUPPORTED), (dict(page_size=512), cp.E_UNSUPPORTED),
    (dict(num_pages=0), cp.E_INVALID), (dict(max_pages=0), cp.E_INVALID),
    (dict(table_stride=3), cp.E_INVALID), (dict(k_pages=0), cp.E_INVALID),
    (dict(v_pages=A + 8), cp.E_INVALID), (dict(block_table=0), cp.E_INVALID),
    (dict(block_table=A + 2), cp.E_INVALID), (dict(k_scales=0), cp.E_INVALID),
    (dict(v_scales=A + 4), cp.E_INVALID), (dict(num_pages=1 << 26), cp.E_UNSUPPORTED),
    (dict(max_pages=1 << 27, table_stride=1 << 27), cp.E_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", BAD_PAGES, ids=[str(kw) for kw, _ in BAD_PAGES])
def test_bad_pages_refused_by_every_entry_point(lib, kw, status):
    ctx = cp.Context(8, 2, 128, 2, 64, 32)
    pages = _pages(**kw)
    for call in (_write, _read, _decode):
        assert call(ctx, pages) == status, call.__name__
        assert ctx.last_error()


def test_bf16_pages_need_no_scales(lib):
    ctx = cp.Context(8, 2, 128, 2, 64, 32)
    if torch.cuda.is_available():
        pytest.skip("would launch on stand-in pointers")
    for call in (_write, _read, _decode):  # past every check: no device to launch on
        assert call(ctx, _pages(format=0, k_scales=0, v_scales=0)) == cp.E_CUDA


def test_bad_arguments_refused(lib):
    ctx = cp.Context(8, 2, 128, 2, 64, 32)
    ok = _pages()
    for call in (_write, _read, _decode):
        assert call(ctx, None) == cp.E_INVALID
        assert call(ctx, ok, seqs=0) == cp.E_INVALID
        assert call(ctx, ok, seqs=cp.MAX_PAGED_SEQS + 1) == cp.E_UNSUPPORTED
        assert call(ctx, ok, lens=0) == cp.E_INVALID
        assert call(ctx, ok, lens=A + 1) == cp.E_INVALID
    for kw in (dict(rows=-1), dict(starts=None, rows=3), dict(k=0), dict(v=A + 2),
               dict(starts=A + 1)):
        assert _write(ctx, ok, **kw) == cp.E_INVALID, kw
    assert _write(ctx, ok, rows=0) == cp.OK                    # nothing to do: no launch
    for kw in (dict(k=0), dict(v=A + 2), dict(first=A + 1)):
        assert _read(ctx, ok, **kw) == cp.E_INVALID, kw
    for kw in (dict(q=0), dict(out=0), dict(q=A + 2), dict(out=A + 8), dict(lse=A + 2),
               dict(ws=0), dict(ws=A + 16), dict(nbytes=0)):
        assert _decode(ctx, ok, **kw) == cp.E_INVALID, kw
    big = cp.Context(8, 2, 128, 1 << 10, 1 << 20, 32)
    assert _read(big, ok, seqs=1) == cp.E_UNSUPPORTED           # cache rows beyond 2^31
    n = ctypes.c_uint64()
    q = ctx.lib.cpattn_paged_decode_workspace
    assert q(None, 1, ctypes.byref(n)) == cp.E_INVALID
    assert q(ctx._h, 1, None) == cp.E_INVALID
    assert q(ctx._h, 0, ctypes.byref(n)) == cp.E_INVALID
    assert q(ctx._h, cp.MAX_PAGED_SEQS + 1, ctypes.byref(n)) == cp.E_UNSUPPORTED
    assert ctx.paged_decode_workspace(cp.MAX_PAGED_SEQS) > 0


def test_null_context_refused(lib):
    p, one = ctypes.byref(_pages()), (ctypes.c_int32 * 1)(1)
    assert lib.cpattn_paged_write_kv(None, p, 1, 1, A, None, A, A, None) == cp.E_INVALID
    assert lib.cpattn_paged_read_kv(None, p, 1, None, A, A, A, None) == cp.E_INVALID
    assert lib.cpattn_paged_decode(None, p, 1, A, A, A, None, A, 1 << 30, None) == cp.E_INVALID
    assert lib.cpattn_prefill_packed(None, 1, one, A, A, A, A, None, A, 1 << 30, None) == cp.E_INVALID
    assert lib.cpattn_prefill_packed_workspace(None, 1, one, ctypes.byref(ctypes.c_uint64())) == cp.E_INVALID


def _packed(ctx, lens, q=A, k=A, v=A, out=A, lse=None, ws=A, nbytes=1 << 40):
    arr, ptr = binding._i32(lens)
    return ctx.lib.cpattn_prefill_packed(ctx._h, len(arr), ptr, q, k, v, out, lse, ws, nbytes, None)


def test_packed_refusals(lib):
    ctx = cp.Context(8, 2, 128, 2, 64, 32)
    assert _packed(ctx, []) == cp.E_INVALID
    assert _packed(ctx, [1] * (cp.MAX_SEQS + 1)) == cp.E_UNSUPPORTED
    assert _packed(ctx, [5, -1]) == cp.E_INVALID
    assert _packed(ctx, [(1 << 31) - 1, (1 << 31) - 1]) == cp.E_UNSUPPORTED
    assert _packed(ctx, [128 * (cp.MAX_ROW_BLOCKS + 1)]) == cp.E_UNSUPPORTED
    assert _packed(ctx, [0, 0]) == cp.OK                        # nothing to do: no launch
    for kw in (dict(q=0), dict(k=0), dict(v=0), dict(out=0), dict(ws=0), dict(q=A + 2),
               dict(out=A + 8), dict(lse=A + 4), dict(ws=A + 16), dict(nbytes=0)):
        assert _packed(ctx, [5, 7], **kw) == cp.E_INVALID, kw
    # longer than the context's chunk_size and its cache: neither plays a part
    if not torch.cuda.is_available():
        assert _packed(ctx, [5000]) == cp.E_CUDA
    assert ctx.prefill_packed_workspace([1, 128, 129, 0]) == (128 + 128 + 256) * 2 * 128 * 2
    with pytest.raises(cp.CpattnError):
        ctx.prefill_packed_workspace([3, -2])


def test_binding_checks_tensors():
    """Wrong types, shapes, devices and strides raise before the library is called."""
    bf, e4 = torch.bfloat16, torch.float8_e4m3fn
    kp, table = torch.zeros(4, 2, 16, 128, dtype=bf), torch.zeros(2, 3, dtype=torch.int32)
    bad = [
        dict(k=kp.float(), v=kp.float()),
        dict(k=kp[0], v=kp[0]),
        dict(v=torch.zeros(4, 2, 32, 128, dtype=bf)),
        dict(v=kp.to(e4)),
        dict(k=kp.to(e4), v=kp.to(e4)),                                 # no scales
        dict(ks=torch.zeros(4, 2, 16), vs=torch.zeros(4, 2, 16)),       # scales with bf16
        dict(k=kp.to(e4), v=kp.to(e4), ks=torch.zeros(4, 2, 8), vs=torch.zeros(4, 2, 16)),
        dict(table=table.long()),
        dict(table=table[0]),
        dict(table=torch.zeros(3, 2, dtype=torch.int32).T),
        dict(k=kp.transpose(1, 2), v=kp.transpose(1, 2)),
        {},                                                             # not on a GPU
    ]
    for kw in bad:
        with pytest.raises(ValueError):
            cp.PagedKV(kw.get("k", kp), kw.get("v", kp), kw.get("table", table), kw.get("ks"),
                       kw.get("vs"))
    with pytest.raises(ValueError):
        binding._want("q", torch.zeros(2, 3, dtype=bf), bf, (2, 3), -1)  # not on a GPU


# ------------------------------------------------------------------ oracle pins

def test_oracle_e4m3_values_are_torchs():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    ours = oracle.e4m3_values()
    assert np.array_equal(np.isnan(codes), np.isnan(ours))
    assert np.array_equal(codes[~np.isnan(codes)], ours[~np.isnan(ours)])


def test_oracle_e4m3_rounding_is_torchs():
    """Every code, every midpoint between two of them and the values beside it."""
    mags = oracle.e4m3_values()[:127]
    mid = (mags[1:] + mags[:-1]) / 2
    x = np.concatenate([mags, mid, np.nextafter(mid.astype(np.float32), np.float32(0)).astype(float),
                        np.nextafter(mid.astype(np.float32), np.float32(1e9)).astype(float)])
    x = np.concatenate([x, -x])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oracle.to_e4m3(x), want)
    assert oracle.to_e4m3(np.array([449.0, 1e30, -1e30])).tolist() == [0x7E, 0x7E, 0xFE]


@pytest.mark.parametrize("seed", range(3))
def test_oracle_quantise_error_is_half_a_step(seed):
    """|s x8 - x| <= 2^-4 |x| in the normal range, half the subnormal step
    2^-10 s below it, plus two fp32 roundings."""
    rng = np.random.default_rng(seed)
    bits = oracle.bf16_bits(torch.from_numpy(rng.standard_normal((40, 128)) *
                                             10.0 ** rng.integers(-30, 30, (40, 1))).to(torch.bfloat16))
    bits[0] = 0
    codes, s = oracle.quantise_rows(bits)
    x = oracle.bits_to_f64(bits)
    back = oracle.e4m3_values()[codes] * s[:, None].astype(np.float64)
    step = np.maximum(np.abs(x) * 2.0 ** -4, s[:, None] * 2.0 ** -10)
    assert np.all(np.abs(back - x) <= step * (1 + 2.0 ** -20))
    assert np.all(codes[0] == 0) and s[0] > 0


def test_oracle_quantise_nonfinite_rows():
    bits = np.full((3, 128), 0x3F80, np.uint16)
    bits[0, 5], bits[1, 7] = 0x7F80, 0xFFC1
    codes, s = oracle.quantise_rows(bits)
    assert np.isnan(s[:2]).all() and np.isfinite(s[2]) and np.all(codes[2] == 0x7E)


def test_oracle_paged_rows_follow_the_table():
    rng = np.random.default_rng(3)
    pool = rng.integers(0, 0x7F00, (7, 2, 16, 4)).astype(np.uint16)
    rows = oracle.paged_rows(pool, None, [5, 0, 3], 16, 14, 35)
    assert rows.shape == (21, 2, 4)
    want = oracle.bits_to_f64(pool)
    for i, t in enumerate(range(14, 35)):
        assert np.array_equal(rows[i], want[[5, 0, 3][t // 16], :, t % 16])


def test_oracle_paged_decode_is_the_softmax():
    """Against a direct sum of exponentials, one sequence empty."""
    rng = np.random.default_rng(4)
    f = lambda *s: oracle.bf16_bits(torch.from_numpy(rng.standard_normal(s)).to(torch.bfloat16))  # noqa: E731
    pools, q = [f(6, 2, 16, 8), f(6, 2, 16, 8)], oracle.bits_to_f64(f(2, 4, 8))
    table = np.array([[4, 1], [0, 2]])
    out, lse, A_, X = oracle.paged_decode_ref(q, pools, None, table, 16, [20, 0], 0.3)
    assert np.all(out[1] == 0) and np.all(lse[1] == -np.inf)
    for h in range(4):
        ws = [math.exp(0.3 * sum(q[0, h, d] * kv for d, kv in enumerate(r[h // 2])))
              for r in oracle.paged_rows(pools[0], None, table[0], 16, 0, 20)]
        v = oracle.paged_rows(pools[1], None, table[0], 16, 0, 20)[:, h // 2]
        want = sum(w * r for w, r in zip(ws, v)) / sum(ws)
        assert np.allclose(out[0, h], want, rtol=1e-12, atol=1e-13)
        assert abs(lse[0, h] - math.log(sum(ws))) < 1e-12
    assert np.all(np.abs(out) <= A_ + 1e-15) and np.all(X >= 0)
