"""Host-side checks of the 4-bit pages and of the serving step's entry points:
refusals before any launch, the binding's checks, the rotation's fixed-point
frequencies, and pins of the oracle.  No GPU needed."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
import long_context_chunked_gb300 as cp
from long_context_chunked_gb300 import binding
from long_context_chunked_gb300 import build as cpbuild
from oracle.step import PI
from test_paged_host import A, _decode, _pages, _read, _write

E2M1 = binding.PAGES_E2M1


@pytest.fixture(scope="module")
def lib():
    cpbuild.build()
    return cp.load()


def _ctx(hd=128):
    return cp.Context(8, 2, hd, 2, 64, 32)


def _plan(ctx, pages=None, seqs=2, rows=5, have=A, new=A, free=A, count=A, lens=A, starts=A, pos=A, slots=A):
    p = None if pages is None else ctypes.byref(pages)
    return ctx.lib.cpattn_paged_plan(ctx._h, p, seqs, rows, have, new, free, count, lens, starts, pos,
                                     slots, None)


def _trim(ctx, pages=None, seqs=2, lens=A, keep=A, free=A, count=A):
    p = None if pages is None else ctypes.byref(pages)
    return ctx.lib.cpattn_paged_trim(ctx._h, p, seqs, lens, keep, free, count, None)


def _desc(**kw):
    c = dict(q_weight=A, k_weight=A, rope_steps=A, weight_f32=0, rotary_dim=128, interleaved=0, eps=1e-6,
             rope_scale=1.0)
    c.update(kw)
    return binding.NormRopeDesc(*[c[n] for n, _ in binding.NormRopeDesc._fields_])


def _dense(ctx, desc=None, rows=3, pos=A, q=A, qs=1024, k=A, ks=256, qo=A, qos=1024, ko=A, kos=256):
    d = None if desc is None else ctypes.byref(desc)
    return ctx.lib.cpattn_norm_rope(ctx._h, d, rows, pos, q, qs, k, ks, qo, qos, ko, kos, None)


def _append(ctx, desc=None, pages="ok", rows=3, pos=A, slots=A, q=A, qs=1024, k=A, ks=256, v=A, vs=256,
            qo=A, qos=1024):
    d = None if desc is None else ctypes.byref(desc)
    p = _pages() if pages == "ok" else pages
    return ctx.lib.cpattn_norm_rope_write_kv(ctx._h, d, None if p is None else ctypes.byref(p), rows, pos,
                                             slots, q, qs, k, ks, v, vs, qo, qos, None)


def _needs_no_gpu():
    if torch.cuda.is_available():
        pytest.skip("would launch on stand-in pointers")


def test_e2m1_pages_are_taken_and_need_scales(lib):
    ctx = _ctx()
    for call in (_write, _read, _decode):
        assert call(ctx, _pages(format=E2M1, k_scales=0)) == cp.E_INVALID
        assert call(ctx, _pages(format=E2M1, v_scales=A + 4)) == cp.E_INVALID
        for fmt in (2, 3, 5):
            assert call(ctx, _pages(format=fmt)) == cp.E_INVALID
    _needs_no_gpu()
    for call in (_write, _read, _decode):  # past every check: no device to launch on
        assert call(ctx, _pages(format=E2M1)) == cp.E_CUDA


def test_plan_and_trim_refusals(lib):
    ctx, ok = _ctx(), _pages()
    for call in (_plan, _trim):
        assert call(ctx, None) == cp.E_INVALID
        assert call(ctx, ok, seqs=0) == cp.E_INVALID
        assert call(ctx, ok, seqs=cp.MAX_PAGED_SEQS + 1) == cp.E_UNSUPPORTED
        assert call(ctx, _pages(page_size=24)) == cp.E_UNSUPPORTED
        for name in ("lens", "free", "count"):
            assert call(ctx, ok, **{name: 0}) == cp.E_INVALID
            assert call(ctx, ok, **{name: A + 2}) == cp.E_INVALID
            assert ctx.last_error()
    for name in ("have", "new", "starts", "pos", "slots"):
        assert _plan(ctx, ok, **{name: 0}) == cp.E_INVALID
        assert _plan(ctx, ok, **{name: A + 1}) == cp.E_INVALID
    assert _plan(ctx, ok, rows=-1) == cp.E_INVALID
    assert _trim(ctx, ok, keep=0) == cp.E_INVALID
    _needs_no_gpu()
    assert _plan(ctx, ok) == cp.E_CUDA and _trim(ctx, ok) == cp.E_CUDA
    assert _plan(ctx, ok, rows=0, pos=0, slots=0) == cp.E_CUDA    # no rows: no arrays of rows


def test_norm_rope_refusals(lib):
    ctx = _ctx()
    for call in (_dense, _append):
        assert call(ctx, None) == cp.E_INVALID
        for kw in (dict(rotary_dim=-8), dict(rotary_dim=136), dict(rotary_dim=4), dict(rotary_dim=12),
                   dict(rope_steps=0), dict(rope_steps=A + 4), dict(eps=-1.0), dict(eps=float("nan")),
                   dict(q_weight=A + 2), dict(k_weight=A + 1)):
            assert call(ctx, _desc(**kw)) == cp.E_INVALID, kw
        for kw in (dict(rows=-1), dict(pos=0), dict(pos=A + 2), dict(q=0), dict(k=A + 8), dict(qo=0),
                   dict(qo=A + 2), dict(qs=1023), dict(qs=1000), dict(ks=248), dict(ks=260), dict(qos=8)):
            assert call(ctx, _desc(), **kw) == cp.E_INVALID, kw
            assert ctx.last_error()
        assert call(ctx, _desc(), rows=0) == cp.OK                # nothing to do: no launch
    for kw in (dict(ko=0), dict(ko=A + 4), dict(kos=128)):
        assert _dense(ctx, _desc(), **kw) == cp.E_INVALID, kw
    for kw in (dict(v=0), dict(v=A + 8), dict(vs=128), dict(vs=257), dict(slots=0), dict(slots=A + 1),
               dict(pages=None), dict(pages=_pages(format=3))):
        assert _append(ctx, _desc(), **kw) == cp.E_INVALID, kw
    _needs_no_gpu()
    assert _dense(ctx, _desc(rotary_dim=0, rope_steps=0, q_weight=0, k_weight=0)) == cp.E_CUDA
    for fmt in (0, 1, E2M1):
        assert _append(ctx, _desc(), pages=_pages(format=fmt)) == cp.E_CUDA


def test_null_context_refused(lib):
    p, d = ctypes.byref(_pages()), ctypes.byref(_desc())
    assert lib.cpattn_paged_plan(None, p, 1, 1, *[A] * 8, None) == cp.E_INVALID
    assert lib.cpattn_paged_trim(None, p, 1, A, A, A, A, None) == cp.E_INVALID
    assert lib.cpattn_norm_rope(None, d, 1, A, *[A, 1024] * 4, None) == cp.E_INVALID
    assert lib.cpattn_norm_rope_write_kv(None, d, p, 1, A, A, *[A, 1024] * 4, None) == cp.E_INVALID


def test_rope_steps_are_the_fixed_point_turns(lib):
    """Within one unit of 2^-64 turns of the exact product, over the frequencies in use
    and the extremes, and the negative of the positive one's."""
    rng = np.random.default_rng(1)
    f = np.concatenate([1e6 ** (-np.arange(128) / 128), 1e4 ** (-np.arange(64) / 64), [0.0, 1.0, 5e-324, 2.0 ** 20],
                        10.0 ** rng.uniform(-25, 6, 200)])
    f = np.concatenate([f, -f])
    steps = np.zeros(f.size, np.uint64)
    assert lib.cpattn_rope_steps(f.ctypes.data, f.size, steps.ctypes.data) == cp.OK
    for x, got in zip(f, steps):
        exact = Fraction(float(x)) / (2 * PI) * 2 ** 64
        off = (int(got) - exact) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 1, x
    assert lib.cpattn_rope_steps(None, 0, None) == cp.OK
    assert lib.cpattn_rope_steps(None, 1, steps.ctypes.data) == cp.E_INVALID
    assert lib.cpattn_rope_steps(f.ctypes.data, -1, steps.ctypes.data) == cp.E_INVALID
    for bad in (np.nan, np.inf, -np.inf, 2.0 ** 21):
        x = np.array([bad])
        assert lib.cpattn_rope_steps(x.ctypes.data, 1, steps.ctypes.data) == cp.E_INVALID


def test_binding_checks_tensors():
    kp, table = torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.zeros(2, 3, dtype=torch.int32)
    rec = torch.zeros(4, 2, 16, 8, dtype=torch.uint8)
    for ks, vs in ((None, None), (rec, None), (rec[..., :7], rec), (rec.float(), rec.float()),
                   (torch.zeros(4, 2, 16), torch.zeros(4, 2, 16)), (rec, rec)):   # (the last: not on a GPU)
        with pytest.raises(ValueError):
            cp.PagedKV(kp, kp, table, ks, vs)
    for kw in (dict(inv_freq=[1.0, 0.5, 0.1]), dict(inv_freq=[[1.0] * 4]), dict(inv_freq=[float("nan")] * 4),
               dict(inv_freq=[], q_weight=torch.zeros(128)),                      # not on a GPU
               dict(inv_freq=[], q_weight=torch.zeros(128, dtype=torch.float16))):
        with pytest.raises(ValueError):
            cp.NormRope(**kw)
    with pytest.raises(ValueError):
        binding._want_rows("q", torch.zeros(2, 3, 128, dtype=torch.bfloat16), 2, 3, 128, -1, torch.bfloat16)


# ------------------------------------------------------------------ oracle pins

def test_oracle_e2m1_rounding_by_hand():
    x = [0, .25, .2501, .75, .7499, 1.25, 1.2501, 1.75, 1.7499, 2.5, 2.5001, 3.5, 3.4999, 5, 5.0001, 7, 1e30]
    want = [0, 0, 1, 2, 1, 2, 3, 4, 3, 4, 5, 6, 5, 6, 7, 7, 7]
    assert oracle.to_e2m1(np.array(x)).tolist() == want
    assert oracle.to_e2m1(-np.array(x)).tolist() == [0] + [w | 8 for w in want[1:]]


@pytest.mark.parametrize("seed", range(3))
def test_oracle_quantise4_error_is_half_a_step(seed):
    """Groups of very different magnitudes, rows from 2^-130 to 2^127."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((60, 256)) * 2.0 ** np.repeat(rng.integers(-9, 1, (60, 8)), 32, 1)
    x = x * 2.0 ** rng.integers(-120, 120, (60, 1))
    bits = oracle.bf16_bits(torch.from_numpy(x).to(torch.bfloat16))
    bits[0] = 0
    x = oracle.bits_to_f64(bits)
    codes, rec = oracle.quantise4_rows(x)
    s = np.ascontiguousarray(rec[:, :4]).view(np.float32)[:, 0].astype(np.float64)
    r = oracle.e4m3_values()[rec[:, 4:]]
    amax = np.abs(x).reshape(60, 8, 32).max(-1)
    big = amax.max(-1) >= 2.0 ** -117
    ratio = amax.max(-1)[big] / s[big]
    assert np.all((512 <= ratio) & (ratio < 1024)) and np.all(np.exp2(np.round(np.log2(s))) == s)
    assert np.all(r <= 176) and np.all(np.abs(r * s[:, None] * 6 - amax) <= np.maximum(
        amax / 16, 6 * s[:, None] * 2.0 ** -10) * (1 + 1e-9))
    back = oracle.values4(codes, rec)
    unit = np.repeat(r * s[:, None], 32, 1)
    y = np.abs(x) / np.where(unit > 0, unit, np.inf)
    half = np.where(y <= 2, .25, np.where(y <= 4, .5, 1.0)) * unit
    half = np.where(unit > 0, half, np.abs(x))
    assert np.all(np.abs(back - x) <= half * (1 + 1e-9))
    assert np.all(codes[0] == 0) and np.all(rec[0, 4:] == 0)


def test_oracle_quantise4_of_nonfinite_rows():
    x = np.ones((3, 128))
    x[0, 5], x[1, 7] = np.inf, np.nan
    codes, rec = oracle.quantise4_rows(x)
    v = oracle.values4(codes, rec)
    assert np.isnan(v[:2]).all() and np.isfinite(v[2]).all() and np.abs(v[2] - 1).max() <= 1 / 16


def test_oracle_values4_by_hand():
    codes = np.zeros((1, 16), np.uint8)
    codes[0, :3] = [0x10, 0x7F, 0x92]            # 0, .5; -6, 6; 1, -.5
    rec = np.array([[0, 0, 0x00, 0x41, 0x3C]], np.uint8)     # s = 8, r = 1.5
    v = oracle.values4(codes, rec)[0]
    assert v[:6].tolist() == [0, 6, -72, 72, 12, -6] and np.all(v[6:] == 0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rotation_keeps_lengths_and_relative_positions(interleaved):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 2, 32))
    f = 1e4 ** (-np.arange(8) / 8)
    turn = lambda v, p: oracle.norm_rope_ref(v, [p] * 5, f, interleaved=interleaved)[0]  # noqa: E731
    assert np.allclose(np.square(turn(x, 777)).sum(-1), np.square(x).sum(-1), rtol=1e-13)
    assert np.array_equal(turn(x, 777)[..., 16:], x[..., 16:])
    q, k = x, rng.standard_normal(x.shape)
    a = (turn(q, 1000) * turn(k, 900)).sum(-1)
    b = (turn(q, 2 ** 30 + 100) * turn(k, 2 ** 30)).sum(-1)
    assert np.allclose(a, b, rtol=1e-9, atol=1e-9)
    one = oracle.norm_rope_ref(np.eye(32)[None, :1], [1], [np.pi / 2] * 4, interleaved=interleaved)[0][0, 0]
    assert abs(one[1 if interleaved else 4] - 1) < 1e-15 and abs(one[0]) < 1e-15


def test_oracle_norm_is_the_root_mean_square():
    rng = np.random.default_rng(3)
    x, w = rng.standard_normal((4, 3, 128)) * 100, rng.standard_normal(128)
    y, _ = oracle.norm_rope_ref(x, [0] * 4, [], w, eps=0.0)
    assert np.allclose(np.square(y / w).mean(-1), 1, rtol=1e-12)
    y, _ = oracle.norm_rope_ref(np.zeros((1, 1, 128)), [9], [1.0] * 4, w)
    assert np.all(y == 0)


def test_oracle_plan_by_hand():
    table = np.full((3, 3), 99)
    table[0, 0] = 7
    free = [1, 2, 3, 4]
    lens, starts, pos, slots, fine = oracle.plan_ref([15, -1, 0], [2, 5, 33], free, table, 16, 40)
    assert (lens, starts, fine) == ([17, -1, 33], [0, 2, 2, 35], True)
    assert table.tolist() == [[7, 4, 99], [99, 99, 99], [3, 2, 1]] and free == []
    assert pos[:5].tolist() == [15, 16, 0, 1, 2] and np.all(pos[35:] == -1) and np.all(slots[35:] == -1)
    assert slots[:4].tolist() == [7 * 16 + 15, 4 * 16, 48, 49] and slots[34] == 1 * 16
    oracle.trim_ref(lens, [15, -1, 0], free, table, 16)
    assert free == [1, 2, 3, 4]


def test_oracle_plan_serves_in_order():
    table = np.full((4, 8), -5)
    free = [1, 2]
    lens, _, pos, slots, fine = oracle.plan_ref([0, 0, 3, 0], [17, 1, 2, 1], free, table, 16, 100)
    assert lens == [17, 0, 5, 0] and not fine and free == []
    assert pos[17] == -1 and slots[17] == -1 and pos[18:20].tolist() == [3, 4] and pos[20] == -1
