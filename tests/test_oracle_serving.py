"""The serving oracle against closed forms, and the host side of the serving
operators: frequencies and every refusal (no GPU: all of them fail before any
CUDA call)."""

import math

import numpy as np
import pytest
import torch

from oracle import ref_fwd_slice
from oracle.serving import dequantize_rows, gather_rows, quantize_rows, ref_tree, rope_ref


def _freq(rot):
    return 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_scores_depend_on_the_distance_only(interleaved):
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((1, 64)), rng.standard_normal((1, 64))
    f = _freq(64)
    dots = [float((rope_ref(q, [p], f, interleaved) * rope_ref(k, [p - 7], f, interleaved)).sum())
            for p in (7, 100, 5000)]
    assert np.allclose(dots, dots[0], rtol=0, atol=1e-9)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_by_hand_and_part_of_the_head(interleaved):
    x = np.zeros((2, 64))
    a, b = (2, 3) if interleaved else (1, 9)
    x[1, a], x[1, 40] = 1.0, 5.0
    f = _freq(16)
    y = rope_ref(x, [0, 3], f, interleaved, factor=2.0)
    assert y[1, a] == pytest.approx(2 * math.cos(3 * f[1]), abs=1e-15)
    assert y[1, b] == pytest.approx(2 * math.sin(3 * f[1]), abs=1e-15)
    assert y[1, 40] == 5.0 and not y[0].any()


def test_rope_gradient_by_differences():
    rng = np.random.default_rng(2)
    x, dy = rng.standard_normal((3, 32)), rng.standard_normal((3, 32))
    pos, f = [5, 70000, -2], _freq(32)
    dx = rope_ref(dy, pos, f, False, 1.5, sign=-1.0)
    for r in range(3):
        for c in range(0, 32, 5):
            h = np.zeros_like(x)
            h[r, c] = 1e-3
            diff = ((rope_ref(x + h, pos, f, False, 1.5) - rope_ref(x - h, pos, f, False, 1.5)) * dy).sum() / 2e-3
            assert diff == pytest.approx(dx[r, c], abs=1e-9)


def test_row_quantisation_edges():
    x = np.zeros((6, 64), dtype=np.float32)
    x[1, 3], x[1, 4] = 448.0, -1.0
    x[2, 0] = 1e-38                      # its scale stays a normal number
    x[3, 0] = np.inf
    x[4, 5] = np.nan
    x[5] = 3.0
    codes, scale = quantize_rows(x)
    assert scale[0] == 1.0 and not codes[0].any()
    assert scale[1] == 1.0
    assert np.isnan(scale[3]) and np.isnan(scale[4])
    assert scale[2] >= np.finfo(np.float32).tiny
    back = dequantize_rows(codes, scale)
    assert back[1, 3] == 448.0 and back[1, 4] == -1.0
    assert abs(back[2, 0] - 1e-38) <= 1e-38 * 2.0 ** -4
    assert np.allclose(back[5], 3.0, rtol=1e-6)


def test_tree_oracle_chain_is_causal_attention():
    rng = np.random.default_rng(3)
    q, k, v = (rng.standard_normal((9, 64)) for _ in range(3))
    mask = np.tril(np.ones((9, 9)))
    o, lse, _ = ref_tree(q, k, v, 0, mask, 0.125)
    ro, rl = ref_fwd_slice(q, k, v, 0.125, True)
    assert np.allclose(o, ro, atol=1e-12) and np.allclose(lse, rl, atol=1e-12)
    # with a context: the last rows of causal attention
    o, lse, _ = ref_tree(q[6:], k, v, 6, mask, 0.125)
    assert np.allclose(o, ro[6:], atol=1e-12) and np.allclose(lse, rl[6:], atol=1e-12)


def test_tree_oracle_ignores_what_is_not_seen():
    rng = np.random.default_rng(4)
    q, k, v = (rng.standard_normal((3, 64)) for _ in range(3))
    k[1], v[1] = np.nan, np.inf
    mask = np.array([[1, 0, 0], [0, 0, 0], [1, 0, 1]])
    o, lse, _ = ref_tree(q, k, v, 0, mask, 0.125)
    assert np.allclose(o[0], v[0]) and not o[1].any() and lse[1] == -np.inf
    assert np.isfinite(o).all()


def test_gather_follows_the_table():
    pool = np.arange(4 * 2 * 16).reshape(4, 2, 16, 1)
    rows = gather_rows(pool, [3, 1], 1, 14, 4)[:, 0]
    assert rows.tolist() == [pool[3, 1, 14, 0], pool[3, 1, 15, 0], pool[1, 1, 0, 0], pool[1, 1, 1, 0]]


def test_rope_frequencies():
    from exact_io_aware_47_b200 import rope_frequencies
    f, a = rope_frequencies(64)
    assert f.dtype == torch.float64 and a == 1.0
    assert np.allclose(f.numpy(), _freq(64), rtol=1e-15)
    g, _ = rope_frequencies(64, scaling="linear", factor=4.0)
    assert np.allclose(g.numpy(), _freq(64) / 4, rtol=1e-15)
    g, _ = rope_frequencies(64, scaling="base", factor=4.0)
    assert g[0] == 1.0 and g[-1].item() == pytest.approx(_freq(64)[-1] / 4, rel=1e-12)
    g, a = rope_frequencies(64, scaling="ramp", factor=4.0, original_len=4096)
    turns = 4096 * _freq(64) / (2 * math.pi)
    fast, slow = turns >= 32, turns <= 1
    assert fast.any() and slow.any()
    assert np.allclose(g.numpy()[fast], _freq(64)[fast], rtol=1e-15)
    assert np.allclose(g.numpy()[slow], _freq(64)[slow] / 4, rtol=1e-15)
    mid = ~fast & ~slow
    part = (turns[mid] - 1) / 31
    assert np.allclose(g.numpy()[mid], _freq(64)[mid] * (part + (1 - part) / 4), rtol=1e-14)
    assert a == pytest.approx(1 + 0.1 * math.log(4))
    for bad in (dict(rot=7), dict(rot=64, factor=0.5), dict(rot=64, scaling="other"),
                dict(rot=64, scaling="ramp", factor=2.0), dict(rot=64, factor=float("nan")),
                dict(rot=64, scaling="ramp", factor=2.0, original_len=4096, ramp=(4.0, 4.0))):
        with pytest.raises(ValueError):
            rope_frequencies(**bad)


@pytest.fixture(scope="module")
def lib():
    from exact_io_aware_47_b200 import _lib, build
    build.build()
    return _lib.load()


P = 1 << 20   # never dereferenced: every case below fails validation first


def _i64(*s):
    import ctypes
    return (ctypes.c_int64 * 3)(*s)


def test_rope_refusals(lib):
    from exact_io_aware_47_b200 import _lib

    def rope(q=P, qs=None, qo=P, qos=None, Hq=2, k=None, ks=None, ko=None, kos=None, Hk=0, pos=None,
             pst=0, f=P, B=2, N=8, d=64, rot=64, inter=0, factor=1.0, dtype=0, fn=lib.fa_rope):
        return fn(q, qs, qo, qos, Hq, k, ks, ko, kos, Hk, pos, pst, f, B, N, d, rot, inter, factor,
                  dtype, None)
    for fn in (lib.fa_rope, lib.fa_rope_bwd):
        assert rope(q=None, fn=fn) == _lib.FA_ERR_INVALID_ARG
        assert rope(f=None, fn=fn) == _lib.FA_ERR_INVALID_ARG
        assert rope(N=0, fn=fn) == _lib.FA_ERR_INVALID_ARG
        assert rope(factor=0.0, fn=fn) == _lib.FA_ERR_INVALID_ARG
        assert rope(dtype=2, fn=fn) == _lib.FA_ERR_INVALID_ARG
        assert rope(pst=-1, fn=fn) == _lib.FA_ERR_INVALID_ARG
        assert rope(Hk=1, fn=fn) == _lib.FA_ERR_INVALID_ARG            # k is missing
        assert rope(k=P, ko=P, Hk=1, fn=fn) == _lib.FA_ERR_INVALID_ARG  # q_out is k
        assert rope(d=32, fn=fn) == _lib.FA_ERR_UNSUPPORTED
        for rot in (0, 8, 24, 80, -16):
            assert rope(rot=rot, fn=fn) == _lib.FA_ERR_UNSUPPORTED
        assert rope(B=1 << 12, Hq=1 << 10, N=1 << 10, fn=fn) == _lib.FA_ERR_UNSUPPORTED
        assert rope(q=P + 8, fn=fn) == _lib.FA_ERR_ALIGNMENT
        assert rope(pos=P + 2, fn=fn) == _lib.FA_ERR_ALIGNMENT
        assert rope(f=P + 4, fn=fn) == _lib.FA_ERR_ALIGNMENT
        assert rope(qs=_i64(1024, 512, 68), fn=fn) == _lib.FA_ERR_ALIGNMENT
        assert rope(qs=_i64(1024, -512, 64), fn=fn) == _lib.FA_ERR_INVALID_ARG
        # outputs whose rows share memory, and outputs that overlap their input
        far = P + (1 << 19)
        assert rope(qo=far, qos=_i64(0, 512, 64), fn=fn) == _lib.FA_ERR_INVALID_ARG
        assert rope(qo=far, qos=_i64(1024, 512, 32), fn=fn) == _lib.FA_ERR_INVALID_ARG
        assert rope(qo=P + 128, fn=fn) == _lib.FA_ERR_INVALID_ARG
        assert rope(qos=_i64(1024, 64, 128), fn=fn) == _lib.FA_ERR_INVALID_ARG


def _cache_cases(call):
    from exact_io_aware_47_b200 import _lib
    I, U, A = _lib.FA_ERR_INVALID_ARG, _lib.FA_ERR_UNSUPPORTED, _lib.FA_ERR_ALIGNMENT
    assert call(kc=None) == I and call(vc=None) == I and call(vc=P) == I
    assert call(ks=None) == I and call(vs=None) == I and call(vs=P) == I
    assert call(fmt=2) == I and call(dtype=7) == I
    assert call(pages=0) == I and call(page=0) == I and call(stride=0) == I
    assert call(table=None, pages=1) == I                       # a page for each sequence
    assert call(Hk=0) == I and call(B=0) == I
    assert call(page=24) == U and call(page=8) == U
    assert call(pages=1 << 30, Hk=2) == U
    assert call(d=96) == U
    assert call(kc=P + 8) == A and call(table=P + 2) == A and call(vs=P + 8) == A


def test_cache_write_refusals(lib):
    from exact_io_aware_47_b200 import _lib

    def write(k=P, kst=None, v=P, vst=None, kc=P, vc=2 * P, ks=P, vs=2 * P, table=P, stride=4,
              start=None, lens=None, B=2, Hk=2, N=4, d=64, pages=8, page=16, fmt=1, dtype=0):
        return lib.fa_cache_write(k, kst, v, vst, kc, vc, ks, vs, table, stride, start, lens, B, Hk,
                                  N, d, pages, page, fmt, dtype, None)
    _cache_cases(write)
    assert write(k=None) == _lib.FA_ERR_INVALID_ARG
    assert write(N=0) == _lib.FA_ERR_INVALID_ARG
    assert write(v=P + 4) == _lib.FA_ERR_ALIGNMENT
    assert write(start=P + 1) == _lib.FA_ERR_ALIGNMENT
    assert write(lens=P + 1) == _lib.FA_ERR_ALIGNMENT
    assert write(vst=_i64(0, 0, 4)) == _lib.FA_ERR_ALIGNMENT
    assert write(kst=_i64(-8, 0, 0)) == _lib.FA_ERR_INVALID_ARG
    assert write(B=1 << 10, Hk=1 << 10, N=1 << 10, pages=1 << 20) == _lib.FA_ERR_UNSUPPORTED


def test_cache_read_refusals(lib):
    from exact_io_aware_47_b200 import _lib

    def read(kc=P, vc=2 * P, ks=P, vs=2 * P, ko=3 * P, vo=4 * P, table=P, stride=4, start=None,
             lens=None, B=2, Hk=2, N=4, d=64, pages=8, page=16, fmt=1, dtype=0):
        return lib.fa_cache_read(kc, vc, ks, vs, ko, vo, table, stride, start, lens, B, Hk, N, d,
                                 pages, page, fmt, dtype, None)
    _cache_cases(read)
    assert read(ko=None) == _lib.FA_ERR_INVALID_ARG
    assert read(vo=3 * P) == _lib.FA_ERR_INVALID_ARG
    assert read(vo=4 * P + 8) == _lib.FA_ERR_ALIGNMENT
    assert read(lens=P + 2) == _lib.FA_ERR_ALIGNMENT


def test_tree_refusals(lib):
    from exact_io_aware_47_b200 import _lib
    ws = lib.fa_fwd_tree_workspace_size(2, 4, 2, 3, 64)
    assert ws > 0 and ws % 256 == 0

    def tree(q=P, kc=P, vc=2 * P, ks=P, vs=2 * P, o=P, lse=P, w=P, wb=ws, table=P, stride=4, ctx=P,
             drafts=None, mask=None, per=0, B=2, Hq=4, Hk=2, T=3, d=64, pages=8, page=16, scale=0.1,
             fmt=1, dtype=0):
        return lib.fa_fwd_tree(q, kc, vc, ks, vs, o, lse, w, wb, table, stride, ctx, drafts, mask, per,
                               B, Hq, Hk, T, d, pages, page, scale, fmt, dtype, None)
    _cache_cases(tree)
    I = _lib.FA_ERR_INVALID_ARG
    assert tree(q=None) == I and tree(o=None) == I and tree(lse=None) == I and tree(ctx=None) == I
    assert tree(Hq=3) == I                                      # heads that do not share evenly
    assert tree(T=0) == I and tree(scale=0.0) == I and tree(scale=float("nan")) == I
    assert tree(B=1 << 12, Hq=1 << 10, Hk=1 << 10, T=1 << 10, pages=1 << 13) == _lib.FA_ERR_UNSUPPORTED
    assert tree(q=P + 8) == _lib.FA_ERR_ALIGNMENT and tree(lse=P + 4) == _lib.FA_ERR_ALIGNMENT
    assert tree(ctx=P + 2) == _lib.FA_ERR_ALIGNMENT and tree(drafts=P + 2) == _lib.FA_ERR_ALIGNMENT
    assert tree(w=None) == _lib.FA_ERR_WORKSPACE and tree(wb=ws - 1) == _lib.FA_ERR_WORKSPACE
    assert tree(w=P + 16) == _lib.FA_ERR_ALIGNMENT
    # more key tiles than the kernel counts
    assert tree(B=1 << 10, stride=1 << 20, page=1 << 12) == _lib.FA_ERR_UNSUPPORTED
    assert lib.fa_fwd_tree_workspace_size(2, 3, 2, 3, 64) == 0
    assert lib.fa_fwd_tree_workspace_size(2, 4, 2, 3, 80) == 0


def test_binding_refuses_what_the_library_cannot_see():
    """Tensors off the GPU (host or meta stand for any other device), wrong
    shapes and types are ValueErrors, before any CUDA call."""
    import exact_io_aware_47_b200 as fa
    host = torch.zeros((2, 4, 8, 64), dtype=torch.bfloat16)
    meta = torch.zeros((2, 4, 8, 64), dtype=torch.bfloat16, device="meta")
    cache = torch.zeros((4, 4, 16, 64), dtype=torch.bfloat16)
    f, _ = fa.rope_frequencies(64)
    for x in (host, meta, host.float(), host[0, 0]):
        with pytest.raises(ValueError):
            fa.rope(x, x, f)
        with pytest.raises(ValueError):
            fa.rope_backward(x, None, f)
        with pytest.raises(ValueError):
            fa.cache_write(x, x, cache, cache)
        with pytest.raises(ValueError):
            fa.forward_tree(x, cache, cache, [1, 1])
    with pytest.raises(ValueError):
        fa.cache_read(cache, cache, [0, 0], 4)
    with pytest.raises(ValueError):
        fa.cache_read(None, cache, [0, 0], 4)
    with pytest.raises(ValueError):
        fa.cache_read(cache, cache, None, 4)


def test_strides_that_span_more_than_any_memory(lib):
    """A batch of 2^24 rows 2^40 elements apart would wrap around 64 bits.  (The
    calls have a rot of 24, or V rows 4 elements apart, which is looked at later:
    the strides alone decide between the two answers.)"""
    from exact_io_aware_47_b200 import _lib

    def rope(B, H, N, strides):
        return lib.fa_rope(P, strides, P, strides, H, None, None, None, None, 0, None, 0, P, B, N, 64, 24, 0,
                           1.0, 0, None)
    I, U = _lib.FA_ERR_INVALID_ARG, _lib.FA_ERR_UNSUPPORTED
    assert rope(1 << 24, 1, 1, _i64(1 << 40, 64, 64)) == I
    assert rope(1, 1 << 24, 1, _i64(64, 1 << 39, 64)) == I
    assert rope(2, 2, 1 << 20, _i64(1 << 30, 1 << 31, 1 << 21)) == I
    assert rope(2, 1, 1, _i64(1 << 40, 64, 64)) == U           # one step of 2^40
    assert rope(1, 1, 1, _i64(1 << 40, 1 << 40, 1 << 40)) == U  # no step at all
    assert rope(2, 4, 8, None) == U

    def write(strides):
        return lib.fa_cache_write(P, strides, P, _i64(0, 0, 4), 2 * P, 3 * P, None, None, P, 1, None, None,
                                  1 << 24, 1, 1, 64, 4, 16, 0, 0, None)
    assert write(_i64(1 << 40, 64, 64)) == I
    assert write(_i64(1 << 16, 64, 64)) == _lib.FA_ERR_ALIGNMENT   # V's


def _shares(x, xs, nx, y, ys, ny, d):
    """Whether any element of two views is the same, by writing all of them down."""
    def elements(at, st, n):
        rows = (at + st[0] * np.arange(n[0])[:, None, None] + st[1] * np.arange(n[1])[:, None]
                + st[2] * np.arange(n[2]))
        return set((rows[..., None] + np.arange(d)).ravel().tolist())
    return bool(elements(x, xs, nx) & elements(y, ys, ny))


def test_rope_outputs_of_q_that_share_memory_with_k(lib):
    """Every case is one that the checks before accept; a rot of 24 is refused
    after them, so that no call gets further."""
    from exact_io_aware_47_b200 import _lib
    I, U = _lib.FA_ERR_INVALID_ARG, _lib.FA_ERR_UNSUPPORTED
    B, N, d, far = 2, 3, 64, 1 << 24

    def rope(qo, qos, Hq, k, ks, ko, kos, Hk, q=None, qs=None):
        """Places in elements; q of its own memory unless given."""
        at = lambda e: P + 2 * e
        return lib.fa_rope(P + far if q is None else at(q), _i64(*(qos if qs is None else qs)), at(qo), _i64(*qos),
                           Hq, at(k), _i64(*ks), at(ko), _i64(*kos), Hk, None, 0, P, B, N, d, 24, 0, 1.0, 0, None)

    # one buffer of a projection, in place: heads side by side, and per head
    for W, sh, qat, kat, Hq, Hk in ((6 * d, d, 0, 4 * d, 4, 2), (6 * d, d, 2 * d, 0, 4, 2), (6 * d, 3 * d, 0, d, 2, 2),
                                    (8 * d, 2 * d, d, 0, 4, 4)):
        st = (N * W, sh, W)
        assert rope(qat, st, Hq, kat, st, kat, st, Hk, q=qat) == U
    st = (N * 6 * d, d, 6 * d)
    other = (N * 9 * d, 3 * d, 9 * d)
    assert rope(0, st, 4, 3 * d, st, 3 * d, st, 2, q=0) == I             # K's first head is Q's last
    assert rope(0, st, 4, 5 * d, st, 5 * d, st, 2, q=0) == I             # K's second head is the next row's first of Q
    assert rope(0, other, 3, d + 8, other, d + 8, other, 2, q=0) == U    # rows 0 .. 63 and 72 .. 135 of 192
    assert rope(0, other, 3, d - 8, other, d - 8, other, 2, q=0) == I    # and 56 .. 119
    contiguous = (4 * N * d, N * d, d)
    assert rope(1 << 20, contiguous, 4, 0, contiguous, 1 << 21, contiguous, 4) == U
    assert rope(64, contiguous, 4, 0, contiguous, 1 << 21, contiguous, 4) == I     # q_out in K
    assert rope(1 << 20, contiguous, 4, 0, contiguous, (1 << 20) + 64, contiguous, 4) == I  # in k_out
    qs = (4 * N * d, N * d, d)
    assert rope(1 << 20, qs, 4, 0, contiguous, 1 << 21, contiguous, 4, q=(1 << 21) + 64) == I  # k_out in Q
    # any strides and places, against all elements written down
    rng = np.random.default_rng(7)
    answers = {I: 0, U: 0}
    for _ in range(400):
        Hq, Hk = int(rng.integers(1, 4)), int(rng.integers(1, 4))

        def strides(H):
            dims, n, span = rng.permutation(3), (B, H, N), d
            st = [0, 0, 0]
            for i in dims:
                st[i] = span + 8 * int(rng.integers(0, 2)) * int(rng.integers(0, 9))
                span = st[i] * n[i]
            return tuple(st)
        qst, kst = strides(Hq), strides(Hk)
        if rng.random() < 0.6:
            kst = qst if Hk <= Hq else kst
            qst = qst if Hk <= Hq else kst
        qat, kat = 8 * int(rng.integers(0, 120)), 8 * int(rng.integers(0, 120))
        want = I if _shares(qat, qst, (B, Hq, N), kat, kst, (B, Hk, N), d) else U
        got = rope(qat, qst, Hq, kat, kst, kat, kst, Hk, q=qat)
        assert got == want, (qat, qst, Hq, kat, kst, Hk)
        answers[got] += 1
    assert min(answers.values()) > 30


@pytest.mark.parametrize("x", [[1.0, 2.0], [0, 1.5], np.array([1.0, 2.0]), torch.tensor([1.0, 2.0]),
                               torch.tensor([1.0, 2.0], dtype=torch.float16), torch.tensor([True, False]),
                               torch.tensor([1j, 2j]), [0, 2 ** 31], [-2 ** 31 - 1, 0],
                               torch.tensor([0, 1 << 32]), np.array([1 << 40, 0]), [0, 1 << 70]])
def test_integer_arguments_are_neither_cut_nor_wrapped(x):
    """Positions p / factor would be cut to whole ones, 2^32 would become 0."""
    from exact_io_aware_47_b200.serving import _int32_arg
    with pytest.raises(ValueError):
        _int32_arg("positions", x, (2,), torch.device("cpu"))


@pytest.mark.parametrize("dtype", [torch.int8, torch.uint8, torch.int16, torch.uint16, torch.int32, torch.uint32,
                                   torch.int64])
def test_integer_arguments_of_other_types(dtype):
    from exact_io_aware_47_b200.serving import _int32_arg
    want = torch.tensor([1, 100], dtype=torch.int32)
    for x in (torch.tensor([1, 100], dtype=dtype), torch.tensor([1, 100], dtype=dtype).numpy(), [1, 100]):
        got = _int32_arg("lens", x, (2,), torch.device("cpu"))
        assert got.dtype == torch.int32 and torch.equal(got, want)
    assert _int32_arg("lens", [-2 ** 31, 2 ** 31 - 1], (2,), torch.device("cpu")).tolist() == [-2 ** 31, 2 ** 31 - 1]
    with pytest.raises(ValueError):
        _int32_arg("lens", [1, 2, 3], (2,), torch.device("cpu"))


def test_the_clearing_flag_belongs_to_reading(lib):
    """Every call has a misaligned output or cache, looked at after the format."""
    from exact_io_aware_47_b200 import _lib
    I, A, clear = _lib.FA_ERR_INVALID_ARG, _lib.FA_ERR_ALIGNMENT, _lib.FA_CACHE_CLEAR

    def read(fmt):
        return lib.fa_cache_read(P, 2 * P, P, 2 * P, 3 * P, 4 * P + 8, P, 4, None, None, 2, 2, 4, 64, 8, 16, fmt, 0, None)

    def write(fmt):
        return lib.fa_cache_write(P, None, P, None, P + 8, 2 * P, P, 2 * P, P, 4, None, None, 2, 2, 4, 64, 8, 16, fmt,
                                  0, None)
    for fmt in (0, 1):
        assert read(fmt) == A and read(fmt | clear) == A and write(fmt) == A and write(fmt | clear) == I
    for fmt in (2, -1, 32, 8, clear | 2):
        assert read(fmt) == I
