"""The serving operators on the GPU (through the C ABI) against the float64
oracle: rotary positions, the paged K/V cache, attention of drafted tokens.

Tolerances, derived from the types (half = eps / 2, half a step of the 16-bit
type, is the error of one rounding to it):

* rope: one rounding of the result, plus fp32 sines and cosines: the angle
  enters fp32 as a fraction of a turn in [-1/2, 1/2] (error 2^-26 turns, i.e.
  2 pi 2^-26 < 2^-23), the function adds at most 2^-23, products and their sum
  3 * 2^-24 of |x_a| + |x_b|: together below 2^-21 (|x_a| + |x_b|) factor.
* cache: codes, scales and values read back are decided in fp32 on both
  sides: equal bit for bit.
* drafted tokens: with e the error of a score, p_j is off by a factor within
  exp(+-2e) (its own and the row sum's), then P is rounded to 16 bits or to
  8-bit pieces of at least that precision (half), sums run in fp32 (2^-24 per
  term), and O is rounded once:
      |dO| <= half |O| + (half + 4 e + L 2^-23) sum_j p_j |v_j|
  e = scale (2^-17 max|q| sum_c |k_jc| + 2 d 2^-24 sum_c |q_c k_jc|) + 2^-21:
  q may be held in 8-bit pieces of its row's largest value to 2^-17, products
  are summed in fp32, and 2^-21 covers the exponential.
      |dLSE| <= 2 e + L 2^-23 + 2^-22 |LSE|.
"""

import math

import numpy as np
import pytest
import torch

from helpers import f64
from oracle.fp8 import e4m3_decode
from oracle.serving import dequantize_rows, gather_rows, quantize_rows, ref_tree, rope_ref

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def fa():
    from exact_io_aware_47_b200 import build
    build.build()
    import exact_io_aware_47_b200 as pkg
    return pkg


def _ok(fa):
    st, word = fa.device_status()
    assert st == 0, f"device status {st} word {word:#x}"


def _half(dtype):
    return torch.finfo(dtype).eps / 2


# --------------------------------------------------------------------------- rope

def _rope_close(got, x, positions, f, interleaved, factor, sign, what=""):
    """got, x [B, H, N, d]; positions [B, N]."""
    rot = 2 * len(f)
    g, xs = f64(got), f64(x)
    mag = np.abs(xs).copy()
    for i in range(len(f)):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + len(f))
        mag[..., a] = mag[..., b] = np.abs(xs[..., a]) + np.abs(xs[..., b])
    for b in range(g.shape[0]):
        ref = rope_ref(xs[b], positions[b], f, interleaved, factor, sign)
        tol = _half(got.dtype) * np.abs(ref) + 2.0 ** -21 * factor * mag[b] + 2.0 ** -25
        bad = np.abs(g[b] - ref) > tol
        assert not bad.any(), f"{what}: {bad.sum()} beyond, worst {(np.abs(g[b] - ref) - tol).max():.3e}"
        assert np.array_equal(g[b][..., rot:], xs[b][..., rot:]), f"{what}: columns past rot"


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 96), (128, 32)])
def test_rope_matches_the_oracle(fa, dtype, interleaved, d, rot):
    g = torch.Generator().manual_seed(rot + d)
    for B, Hq, Hk, N in ((1, 1, 1, 1), (3, 8, 2, 37), (2, 5, 5, 130)):
        q, k = (torch.randn(B, H, N, d, generator=g).to(dtype).cuda() for H in (Hq, Hk))
        pos = torch.randint(-5, 1 << 20, (B, N), generator=g, dtype=torch.int32)
        f, _ = fa.rope_frequencies(rot, scaling="linear", factor=2.0)
        for fn, sign in ((fa.rope, 1.0), (fa.rope_backward, -1.0)):
            qo, ko = fn(q, k, f.cuda(), positions=pos.cuda(), interleaved=interleaved, factor=1.25)
            _ok(fa)
            for got, x in ((qo, q), (ko, k)):
                _rope_close(got, x, pos.numpy(), f.numpy(), interleaved, 1.25, sign, f"{B} {N} {sign}")


def test_rope_positions_and_layouts(fa):
    """Shared and default positions, host arguments, packed and token-major
    tensors, a broadcast input, outputs of other layouts, Q alone."""
    torch.manual_seed(5)
    B, Hq, Hk, N, d = 2, 4, 2, 33, 64
    f, _ = fa.rope_frequencies(32)
    fc = f.cuda()
    tok = torch.randn(B, N, Hq + 2 * Hk, d).to(BF16).cuda()
    q, k, v = tok.split([Hq, Hk, Hk], dim=2)
    q, k = q.transpose(1, 2), k.transpose(1, 2)
    iota = np.tile(np.arange(N), (B, 1))
    q1, k1 = fa.rope(q, k, fc)
    _rope_close(q1, q, iota, f.numpy(), False, 1.0, 1.0, "default positions")
    assert q1.is_contiguous() and k1.is_contiguous()
    shared = [7 * i % 50 for i in range(N)]
    q2, k2 = fa.rope(q, k, f.tolist(), positions=shared)
    _rope_close(k2, k, np.tile(shared, (B, 1)), f.numpy(), False, 1.0, 1.0, "shared positions")
    # Q alone, packed
    qp = q[0].contiguous()
    qo, none = fa.rope(qp, None, fc, positions=torch.tensor(shared).cuda())
    assert none is None and torch.equal(qo, q2[0])
    # one head broadcast over the batch
    wide = k[:1].expand(B, Hk, N, d)
    _, ko = fa.rope(q, wide, fc)
    assert torch.equal(ko[0], k1[0]) and torch.equal(ko[1], k1[0])
    # into a token-major output
    buf = torch.full((B, N, Hq, d), 9.0, dtype=BF16, device="cuda")
    qo, _ = fa.rope(q, None, fc, q_out=buf.transpose(1, 2))
    assert torch.equal(buf.transpose(1, 2), q1)
    # in place, inside the fused projection; V stays as it was
    before = tok.clone()
    fa.rope(q, k, fc, q_out=q, k_out=k)
    _ok(fa)
    assert torch.equal(q, q1) and torch.equal(k, k1)
    assert torch.equal(tok[:, :, Hq + Hk:], before[:, :, Hq + Hk:])
    from exact_io_aware_47_b200 import _lib
    with pytest.raises(_lib.FAError):                     # rows of the output share memory
        fa.rope(q, None, fc, q_out=torch.empty(1, Hq, N, d, dtype=BF16, device="cuda").expand(B, Hq, N, d))
    with pytest.raises(ValueError):
        fa.rope(q[..., ::2], None, fc)
    with pytest.raises(ValueError):
        fa.rope(q, k, fc, positions=torch.zeros(N + 1, dtype=torch.int32))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_backward_is_the_gradient(fa, interleaved):
    """Against differences of the forward (it is linear, so a wide difference is
    exact but for roundings: each of two results is off by half a step), and as
    the adjoint."""
    torch.manual_seed(6)
    B, H, N, d = 1, 2, 5, 64
    x = torch.randn(B, H, N, d).to(FP16).cuda()
    dy = torch.randn(B, H, N, d).to(FP16).cuda()
    pos = torch.tensor([0, 3, 999, 12345, 100000], dtype=torch.int32).cuda()
    f, _ = fa.rope_frequencies(48)
    fc = f.cuda()
    dx, _ = fa.rope_backward(dy, None, fc, positions=pos, interleaved=interleaved)
    for (h, n, c) in ((0, 1, 0), (1, 3, 17), (0, 4, 47), (1, 2, 60)):
        step = torch.zeros_like(x)
        step[0, h, n, c] = 8.0
        up, _ = fa.rope(step, None, fc, positions=pos, interleaved=interleaved)
        down, _ = fa.rope(-step, None, fc, positions=pos, interleaved=interleaved)
        diff = (f64(up) - f64(down)) / 16.0
        got = float((diff * f64(dy)).sum())
        # roundings: of up and down (relative half) and of dx itself
        tol = _half(FP16) * 2 * float((np.abs(diff) * np.abs(f64(dy))).sum()) + _half(FP16) * abs(got) + 2e-6
        assert abs(got - float(dx[0, h, n, c])) <= tol
    y, _ = fa.rope(x, None, fc, positions=pos, interleaved=interleaved)
    lhs, rhs = (f64(y) * f64(dy)).sum(), (f64(x) * f64(dx)).sum()
    tol = _half(FP16) * ((np.abs(f64(y) * f64(dy))).sum() + (np.abs(f64(x) * f64(dx))).sum()) + 1e-4
    assert abs(lhs - rhs) <= tol


# --------------------------------------------------------------------------- cache

def _pool(pages, Hk, page, d, dtype, e4m3):
    """A pool full of NaN: what is not written must not matter."""
    if e4m3:
        c = [torch.full((pages, Hk, page, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
        c = [x.view(torch.float8_e4m3fn) for x in c]
        s = [torch.full((pages, Hk, page), math.nan, device="cuda") for _ in range(2)]
        return c[0], c[1], s[0], s[1]
    c = [torch.full((pages, Hk, page, d), math.nan, dtype=dtype, device="cuda") for _ in range(2)]
    return c[0], c[1], None, None


def _table(B, per, pages, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(pages, generator=g)[:B * per].reshape(B, per).to(torch.int32)


def _raw(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x.view(torch.int16)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("d,page,N", [(128, 16, 1), (64, 16, 40), (128, 48, 131), (64, 128, 300)])
def test_cache_write_and_read(fa, dtype, e4m3, d, page, N):
    B, Hk = 4, 3
    g = torch.Generator().manual_seed(N + d)
    start, lens = [0, 5, 17, 2], [N, max(0, N - 7), 0, N]
    per = (N + 17 + page - 1) // page
    pages = B * per + 2
    table = _table(B, per, pages, N)
    kc, vc, ks, vs = _pool(pages, Hk, page, d, dtype, e4m3)
    k = torch.randn(B, N, Hk, d, generator=g).to(dtype)
    v = (torch.randn(B, Hk, N, d, generator=g) * torch.exp(2 * torch.randn(B, Hk, N, 1, generator=g))).to(dtype)
    k[0, 0, 0] = 0                                           # a row of zeros
    v[3, 1, 0] = 1e-7
    kd, vd = k.cuda().transpose(1, 2), v.cuda()
    want = [_raw(x).clone() for x in (kc, vc)]
    fa.cache_write(kd, vd, kc, vc, start, lens=lens, block_table=table.cuda(), k_scale=ks, v_scale=vs)
    _ok(fa)
    scales = [x.clone().fill_(math.nan) if e4m3 else None for x in (ks, vs)]
    for b in range(B):
        for n in range(lens[b]):
            j = start[b] + n
            at = (table[b, j // page].item(), slice(None), j % page)
            for i, x in enumerate((k[b, n], v[b, :, n])):
                if e4m3:
                    codes, sc = quantize_rows(x.float().numpy())
                    want[i][at] = torch.from_numpy(codes).cuda()
                    scales[i][at] = torch.from_numpy(sc).cuda()
                else:
                    want[i][at] = x.view(torch.int16).cuda()
    for i, (c, s) in enumerate(((kc, ks), (vc, vs))):
        # every byte of the pool: what was written, and that nothing else was
        # (the sign of a zero does not matter)
        got, ref = _raw(c), want[i]
        if e4m3:
            got, ref = (torch.where(x == 0x80, torch.zeros_like(x), x) for x in (got, ref))
            assert torch.equal(torch.nan_to_num(s, nan=-1.0), torch.nan_to_num(scales[i], nan=-1.0))
        assert torch.equal(got, ref), f"cache {i}"
    ko, vo = (torch.full((B, Hk, N, d), 3.0, dtype=dtype, device="cuda") for _ in range(2))
    fa.cache_read(kc, vc, start, N, lens=lens, block_table=table.cuda(), k_scale=ks, v_scale=vs,
                  k_out=ko, v_out=vo)
    _ok(fa)
    for out, c, s in ((ko, kc, ks), (vo, vc, vs)):
        ref = torch.full((B, Hk, N, d), 3.0, dtype=dtype)
        host, hs = c.cpu(), None if s is None else s.cpu()
        for b in range(B):
            for n in range(lens[b]):
                j = start[b] + n
                at = (table[b, j // page].item(), slice(None), j % page)
                if e4m3:
                    code = host.view(torch.uint8)[at].numpy()
                    ref[b, :, n] = (torch.from_numpy(e4m3_decode(code)).float() * hs[at].unsqueeze(-1)).to(dtype)
                else:
                    ref[b, :, n] = host[at]
        assert torch.equal(out.cpu(), ref)


def test_cache_without_a_table_and_new_outputs(fa):
    B, Hk, page, d = 2, 2, 32, 64
    kc, vc, ks, vs = _pool(3, Hk, page, d, BF16, True)
    k = torch.randn(B, Hk, page, d).to(BF16).cuda()
    fa.cache_write(k, 2 * k, kc.view(torch.uint8), vc.view(torch.uint8), k_scale=ks, v_scale=vs)
    ko, vo = fa.cache_read(kc, vc, [0, 4], 20, lens=[20, 3], k_scale=ks, v_scale=vs)
    _ok(fa)
    assert ko.dtype == BF16 and torch.equal(vo, 2 * ko)       # scales double, codes are the same
    assert not ko[1, :, 3:].any()
    err = (f64(ko[0]) - f64(k[0, :, :20]))
    amax = np.abs(f64(k[0, :, :20])).max(-1, keepdims=True)
    # e4m3: half a step relative, or half the smallest step of the row's scale; then one rounding
    tol = np.maximum(2.0 ** -4 * np.abs(f64(k[0, :, :20])), 2.0 ** -10 * amax / 448) * (1 + 2.0 ** -6) \
        + _half(BF16) * np.abs(f64(ko[0]))
    assert (np.abs(err) <= tol).all()
    assert torch.equal(ko[1, :, :3].float(), fa.cache_read(kc, vc, [0, 0], 32, k_scale=ks, v_scale=vs)[0][1, :, 4:7].float())


def test_cache_reports_what_it_cannot_place(fa):
    """Bad positions, lengths and pages: reported, and nothing outside the
    sequence's own slots is touched."""
    from exact_io_aware_47_b200 import _lib
    B, Hk, page, d, N = 2, 1, 16, 64, 8
    k = torch.randn(B, Hk, N, d).to(BF16).cuda()
    for start, lens, table in (([12, 0], [8, 8], [[0], [1]]), ([-1, 0], [8, 8], [[0], [1]]),
                               ([0, 0], [9, 8], [[0], [1]]), ([0, 0], [-3, 8], [[0], [1]]),
                               ([0, 0], [8, 8], [[4], [1]]), ([0, 0], [8, 8], [[-1], [1]]),
                               ([2 ** 31 - 1, 0], [8, 8], [[0], [1]])):
        kc, vc, _, _ = _pool(4, Hk, page, d, BF16, False)
        t = torch.tensor(table, dtype=torch.int32).cuda()
        fa.cache_write(k, k, kc, vc, start, lens=lens, block_table=t)
        assert fa.device_status()[0] == _lib.FA_ERR_DEVICE_SEQLEN
        assert torch.equal(kc[1, 0, :8], k[1, 0])              # the other sequence is written
        assert torch.isnan(kc[1, 0, 8:]).all() and torch.isnan(kc[2:]).all() and torch.isnan(vc[2:]).all()
        ko, vo = (torch.full((B, Hk, N, d), 3.0, dtype=BF16, device="cuda") for _ in range(2))
        fa.cache_read(kc, vc, start, N, lens=lens, block_table=t, k_out=ko, v_out=vo)
        assert fa.device_status()[0] == _lib.FA_ERR_DEVICE_SEQLEN
        assert torch.equal(ko[1], k[1])


def test_cache_rows_that_are_not_finite(fa):
    from exact_io_aware_47_b200 import _lib
    k = torch.randn(1, 1, 4, 64).to(BF16).cuda()
    k[0, 0, 1, 3] = math.inf
    k[0, 0, 2, 60] = math.nan
    kc, vc, ks, vs = _pool(1, 1, 16, 64, BF16, True)
    fa.cache_write(k, k, kc, vc, k_scale=ks, v_scale=vs)
    assert fa.device_status()[0] == _lib.FA_ERR_DEVICE_SCALE
    ko, _ = fa.cache_read(kc, vc, [0], 4, k_scale=ks, v_scale=vs)
    _ok(fa)
    assert torch.isnan(ko[0, 0, 1:3]).all() and torch.isfinite(ko[0, 0, [0, 3]]).all()


# --------------------------------------------------------------------------- drafted tokens

class Tree:
    """A batch over a paged cache whose unused slots hold NaN."""

    def __init__(self, B=2, Hq=4, Hk=2, T=3, ctx=(20, 33), drafts=None, d=64, page=16, dtype=BF16,
                 e4m3=True, mask="tree", seed=0, sink=0.0, spread=0.0):
        rng = np.random.default_rng(seed)
        self.B, self.Hq, self.Hk, self.T, self.d, self.page = B, Hq, Hk, T, d, page
        self.ctx, self.drafts, self.dtype, self.e4m3 = list(ctx), drafts, dtype, e4m3
        n = [T] * B if drafts is None else list(drafts)
        self.n = n
        per = max(1, max((c + T + page - 1) // page for c in ctx))
        pages = B * per + 2
        self.table = _table(B, per, pages, seed)
        self.kc, self.vc, self.ks, self.vs = _pool(pages, Hk, page, d, dtype, e4m3)
        self.keys, self.values = {}, {}
        for b in range(B):
            L = ctx[b] + n[b]
            for h in range(Hk):
                for store, cache, scale, what in ((self.keys, self.kc, self.ks, 0), (self.values, self.vc, self.vs, 1)):
                    x = rng.standard_normal((L, d))
                    if what == 0 and sink and L:
                        x[0] *= sink                           # one key that most of the weight goes to
                    if spread:
                        x *= np.exp(spread * rng.standard_normal((L, 1)))
                    x = torch.from_numpy(x).to(dtype)
                    if e4m3:
                        codes, sc = quantize_rows(x.float().numpy())
                        store[b, h] = dequantize_rows(codes, sc)
                        rows, srows = torch.from_numpy(codes).cuda(), torch.from_numpy(sc).cuda()
                    else:
                        store[b, h] = f64(x)
                        rows, srows = x.cuda(), None
                    for p0 in range(0, L, page):
                        m, pg = min(page, L - p0), self.table[b, p0 // page].item()
                        if e4m3:
                            cache.view(torch.uint8)[pg, h, :m] = rows[p0:p0 + m]
                            scale[pg, h, :m] = srows[p0:p0 + m]
                        else:
                            cache[pg, h, :m] = rows[p0:p0 + m]
        self.q = torch.from_numpy(rng.standard_normal((B, Hq, T, d))).to(dtype).cuda()
        if isinstance(mask, str) and mask == "tree":
            m = np.zeros((B, T, T), dtype=np.uint8)
            for b in range(B):
                for t in range(T):
                    m[b, t, t] = 1
                    if t:
                        m[b, t] |= m[b, rng.integers(0, t)]
            self.mask = m
        else:
            self.mask = mask
        self.scale = d ** -0.5

    def run(self, fa, **kw):
        a = dict(draft_lens=None if self.drafts is None else torch.tensor(self.drafts, dtype=torch.int32).cuda(),
                 tree_mask=None if self.mask is None else torch.as_tensor(self.mask).cuda(),
                 block_table=self.table.cuda(), k_scale=self.ks, v_scale=self.vs)
        a.update(kw)
        return fa.forward_tree(self.q, self.kc, self.vc, torch.tensor(self.ctx, dtype=torch.int32).cuda(), **a)

    def check(self, o, lse, what=""):
        half = _half(self.dtype)
        og, lg = f64(o), f64(lse)
        for b in range(self.B):
            m = np.tril(np.ones((self.T, self.T))) if self.mask is None else np.asarray(self.mask)
            m = m if m.ndim == 2 else m[b]
            n, L = self.n[b], self.ctx[b] + self.n[b]
            for h in range(self.Hq):
                k, v = self.keys[b, h // (self.Hq // self.Hk)], self.values[b, h // (self.Hq // self.Hk)]
                q = f64(self.q[b, h])[:n]
                ro, rl, sp = ref_tree(q, k, v, self.ctx[b], m[:n], self.scale)
                fin = np.isfinite(k).all(-1)
                ka = np.abs(k[fin]).sum(-1).max() if fin.any() else 0.0
                qk = (np.abs(q) @ np.abs(k[fin]).T).max(-1) if fin.any() else np.zeros(n)
                e = self.scale * (2.0 ** -17 * np.abs(q).max(-1) * ka + 2 * self.d * 2.0 ** -24 * qk) + 2.0 ** -21
                empty = rl == -np.inf
                assert (lg[b, h, :n][empty] == -np.inf).all() and not og[b, h, :n][empty].any(), f"{what} {b} {h}"
                tol = half * np.abs(ro) + (half + 4 * e + L * 2.0 ** -23)[:, None] * sp + 2.0 ** -25
                bad = ~(np.abs(og[b, h, :n] - ro) <= tol)
                assert not bad.any(), (f"{what} b{b} h{h}: {bad.sum()} of {bad.size} beyond, worst "
                                       f"{(np.abs(og[b, h, :n] - ro) - tol).max():.3e}, first {np.argwhere(bad)[0]}")
                ltol = 2 * e + L * 2.0 ** -23 + 2.0 ** -22 * np.abs(rl)
                assert (np.abs(lg[b, h, :n] - rl)[~empty] <= ltol[~empty]).all(), \
                    f"{what} b{b} h{h}: LSE {np.abs(lg[b, h, :n] - rl)[~empty].max():.3e}"


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_tree_small(fa, dtype, e4m3, d):
    """Lengths around the edges of pages and key tiles, with and without drafts."""
    for T, group, ctx, page in ((1, 1, (0, 1, 15), 16), (1, 4, (127, 128, 129), 32),
                                (5, 2, (0, 60, 123), 48), (8, 4, (300, 16, 511), 64),
                                (16, 4, (77, 256, 250), 128)):
        c = Tree(B=3, Hq=2 * group, Hk=2, T=T, ctx=ctx, d=d, page=page, dtype=dtype, e4m3=e4m3, seed=T + d)
        o, lse = c.run(fa)
        _ok(fa)
        c.check(o, lse, f"T{T} g{group} page{page}")


@pytest.mark.parametrize("dtype,e4m3", [(BF16, True), (FP16, True), (BF16, False), (FP16, False)])
@pytest.mark.parametrize("T,group", [(32, 1), (33, 1), (16, 8), (64, 3), (130, 1), (1, 17)])
def test_tree_many_rows(fa, dtype, e4m3, T, group):
    c = Tree(B=2, Hq=group, Hk=1, T=T, ctx=(200, 61), d=128 if T != 64 else 64, page=32, dtype=dtype,
             e4m3=e4m3, seed=T)
    o, lse = c.run(fa)
    _ok(fa)
    c.check(o, lse, f"T{T} g{group}")


@pytest.mark.parametrize("e4m3", [True, False])
def test_tree_lengths_differ_widely(fa, e4m3):
    """One sequence much longer than the others (its keys are split over the
    device and joined), empty contexts, a shared mask, no table."""
    c = Tree(B=5, Hq=4, Hk=1, T=4, ctx=(9000, 0, 1, 640, 2500), d=128, page=64, dtype=BF16, e4m3=e4m3, seed=8,
             mask=np.tril(np.ones((4, 4), dtype=np.uint8)))
    o, lse = c.run(fa)
    _ok(fa)
    c.check(o, lse, "long and short")
    o2, lse2 = c.run(fa, tree_mask=None)                    # the same mask, said as a chain
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o3, lse3 = c.run(fa)                                    # and the same bits again
    assert torch.equal(o, o3) and torch.equal(lse, lse3)


def _random_batch(fa, dtype, d, e4m3, T, B, Hk, longest):
    """Contexts of 0 .. longest - 1 positions, against float64 on the GPU."""
    group, page = 4, 48
    g = torch.Generator(device="cuda").manual_seed(T + d)
    ctx = torch.randint(0 if longest < 1000 else 1, longest, (B,), generator=g, device="cuda").to(torch.int32)
    per = (longest + T + page - 1) // page
    table = torch.randperm(B * per, generator=g, device="cuda").view(B, per).to(torch.int32)
    kc, vc, ks, vs = _pool(B * per, Hk, page, d, dtype, e4m3)
    n = longest + T
    k, v = (torch.randn(B, Hk, n, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    fa.cache_write(k, v, kc, vc, lens=ctx + T, block_table=table, k_scale=ks, v_scale=vs)
    q = torch.randn(B, Hk * group, T, d, generator=g, device="cuda").to(dtype)
    o, lse = fa.forward_tree(q, kc, vc, ctx, block_table=table, k_scale=ks, v_scale=vs)
    _ok(fa)
    half, scale = _half(dtype), d ** -0.5
    causal = torch.ones(T, T, dtype=torch.bool, device="cuda").tril()
    for b in range(B):
        L = int(ctx[b]) + T
        at = torch.arange(L, device="cuda")
        pg, row = table[b].long()[at // page], at % page

        def rows(c, s):
            if not e4m3:
                return c[pg, :, row].transpose(0, 1).double()
            x = c.view(torch.uint8)[pg, :, row].view(torch.float8_e4m3fn).double()
            return (x * s[pg, :, row].double().unsqueeze(-1)).transpose(0, 1)
        kd, vd = rows(kc, ks), rows(vc, vs)                  # [Hk, L, d]
        qd = q[b].double().view(Hk, group * T, d)
        s = qd @ kd.transpose(1, 2) * scale
        seen = torch.ones(T, L, dtype=torch.bool, device="cuda")
        seen[:, L - T:] = causal
        s = s.view(Hk, group, T, L).masked_fill(~seen, -math.inf).view(Hk, group * T, L)
        rl = torch.logsumexp(s, -1)
        pr = (s - rl.unsqueeze(-1)).exp()
        ro, sp = pr @ vd, pr @ vd.abs()
        ka = kd.abs().sum(-1).amax(-1)[:, None]
        qk = (qd.abs() @ kd.abs().transpose(1, 2)).amax(-1)
        e = scale * (2.0 ** -17 * qd.abs().amax(-1) * ka + 2 * d * 2.0 ** -24 * qk) + 2.0 ** -21
        tol = half * ro.abs() + (half + 4 * e + L * 2.0 ** -23).unsqueeze(-1) * sp + 2.0 ** -25
        err = (o[b].double().view(Hk, group * T, d) - ro).abs()
        assert bool((err <= tol).all()), f"b{b} L{L}: worst {(err - tol).max().item():.3e}"
        lerr = (lse[b].double().view(Hk, group * T) - rl).abs()
        assert bool((lerr <= 2 * e + L * 2.0 ** -23 + 2.0 ** -22 * rl.abs()).all()), f"b{b}: LSE {lerr.max().item():.3e}"


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("dtype,d", [(BF16, 128), (FP16, 64), (FP16, 128)])
@pytest.mark.parametrize("T", [1, 7, 13, 30])
def test_tree_many_tiles_in_a_row(fa, dtype, d, e4m3, T):
    """Enough keys that every SM works through tens of tiles and several items
    (all rings go round many times)."""
    _random_batch(fa, dtype, d, e4m3, T, 14, 8, 7000)


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("dtype,d", [(BF16, 128), (FP16, 64)])
@pytest.mark.parametrize("T", [1, 5, 16, 20])
def test_tree_many_short_items(fa, dtype, d, e4m3, T):
    """Items of one to four tiles, several per SM: pieces of the work begin and
    end in what an item counts beside its keys."""
    _random_batch(fa, dtype, d, e4m3, T, 150, 4, 400)


@pytest.mark.parametrize("dtype,e4m3", [(BF16, True), (FP16, True), (BF16, False)])
def test_tree_one_key_takes_most_of_the_weight(fa, dtype, e4m3):
    """A first key with scores far above the others', whose sum still counts:
    small probabilities may not be lost beside a large one."""
    for sink in (4.0, 8.0):
        c = Tree(B=2, Hq=4, Hk=1, T=2, ctx=(3000, 900), d=128, page=64, dtype=dtype, e4m3=e4m3, seed=11, sink=sink)
        o, lse = c.run(fa)
        _ok(fa)
        c.check(o, lse, f"sink {sink}")


@pytest.mark.parametrize("e4m3", [True, False])
def test_tree_rows_of_very_different_scales(fa, e4m3):
    c = Tree(B=2, Hq=4, Hk=2, T=4, ctx=(500, 130), d=64, page=16, dtype=BF16, e4m3=e4m3, seed=12, spread=1.5)
    o, lse = c.run(fa)
    _ok(fa)
    c.check(o, lse, "spread")


@pytest.mark.parametrize("e4m3", [True, False])
def test_tree_draft_lengths_and_empty_rows(fa, e4m3):
    """Rows behind draft_lens stay as they were; rows whose mask leaves no key
    (no context) are O = 0, LSE = -inf."""
    T = 6
    mask = np.eye(T, dtype=np.uint8)
    mask[2] = 0
    c = Tree(B=4, Hq=4, Hk=2, T=T, ctx=(0, 40, 0, 0), drafts=[6, 2, 0, 1], d=128, page=16, dtype=BF16,
             e4m3=e4m3, mask=mask, seed=13)
    out = torch.full((4, 4, T, 128), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((4, 4, T), 7.0, device="cuda")
    c.run(fa, out=out, lse=lse)
    _ok(fa)
    c.check(out, lse, "drafts")
    assert (lse[0, :, 2] == -math.inf).all()
    for b, n in enumerate(c.n):
        assert (out[b, :, n:] == 7.0).all() and (lse[b, :, n:] == 7.0).all()
    o2, lse2 = c.run(fa)                                    # new tensors: no result there
    assert not o2[2].any() and (lse2[2] == -math.inf).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, "lowest"])
@pytest.mark.parametrize("e4m3", [True, False])
def test_tree_masked_keys_may_hold_anything(fa, bad, e4m3):
    """A drafted token whose K or V is not finite (or the type's lowest value)
    touches only the queries that see it."""
    T, d, ctx = 4, 64, 30
    mask = np.tril(np.ones((T, T), dtype=np.uint8))
    mask[2, 1] = mask[3, 1] = 0
    value = torch.finfo(BF16).min if bad == "lowest" else bad
    for which in (0, 1):
        c = Tree(B=1, Hq=2, Hk=1, T=T, ctx=(ctx,), d=d, page=16, dtype=BF16, e4m3=e4m3, mask=mask, seed=14)
        clean, clean_lse = c.run(fa)
        page, row = c.table[0, (ctx + 1) // 16].item(), (ctx + 1) % 16
        cache, scale = ((c.kc, c.ks), (c.vc, c.vs))[which]
        if e4m3:
            scale[page, 0, row] = value
        else:
            cache[page, 0, row, 5] = value
        o, lse = c.run(fa)
        fa.device_status()
        for t in (0, 2, 3):
            assert torch.equal(o[0, :, t], clean[0, :, t]) and torch.equal(lse[0, :, t], clean_lse[0, :, t])
        if which and bad != "lowest" and not e4m3:          # column 5 of V at the query that sees it
            got, rest = o[0, :, 1, 5], o[0, :, 1, [c for c in range(d) if c != 5]]
            assert torch.isnan(got).all() if math.isnan(value) else (got == value).all()
            assert torch.equal(rest, clean[0, :, 1, [c for c in range(d) if c != 5]])
        if bad != "lowest" and math.isnan(value):
            assert torch.isnan(o[0, :, 1]).any()


def test_tree_refuses_masks_and_workspaces_that_it_cannot_use(fa):
    """A mask of additive terms means the opposite of one of flags, and a
    workspace elsewhere would be written to; nothing is launched for either."""
    c = Tree(B=2, Hq=2, Hk=1, T=2, ctx=(30, 30), d=64, page=16, dtype=BF16, seed=16)
    good, _ = c.run(fa)

    def run(**kw):
        return fa.forward_tree(c.q, c.kc, c.vc, torch.tensor([30, 30], dtype=torch.int32).cuda(),
                               k_scale=c.ks, v_scale=c.vs, block_table=c.table.cuda(), **kw)[0]
    flags = torch.as_tensor(c.mask).cuda()
    need = fa.tree_workspace_bytes(2, 2, 1, 2, 64)
    for bad in (flags.float(), torch.zeros(2, 2), [[0.0, -math.inf], [0.0, 0.0]]):
        with pytest.raises(ValueError):
            run(tree_mask=bad)
    for bad in (torch.empty(need, dtype=torch.uint8), torch.empty(2 * need, dtype=torch.uint8).cuda()[::2],
                need):
        with pytest.raises(ValueError):
            run(tree_mask=flags, workspace=bad)
    o = run(tree_mask=flags, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    _ok(fa)
    assert torch.equal(o, good)


def test_tree_reports_bad_lengths_and_pages(fa):
    from exact_io_aware_47_b200 import _lib
    c = Tree(B=2, Hq=2, Hk=1, T=2, ctx=(30, 30), d=64, page=16, dtype=BF16, seed=15)
    good, _ = c.run(fa)
    _ok(fa)
    per = c.table.shape[1]
    for ctx, drafts, table in (([-4, 30], None, None), ([per * 16 + 9, 30], None, None), ([30, 30], [3, 2], None),
                               ([30, 30], [-1, 2], None), ([30, 30], None, 1000), ([30, 30], None, -7)):
        t = c.table.clone()
        if table is not None:
            t[0, 1] = table
        kw = dict(block_table=t.cuda())
        if drafts:
            kw["draft_lens"] = torch.tensor(drafts, dtype=torch.int32).cuda()
        o, _ = fa.forward_tree(c.q, c.kc, c.vc, torch.tensor(ctx, dtype=torch.int32).cuda(), k_scale=c.ks,
                               v_scale=c.vs, tree_mask=torch.as_tensor(c.mask).cuda(), **kw)
        assert fa.device_status()[0] == _lib.FA_ERR_DEVICE_SEQLEN
        assert torch.equal(o[1], good[1])                   # the other sequence is right


@pytest.mark.parametrize("e4m3,T", [(True, 3), (False, 3), (True, 70), (False, 70)])
def test_tree_wait_timeout_is_reported_and_the_context_stays_usable(fa, e4m3, T):
    """Ordinary waits, given 1 ns (as in test_gpu_timeout.py)."""
    from exact_io_aware_47_b200 import _lib
    c = Tree(B=3, Hq=4, Hk=2, T=T, ctx=(700, 0, 3000), d=128, page=16, dtype=BF16, e4m3=e4m3, seed=17)
    good, _ = c.run(fa)
    _ok(fa)
    prev = _lib.fa_set_wait_limit_ns(1)
    try:
        c.run(fa)
    finally:
        _lib.fa_set_wait_limit_ns(prev)
    st, word = fa.device_status()
    assert st == _lib.FA_ERR_DEVICE_TIMEOUT, f"status {st} word {word:#x}"
    assert (word >> 8) & 0xFF in range(60, 90), f"site of word {word:#x}"
    again, _ = c.run(fa)
    _ok(fa)
    assert torch.equal(good, again)


def test_tree_shared_pages_and_other_streams(fa):
    """Two sequences with the same prefix pages; a call on a side stream; two
    captured graphs that share one workspace, replayed in turn."""
    c = Tree(B=2, Hq=4, Hk=2, T=4, ctx=(96, 96), d=128, page=32, dtype=BF16, seed=16)
    for b in (0, 1):
        for h in range(2):
            c.keys[1, h], c.values[1, h] = c.keys[0, h], c.values[0, h]
    c.table[1] = c.table[0]
    o, lse = c.run(fa)
    _ok(fa)
    c.check(o, lse, "shared pages")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, lse2 = c.run(fa)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)

    ctx = torch.tensor(c.ctx, dtype=torch.int32).cuda()
    mask, table = torch.as_tensor(c.mask).cuda(), c.table.cuda()
    ws = torch.empty(fa.tree_workspace_bytes(2, 4, 2, 4, 128), dtype=torch.uint8, device="cuda")
    qs, outs, graphs = [c.q.clone(), -c.q], [], []
    for q in qs:
        buf = (torch.empty_like(q), torch.empty(2, 4, 4, device="cuda"))
        call = lambda: fa.forward_tree(q, c.kc, c.vc, ctx, tree_mask=mask, block_table=table, k_scale=c.ks,
                                       v_scale=c.vs, out=buf[0], lse=buf[1], workspace=ws)
        with torch.cuda.stream(side):
            call()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
        outs.append(buf)
    want = [fa.forward_tree(q, c.kc, c.vc, ctx, tree_mask=mask, block_table=table, k_scale=c.ks, v_scale=c.vs)
            for q in qs]
    for _ in range(3):
        for buf in outs:
            buf[0].fill_(5.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for buf, w in zip(outs, want):
            assert torch.equal(buf[0], w[0]) and torch.equal(buf[1], w[1])


def test_offsets_past_32_bits(fa):
    """A pool of more than 2^32 bytes: writing to, reading from and attending
    over its last pages."""
    Hk, page, d = 8, 256, 128
    pages = (1 << 32) // (Hk * page * d) + 5                # e4m3: one byte per element
    kc, vc = (torch.empty((pages, Hk, page, d), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    ks, vs = (torch.empty((pages, Hk, page), device="cuda") for _ in range(2))
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32).cuda()
    small = [torch.zeros((2, Hk, page, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    sscale = [torch.ones((2, Hk, page), device="cuda") for _ in range(2)]
    stable = torch.tensor([[1, 0]], dtype=torch.int32).cuda()
    k = torch.randn(1, Hk, 400, d, device="cuda").to(BF16)
    v = torch.randn(1, Hk, 400, d, device="cuda").to(BF16)
    q = torch.randn(1, 16, 1, d, device="cuda").to(BF16)
    got = []
    for c, s, t in (((kc, vc), (ks, vs), table), (small, sscale, stable)):
        fa.cache_write(k, v, c[0], c[1], block_table=t, k_scale=s[0], v_scale=s[1])
        got.append((*fa.cache_read(c[0], c[1], [0], 400, block_table=t, k_scale=s[0], v_scale=s[1]),
                    *fa.forward_tree(q, c[0], c[1], [399], block_table=t, k_scale=s[0], v_scale=s[1])))
    _ok(fa)
    for a, b in zip(*got):
        assert torch.equal(a, b)


# --------------------------------------------------------------------------- together

@pytest.mark.parametrize("e4m3", [True, False])
def test_decoding_with_drafts_end_to_end(fa, e4m3):
    """A prompt and two drafted steps, as a server runs them: rotate, write,
    attend; the drafted chain equals dense causal attention of the same
    (dequantised) keys and values, and the prefix read back feeds the dense
    kernel."""
    torch.manual_seed(21)
    B, H, d, page, n0, T = 2, 4, 64, 16, 90, 6
    N = n0 + 2 * T
    f = fa.rope_frequencies(64)[0].cuda()
    q, k, v = (torch.randn(B, H, N, d).to(BF16).cuda() for _ in range(3))
    per = (N + page - 1) // page
    table = _table(B, per, B * per, 3).cuda()
    kc, vc, ks, vs = _pool(B * per, H, page, d, BF16, e4m3)
    outs = []
    for at, n in ((0, n0), (n0, T), (n0 + T, T)):
        pos = torch.arange(at, at + n, dtype=torch.int32, device="cuda")
        part = [x[:, :, at:at + n] for x in (q, k, v)]
        qr, kr = fa.rope(part[0], part[1], f, positions=pos)
        start = torch.full((B,), at, dtype=torch.int32, device="cuda")
        fa.cache_write(kr, part[2], kc, vc, start, block_table=table, k_scale=ks, v_scale=vs)
        if at:
            outs.append(fa.forward_tree(qr, kc, vc, start, block_table=table, k_scale=ks, v_scale=vs))
    _ok(fa)
    qr, _ = fa.rope(q, None, f)
    kd, vd = fa.cache_read(kc, vc, [0] * B, N, block_table=table, k_scale=ks, v_scale=vs)
    o, lse = fa.forward(qr, kd, vd, causal=True)
    _ok(fa)
    from helpers import LSE_MAX_ABS, O_MAX_ABS, O_MEAN_ABS
    for i, (ot, lt) in enumerate(outs):
        at = n0 + i * T
        # the dense kernel's own tolerance; K and V read back are rounded once
        # more (half of a score's and a value's size)
        err = np.abs(f64(ot) - f64(o[:, :, at:at + T]))
        assert err.max() <= 2 * O_MAX_ABS and err.mean() <= 2 * O_MEAN_ABS
        slack = 0.0 if not e4m3 else \
            _half(BF16) * np.abs(f64(qr)).max() * np.abs(f64(kd)).sum(-1).max() * d ** -0.5
        assert np.abs(f64(lt) - f64(lse[:, :, at:at + T])).max() <= 2 * LSE_MAX_ABS + slack


def test_training_with_rotary_positions(fa):
    """rope -> forward -> backward -> rope_backward against float64 autograd."""
    from helpers import GRAD_REL_MAX, O_MAX_ABS
    torch.manual_seed(22)
    B, H, N, d = 1, 2, 200, 64
    f, _ = fa.rope_frequencies(32, scaling="ramp", factor=2.0, original_len=128)
    q, k, v, do = (torch.randn(B, H, N, d).to(BF16).cuda() for _ in range(4))
    qr, kr = fa.rope(q, k, f.cuda(), interleaved=True)
    o, lse = fa.forward(qr, kr, v, causal=True)
    dqr, dkr, dv = fa.backward(qr, kr, v, o, lse, do, causal=True)
    dq, dk = fa.rope_backward(dqr, dkr, f.cuda(), interleaved=True)
    _ok(fa)
    leaves = [x.double().cpu().requires_grad_() for x in (q, k, v)]

    def rot(x):
        ang = torch.arange(N, dtype=torch.float64)[:, None] * f
        c, s = ang.cos(), ang.sin()
        a, b = x[..., :32:2], x[..., 1:32:2]
        return torch.cat((torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2), x[..., 32:]), -1)
    s = rot(leaves[0]) @ rot(leaves[1]).transpose(-1, -2) * d ** -0.5
    s = s.masked_fill(torch.triu(torch.ones(N, N, dtype=torch.bool), 1), -math.inf)
    ref = s.softmax(-1) @ leaves[2]
    grads = torch.autograd.grad(ref, leaves, do.double().cpu())
    assert (o.double().cpu() - ref).abs().max() <= O_MAX_ABS
    for got, want in zip((dq, dk, dv), grads):
        assert (got.double().cpu() - want).abs().max() <= GRAD_REL_MAX * want.abs().max()


# --------------------------------------------------------------------------- scales of V rows

class SinkTree(Tree):
    """Bf16 or fp16 queries over an e4m3 cache whose key `at` of every head has
    a score of `gap` (the others': about a normal distribution), zeros as its V
    row unless `keep`, and V of standard deviation std elsewhere."""

    def __init__(self, gap, std, at=(0,), keep=False, **kw):
        super().__init__(e4m3=True, **kw)
        rng = np.random.default_rng(99)
        q = rng.standard_normal((self.B, self.Hq, self.T, self.d))
        q[..., 0] = 8.0
        self.q = torch.from_numpy(q).to(self.dtype).cuda()
        for b in range(self.B):
            L = self.ctx[b] + self.n[b]
            for h in range(self.Hk):
                k, v = rng.standard_normal((L, self.d)), std * rng.standard_normal((L, self.d))
                k[:, 0] = 0.0
                for j in at:
                    k[j] = 0.0
                    k[j, 0] = gap / (8.0 * self.scale)
                    if not keep:
                        v[j] = 0.0
                self.put(b, h, k, v)

    def put(self, b, h, k, v):
        """K and V rows of one sequence and head, quantised into the cache."""
        for store, cache, scale, x in ((self.keys, self.kc, self.ks, k), (self.values, self.vc, self.vs, v)):
            codes, sc = quantize_rows(torch.from_numpy(x).to(self.dtype).float().numpy())
            store[b, h] = dequantize_rows(codes, sc)
            at = np.arange(len(x))
            pages = self.table[b].numpy()[at // self.page]
            cache.view(torch.uint8)[pages, h, at % self.page] = torch.from_numpy(codes).cuda()
            scale[pages, h, at % self.page] = torch.from_numpy(sc).cuda()

    def check_relative(self, o, lse, what="", absolute=0.0):
        """As check(), with no absolute term beside the output type's own
        smallest step (fp16's 2^-24; bf16's is far below all of these).
        `absolute`: of a key, relative to the row's largest probability."""
        half = _half(self.dtype)
        least = 2.0 ** -25 if self.dtype == FP16 else 0.0
        og, lg = f64(o), f64(lse)
        for b in range(self.B):
            m = np.asarray(self.mask)[b]
            n, L = self.n[b], self.ctx[b] + self.n[b]
            for h in range(self.Hq):
                k, v = self.keys[b, h // (self.Hq // self.Hk)], self.values[b, h // (self.Hq // self.Hk)]
                q = f64(self.q[b, h])[:n]
                ro, rl, sp = ref_tree(q, k, v, self.ctx[b], m[:n], self.scale)
                qk = (np.abs(q) @ np.abs(k).T).max(-1)
                e = self.scale * (2.0 ** -17 * np.abs(q).max(-1) * np.abs(k).sum(-1).max()
                                  + 2 * self.d * 2.0 ** -24 * qk) + 2.0 ** -21
                seen = np.ones((n, L), bool)
                seen[:, self.ctx[b]:] = m[:n, :n] != 0
                top = np.exp(np.where(seen, self.scale * (q @ k.T), -np.inf).max(-1) - rl)
                tol = half * np.abs(ro) + (half + 4 * e + L * 2.0 ** -23)[:, None] * sp + least \
                    + L * absolute * top[:, None]
                err = np.abs(og[b, h, :n] - ro)
                assert (err <= tol).all(), f"{what} b{b} h{h}: worst {(err / tol).max():.3g} times the tolerance"
                ltol = 2 * e + L * 2.0 ** -23 + 2.0 ** -22 * np.abs(rl)
                assert (np.abs(lg[b, h, :n] - rl) <= ltol).all(), \
                    f"{what} b{b} h{h}: LSE {(np.abs(lg[b, h, :n] - rl) / ltol).max():.3g} times the tolerance"


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,group", [(1, 4), (8, 4), (16, 4), (32, 4)])
def test_tree_zero_v_row_that_takes_the_weight(fa, dtype, d, T, group):
    """A key whose V row is zero (stored with the scale 1) and whose score is far
    above the others' takes weight and adds nothing; what the others add may not
    be lost beside it."""
    for gap, std in ((12.0, 0.1), (10.0, 0.01), (12.0, 0.01), (7.0, 1e-3), (0.0, 1e-3)):
        c = SinkTree(gap, std, B=2, Hq=group, Hk=1, T=T, ctx=(3000, 900), d=d, page=64, dtype=dtype, seed=31)
        o, lse = c.run(fa)
        _ok(fa)
        c.check_relative(o, lse, f"gap {gap} std {std}")


@pytest.mark.parametrize("T", [1, 8, 16, 32])
def test_tree_zero_v_rows_small_values_and_far_scores(fa, T):
    """V far below one, zero rows in many places (a drafted one, all of a tile,
    every third key), scores so far apart that the other keys count for 2^-87."""
    kw = dict(B=1, Hq=4, Hk=1, T=T, ctx=(1500,), d=128, page=32, dtype=BF16, seed=32)
    for gap, std, at in ((0.0, 1e-5, (0,)), (3.0, 1e-6, (700,)), (12.0, 0.01, (1500,)), (5.0, 0.01, range(128, 256)),
                         (2.0, 0.01, range(0, 1500, 3)), (60.0, 0.1, (0,)), (60.0, 0.1, (900, 1400))):
        c = SinkTree(gap, std, at=at, **kw)
        o, lse = c.run(fa)
        _ok(fa)
        c.check_relative(o, lse, f"gap {gap} std {std} at {at}")


@pytest.mark.parametrize("T", [1, 8, 16, 32])
def test_tree_every_v_row_zero(fa, T):
    c = SinkTree(3.0, 0.0, B=2, Hq=4, Hk=1, T=T, ctx=(1000, 5), d=128, page=32, dtype=BF16, seed=33)
    o, lse = c.run(fa)
    _ok(fa)
    assert not o.any()
    c.check_relative(o, lse, "zeros")


@pytest.mark.parametrize("T", [1, 32])
def test_tree_v_rows_of_scale_one(fa, T):
    """Rows whose largest value is 448 have the scale of a row of zeros."""
    for at, gap in (((), 0.0), ((0,), 12.0), ((0, 200), 3.0)):
        c = SinkTree(gap, 0.1, at=at, B=1, Hq=4, Hk=1, T=T, ctx=(700,), d=128, page=32, dtype=BF16, seed=34)
        rng = np.random.default_rng(35)
        v = 40.0 * rng.standard_normal((c.ctx[0] + T, 128))
        v[:, 3] = 448.0
        v[list(at)] = 0.0
        c.put(0, 0, c.keys[0, 0], v)
        assert (c.vs[c.table[0].long().cuda(), 0].flatten()[:len(v)] == 1.0).all()
        o, lse = c.run(fa)
        _ok(fa)
        c.check_relative(o, lse, f"at {at}")


@pytest.mark.parametrize("T", [1, 8, 16, 32])
@pytest.mark.parametrize("std", [1e-28, 1e-29, 1e-31, 1e-33, 1e-37])
def test_tree_v_rows_of_the_smallest_scales(fa, T, std):
    """bf16 values down to the smallest that cache_write has a scale for (2^-126):
    products p * v_scale are held to 2^-28 of the largest, or of 2^-90 of the
    largest p (fa.h), and a code is at most 448."""
    c = SinkTree(0.0, std, keep=True, B=1, Hq=4, Hk=1, T=T, ctx=(700,), d=128, page=32, dtype=BF16, seed=36)
    assert (c.vs[c.table[0].long().cuda(), 0].flatten()[:700] < 2.0 ** -90).all()
    o, lse = c.run(fa)
    _ok(fa)
    c.check_relative(o, lse, f"std {std}", absolute=448 * 2.0 ** -118)


@pytest.mark.parametrize("T", [1, 32])
def test_tree_a_v_scale_of_zero(fa, T):
    """Codes times a scale of zero are zeros, like any other row of them."""
    c = SinkTree(12.0, 0.01, keep=True, B=1, Hq=4, Hk=1, T=T, ctx=(700,), d=128, page=32, dtype=BF16, seed=37)
    c.vs[c.table[0, 0].item(), 0, 0] = 0.0
    c.values[0, 0][0] = 0.0
    o, lse = c.run(fa)
    _ok(fa)
    c.check_relative(o, lse, "scale 0")


# --------------------------------------------------------------------------- memory that is shared

def test_rope_in_place_inside_one_projection_per_head(fa):
    """Q, K and V of a head side by side: address ranges overlap, rows do not."""
    torch.manual_seed(41)
    B, N, H, d = 2, 19, 3, 64
    buf = torch.randn(B, N, H, 3, d).to(BF16).cuda()
    q, k, v = (buf[:, :, :, i].transpose(1, 2) for i in range(3))
    f = fa.rope_frequencies(d)[0].cuda()
    want = fa.rope(q.contiguous(), k.contiguous(), f)
    before = v.clone()
    fa.rope(q, k, f, q_out=q, k_out=k)
    _ok(fa)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, before)
    from exact_io_aware_47_b200 import _lib
    kept = buf.clone()
    with pytest.raises(_lib.FAError):                       # Q's output begins inside K's first row
        fa.rope(q.contiguous(), k, f, q_out=buf.view(-1)[d + 8:][:B * H * N * d].view(B, H, N, d), k_out=k)
    assert torch.equal(buf, kept)


def test_wide_integers_on_the_device(fa):
    """int64 device tensors: the same results, and a value past int32 is told as
    out of range instead of being taken for a small one."""
    from exact_io_aware_47_b200 import _lib
    torch.manual_seed(42)
    q = torch.randn(2, 2, 5, 64).to(BF16).cuda()
    f = fa.rope_frequencies(64)[0].cuda()
    pos = torch.randint(0, 1 << 20, (2, 5)).cuda()
    a, b = (fa.rope(q, None, f, positions=p)[0] for p in (pos, pos.to(torch.int32)))
    assert torch.equal(a, b)
    with pytest.raises(ValueError):
        fa.rope(q, None, f, positions=pos / 2)
    with pytest.raises(ValueError):
        fa.rope(q, None, f, positions=(pos / 2).cpu())
    c = Tree(B=2, Hq=2, Hk=1, T=2, ctx=(30, 20), d=64, page=16, dtype=BF16, seed=43)
    good = c.run(fa)
    ctx, mask = torch.tensor(c.ctx).cuda(), torch.as_tensor(c.mask).cuda()

    def run(ctx, table=c.table.cuda().long()):
        return fa.forward_tree(c.q, c.kc, c.vc, ctx, tree_mask=mask, block_table=table, k_scale=c.ks, v_scale=c.vs)
    got = run(ctx)
    _ok(fa)
    assert torch.equal(got[0], good[0]) and torch.equal(got[1], good[1])
    got = run(ctx + torch.tensor([1 << 32, 0]).cuda())      # 30 if it wrapped
    assert fa.device_status()[0] == _lib.FA_ERR_DEVICE_SEQLEN
    assert torch.equal(got[0][1], good[0][1])
    with pytest.raises(ValueError):
        run([30 + (1 << 32), 20])
    with pytest.raises(ValueError):
        run([30.0, 20.0])
    with pytest.raises(ValueError):
        run(ctx, c.table.cuda().float())


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_cache_read_leaves_no_row_of_a_new_tensor_unwritten(fa, e4m3, d):
    """Rows behind lens, of positions past the table and of pages that are not in
    the pool are zeros in new tensors, whatever their memory held; tensors that
    the caller gives keep them."""
    from exact_io_aware_47_b200 import _lib
    B, Hk, page, N = 3, 2, 16, 150
    per = 10
    table = _table(B, per, B * per + 1, 44)
    kc, vc, ks, vs = _pool(B * per + 1, Hk, page, d, BF16, e4m3)
    g = torch.Generator(device="cuda").manual_seed(44)
    k, v = (torch.randn(B, Hk, per * page, d, generator=g, device="cuda").to(BF16) for _ in range(2))
    fa.cache_write(k, v, kc, vc, block_table=table.cuda(), k_scale=ks, v_scale=vs)
    _ok(fa)
    table[1, 3], table[2, 0] = B * per + 1, -1
    t = table.cuda()
    kw = dict(block_table=t, k_scale=ks, v_scale=vs)
    whole = [torch.full((B, Hk, N, d), 3.0, dtype=BF16, device="cuda") for _ in range(2)]
    for start, lens in (([0, 0, 0], None), ([140, 7, 3], None), ([0, 0, 0], [150, 60, 0]), ([30, 2, 0], [150, 149, 33]),
                        ([0, 0, 2 ** 31 - 1], None), ([0, -3, 0], [0, 150, 150]), ([0, 0, 0], [-1, 200, 150])):
        for x in whole:
            x.fill_(3.0)
        got = fa.cache_read(kc, vc, start, N, lens=lens, k_out=whole[0], v_out=whole[1], **kw)
        assert fa.device_status()[0] == _lib.FA_ERR_DEVICE_SEQLEN
        assert got[0] is whole[0]
        junk = [torch.full((B, Hk, N, d), 7.0, dtype=BF16, device="cuda") for _ in range(2)]
        torch.cuda.synchronize()
        del junk
        new = fa.cache_read(kc, vc, start, N, lens=lens, **kw)
        half = fa.cache_read(kc, vc, start, N, lens=lens, v_out=whole[1].clone(), **kw)
        assert fa.device_status()[0] == _lib.FA_ERR_DEVICE_SEQLEN
        for i in range(2):
            kept = (whole[i] == 3.0).all(-1, keepdim=True)
            assert kept.any() and not kept.all()
            assert torch.equal(new[i], torch.where(kept, torch.zeros_like(new[i]), whole[i])), f"{start} {lens} {i}"
        assert torch.equal(half[0], new[0]) and torch.equal(half[1], whole[1])


@pytest.mark.parametrize("e4m3", [True, False])
def test_tree_leaves_no_row_of_a_new_tensor_unwritten(fa, e4m3):
    """More drafted tokens than a sequence's table has positions: the last ones
    have no key and no result, and the new tensors say so."""
    from exact_io_aware_47_b200 import _lib
    c = Tree(B=2, Hq=2, Hk=1, T=20, ctx=(0, 0), drafts=[16, 16], d=64, page=16, dtype=BF16, e4m3=e4m3, mask=None,
             seed=45)
    table = c.table[:, :1].contiguous().cuda()
    want = c.run(fa, block_table=table)
    _ok(fa)
    junk = [torch.full((2, 2, 20, 64), 7.0, dtype=BF16, device="cuda"), torch.full((2, 2, 20), 7.0, device="cuda")]
    torch.cuda.synchronize()
    del junk
    o, lse = c.run(fa, block_table=table, draft_lens=None)
    assert fa.device_status()[0] == _lib.FA_ERR_DEVICE_SEQLEN
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert not o[:, :, 16:].any() and (lse[:, :, 16:] == -math.inf).all()


# --------------------------------------------------------------------------- drafted values that are not finite

def _poisoned(fa, dtype, e4m3, d, T, group, ctx, Hk, value, chain, page=32, drafts=None):
    """The batch twice: clean, and with one element of V that is not finite in one
    drafted token of every third sequence and head.  Queries that do not see the
    token keep every bit, those that see it all columns but the element's."""
    B, Hq = len(ctx), Hk * group
    g = torch.Generator(device="cuda").manual_seed(T + d + B)
    n = torch.tensor([T] * B if drafts is None else drafts, device="cuda")
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    per = (max(ctx) + T + page - 1) // page
    table = torch.randperm(B * per, generator=g, device="cuda").view(B, per).to(torch.int32)
    kc, vc, ks, vs = _pool(B * per, Hk, page, d, dtype, e4m3)
    k, v = (torch.randn(B, Hk, max(ctx) + T, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    fa.cache_write(k, v, kc, vc, lens=(c + n).to(torch.int32), block_table=table, k_scale=ks, v_scale=vs)
    q = torch.randn(B, Hq, T, d, generator=g, device="cuda").to(dtype)
    mask = torch.ones(T, T, device="cuda").tril()
    if not chain:
        mask = mask * (torch.rand(T, T, generator=g, device="cuda") < 0.5)
        mask.fill_diagonal_(1)                               # (a token sees itself: some query sees each)
    mask = mask.to(torch.uint8)
    kw = dict(draft_lens=None if drafts is None else n.to(torch.int32), tree_mask=None if chain else mask,
              block_table=table, k_scale=ks, v_scale=vs)
    clean, clean_lse = fa.forward_tree(q, kc, vc, c, **kw)
    _ok(fa)
    assert torch.isfinite(clean).all()
    raw = vc.view(torch.uint8) if e4m3 else vc
    hit = torch.zeros(B, Hq, T, d, dtype=torch.bool, device="cuda")
    for b in range(0, B, 3):
        for h in range(b % 2, Hk, 2):
            u, col = (5 * b + 7 * h) % max(1, int(n[b])), (11 * b + 17 * h + 3) % d
            if u >= int(n[b]):
                continue
            j = ctx[b] + u
            raw[int(table[b, j // page]), h, j % page, col] = 0x7F + 0x80 * (b % 2) if e4m3 else value
            sees = (mask[:, u] != 0) & (torch.arange(T, device="cuda") < n[b])
            hit[b, h * group:(h + 1) * group, :, col] |= sees
    assert hit.any() and not hit.all()
    o, lse = fa.forward_tree(q, kc, vc, c, **kw)
    _ok(fa)
    assert torch.equal(lse, clean_lse)
    got = o[hit]
    if e4m3 or math.isnan(value):
        assert torch.isnan(got).all(), f"{int((~torch.isnan(got)).sum())} of {got.numel()} lost"
    else:
        assert (got == value).all(), f"{int((got != value).sum())} of {got.numel()} lost"
    assert torch.equal(o[~hit], clean[~hit]), f"{int((o[~hit] != clean[~hit]).sum())} reached others"


_NOT_FINITE = [(BF16, True, math.nan), (FP16, True, math.nan), (BF16, False, math.nan), (FP16, False, math.inf),
               (BF16, False, -math.inf), (FP16, False, math.nan)]


@pytest.mark.parametrize("dtype,e4m3,value", _NOT_FINITE)
@pytest.mark.parametrize("T,group", [(1, 8), (2, 4), (8, 4), (16, 4), (33, 4), (130, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_tree_drafted_values_that_are_not_finite(fa, dtype, e4m3, value, T, group, d):
    """Every tile of rows, drafted tokens on either side of a tile's edge, short
    and long contexts (whose items are cut over many CTAs), with and without masks."""
    for chain in (True, False) if T > 1 else (True,):
        _poisoned(fa, dtype, e4m3, d, T, group, [30, 0, 120, 4000], 2, value, chain)
        _poisoned(fa, dtype, e4m3, d, T, group, [9000], 1, value, chain, page=48)
    if T > 2:
        _poisoned(fa, dtype, e4m3, d, T, group, [125, 40, 0, 500], 2, value, False, drafts=[T - 1, 0, T, T // 2])


@pytest.mark.parametrize("dtype,e4m3,value", _NOT_FINITE)
@pytest.mark.parametrize("T,group", [(2, 4), (8, 4), (16, 4), (33, 4)])
def test_tree_many_items_some_of_them_not_finite(fa, dtype, e4m3, value, T, group):
    """Items of one to three tiles, about ten in a row per SM: what one of them
    found may not be taken for another's."""
    _poisoned(fa, dtype, e4m3, 128, T, group, [(37 * b) % 290 for b in range(400)], 4, value, False)
