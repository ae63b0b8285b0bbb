"""GPU parity of the 4-bit packed history against its definition in 64 bits: records bit for
bit, attention over the values that the records stand for within the bounds of
packed_ref.attend_tol."""
import numpy as np
import pytest
import torch

from tests import hga_cases as hc
from tests import packed_ref as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    hc.ensure_built()
    assert torch.cuda.is_available()
    yield
    import hierarchical_sparse_long_b200 as hga
    assert hga.hga_get_device_status() == 0


def f64(t):
    return t.double().cpu().numpy()


def host(a, dtype=BF16):
    """A host array's values in dtype, on the device."""
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(dtype)


def keys(rng, *shape):
    """Keys with an offset per slice of 64 tokens and two strong channels."""
    x = rng.standard_normal(shape)
    x[..., 3] += 6.0
    x[..., 17] *= 5.0
    return x


# ------------------------------------------------------------------ records
# (B, Hkv, D, dtype, first chunk, chunks, cap, head stride beyond the chunks)
PACK = [
    (1, 1, 64, "bf16", 0, 1, 1, 0),
    (1, 1, 128, "fp32", 0, 1, 3, 0),
    (2, 3, 128, "bf16", 2, 5, 9, 37),
    (3, 2, 64, "fp32", 1, 3, 4, 1),
    (1, 5, 64, "bf16", 4, 7, 11, 128),
    (1, 8, 128, "bf16", 0, 40, 41, 0),
]


@pytest.mark.parametrize("case", PACK, ids=str)
def test_records_are_the_definition_bit_for_bit(case):
    import hierarchical_sparse_long_b200 as hga
    B, H, D, dtype, first, n, cap, extra = case
    rng = np.random.default_rng(sum(case[:3]) + n)
    dt = BF16 if dtype == "bf16" else torch.float32
    stride = n * 64 + extra
    k, v = host(keys(rng, B, H, stride, D), dt), host(rng.standard_normal((B, H, stride, D)), dt)
    hist = torch.full((B, H, cap, hga.hga_packed_chunk_bytes(D)), 0xA5, device="cuda", dtype=torch.uint8)
    summ = torch.full((B, H, cap, D), 7.0, device="cuda")
    hga.hga_pack_history(k, v, stride, B, H, D, first, n, hist, cap, summ, cap)
    rec, kv, vv = ref.pack(f64(k)[:, :, :n * 64], f64(v)[:, :, :n * 64])
    got = hist.cpu().numpy()
    assert np.array_equal(got[:, :, first:first + n], rec)
    assert np.all(got[:, :, :first] == 0xA5) and np.all(got[:, :, first + n:] == 0xA5)
    want = torch.full_like(summ, 7.0)
    chunk0 = torch.empty(B, H, n, D, device="cuda")
    hga.hga_build_summaries(k, stride, B, H, D, 64, 0, n, chunk0, n)
    want[:, :, first:first + n] = chunk0
    assert torch.equal(summ, want)
    # and back, to either type, rows behind the chunks left as they were
    for out in (BF16, torch.float32):
        k2 = torch.full((B, H, stride, D), 7.0, device="cuda", dtype=out)
        v2 = torch.full_like(k2, 7.0)
        hga.hga_unpack_history(hist, cap, B, H, D, first, n, k2, v2, stride)
        for t, x in ((k2, kv), (v2, vv)):
            assert np.array_equal(f64(t)[:, :, :n * 64], x)
            assert torch.all(t[:, :, n * 64:] == 7.0)


def test_without_summaries_and_no_chunks():
    import hierarchical_sparse_long_b200 as hga
    rng = np.random.default_rng(3)
    k, v = host(keys(rng, 1, 2, 128, 64)), host(rng.standard_normal((1, 2, 128, 64)))
    hist = torch.zeros(1, 2, 2, 72 * 64, device="cuda", dtype=torch.uint8)
    hga.hga_pack_history(k, v, 128, 1, 2, 64, 0, 2, hist, 2)
    assert np.array_equal(hist.cpu().numpy(), ref.pack(f64(k), f64(v))[0])
    before = hist.clone()
    hga.hga_pack_history(k, v, 128, 1, 2, 64, 2, 0, hist, 2)
    hga.hga_unpack_history(hist, 2, 1, 2, 64, 0, 0, k, v, 128)
    assert torch.equal(hist, before)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 128])
def test_extreme_groups(D, dtype):
    """Constant, tiny, huge and non-finite groups, and values on the borders between codes."""
    import hierarchical_sparse_long_b200 as hga
    rng = np.random.default_rng(D)
    dt = BF16 if dtype == "bf16" else torch.float32
    n = 5
    k, v = keys(rng, 1, 1, n * 64, D), rng.standard_normal((1, 1, n * 64, D))
    k[..., 0] = 1.5                                     # no range: read back as they are
    k[..., 1] = 2.0 ** -110 * rng.standard_normal(n * 64)  # a range below the smallest step
    k[..., 2] = 1e30 * rng.standard_normal(n * 64)
    k[..., 4] = np.arange(n * 64) % 16                  # the grid's own points
    k[..., 5] = np.arange(n * 64) % 31 / 2              # and halfway between
    k[..., 6] = 1000 + 0.01 * rng.standard_normal(n * 64)
    k[:, :, 7, 7] = np.nan
    k[:, :, 70, 8] = np.inf
    k[:, :, 130, 9], k[:, :, 131, 9] = np.inf, -np.inf
    v[:, :, 5] = -0.75
    v[:, :, 6] = np.arange(D) % 16
    v[:, :, 7] = np.arange(D) % 31 / 2
    v[:, :, 9, 33] = np.nan
    v[:, :, 10, 2] = -np.inf
    v[:, :, 11] *= 1e30
    v[:, :, 12] *= 2.0 ** -110
    k, v = host(k, dt), host(v, dt)
    hist = torch.zeros(1, 1, n, 72 * D, device="cuda", dtype=torch.uint8)
    hga.hga_pack_history(k, v, n * 64, 1, 1, D, 0, n, hist, n)
    rec, kv, vv = ref.pack(f64(k), f64(v))
    assert np.array_equal(hist.cpu().numpy(), rec)
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    hga.hga_unpack_history(hist, n, 1, 1, D, 0, n, k2, v2, n * 64)
    assert np.array_equal(f64(k2), kv, equal_nan=True) and np.array_equal(f64(v2), vv, equal_nan=True)
    assert np.all(np.isnan(f64(k2)[0, 0, :64, 7])) and np.all(f64(k2)[0, 0, :, 0] == 1.5)
    g = 32 // 64 * 64
    assert np.all(np.isnan(f64(v2)[0, 0, 9, g:g + 64]))
    # the documented bound of a finite group: half a step, the roundings of z and of the
    # value, and the range that rounding s lost (15 steps of 2^-8, over at most both ends)
    for t, t2, axis in ((f64(k).reshape(n, 64, D), f64(k2).reshape(n, 64, D), 1),
                        (f64(v).reshape(n * 64, D // 64, 64), f64(v2).reshape(n * 64, D // 64, 64), 2)):
        s, z, _ = ref.quant(t, axis)
        with np.errstate(invalid="ignore"):
            bound = 0.5 * s + 2.0 ** -8 * abs(z) + 2.0 ** -8 * abs(t2) + 15 * 2.0 ** -8 * s + (s == 0) * 2.0 ** -96
            assert np.all((abs(t - t2) <= bound) | ~np.isfinite(s))


@pytest.mark.parametrize("offset", [0.0, 3.0, 1000.0])
def test_values_next_to_the_borders_between_codes(offset):
    """fp32 values at, and 1 to 2^12 steps of fp32 to either side of, every border of grids with
    steps of 8 significant bits; far offsets, whose z is rounded by more than a step, too."""
    import hierarchical_sparse_long_b200 as hga
    rng = np.random.default_rng(5)
    D, n = 128, 3
    k, v = np.empty((1, 1, n * 64, D), np.float32), np.empty((1, 1, n * 64, D), np.float32)
    for at in np.ndindex(n, D):  # a channel of a chunk is a group of K
        step = np.float32(rng.integers(128, 256)) * np.float32(2.0) ** -9
        x = (rng.integers(0, 15, 64) + np.float32(0.5)).astype(np.float32) * step + np.float32(offset)
        x = (x.view(np.int32) + rng.choice([0, 1, -1, 3, -17, 4096, -4096], 64).astype(np.int32)).view(np.float32)
        x[0], x[1] = offset, offset + 15 * step
        k[0, 0, 64 * at[0]:64 * at[0] + 64, at[1]] = x
        v[0, 0, 64 * at[0] + at[1] % 64, 64 * (at[1] // 64):64 * (at[1] // 64) + 64] = x
    hist = torch.zeros(1, 1, n, 72 * D, device="cuda", dtype=torch.uint8)
    k, v = host(k, torch.float32), host(v, torch.float32)
    hga.hga_pack_history(k, v, n * 64, 1, 1, D, 0, n, hist, n)
    assert np.array_equal(hist.cpu().numpy(), ref.pack(f64(k), f64(v))[0])


# Groups of 64 elements whose distances x - z, or (16 + c) s + z, do not fit 24 bits; every grid
# below is exactly representable, so that borders fall where they are meant to.
def _huge_ranges(rng, n):
    """Finite grids of which x - z, up to 31 s, passes the largest fp32 number."""
    lo = np.array([0.0, 1e37, 1e38, -1e38, -3e37])[rng.integers(0, 5, n)][:, None]
    hi = lo + 10.0 ** rng.uniform(36, 38.3, n)[:, None]
    x = np.linspace(lo[:, 0], np.minimum(hi, 3.3e38)[:, 0], 64, axis=1)
    x[n // 2:] = lo[n // 2:] + rng.random((n - n // 2, 64)) * (np.minimum(hi, 3.3e38) - lo)[n // 2:]
    x[:, 0] = lo[:, 0]
    return x


def _far_offsets(rng, n):
    """Steps of 8 bits at offsets of 2^12 to 2^23 steps: elements at, and a few places beside, the borders."""
    step = rng.integers(128, 256, n)[:, None] / 128.0
    x = 2.0 ** rng.integers(12, 24, n)[:, None] + 16 * step + rng.integers(0, 31, (n, 64)) / 2 * step
    x = _beside(rng, x, 2)
    x[:, :2] = x[:, :1] + np.array([0, 15]) * step
    return x


def _small_z(rng, n):
    """Smallest elements a few places of fp32 from 16 steps: z is 2^-19 to 2^-16 of the step."""
    step = rng.integers(128, 256, n)[:, None] / 128.0
    lo = 16 * step * (1 + rng.integers(-8, 9, n)[:, None] * 2.0 ** -23)
    x = np.maximum(_beside(rng, 16 * step + rng.integers(0, 31, (n, 64)) / 2 * step, 2), lo)
    x[:, :2] = lo + np.array([0, 15]) * step
    return x


def _border_at_zero(rng, n):
    """Grids with the border between two codes at 0, or 2^-8 of a step from it, and elements closer still."""
    step, m = rng.integers(128, 256, n)[:, None] / 128.0, rng.integers(0, 15, n)[:, None]
    z = -(m + 16.5) * step
    ok = (ref.to_bf16(z) == z) | (rng.random((n, 1)) < 0.3)
    x = rng.choice([-1, 1], (n, 64)) * 2.0 ** rng.integers(-38, -9, (n, 64)) * step + (rng.random((n, 1)) < 0.5) * 2.0 ** -8 * step
    x[:, 2:12] = (rng.integers(0, 31, (n, 10)) / 2 - m - 0.5) * step
    x[:, :2] = (np.array([0, 15]) - m - 0.5) * step
    return np.where(ok, x, rng.standard_normal((n, 64)))


def _beside(rng, x, places):
    """fp32 values up to so many places beside x."""
    x = np.asarray(x, np.float32)
    return (x.view(np.int32) + rng.integers(-places, places + 1, x.shape).astype(np.int32)).view(np.float32).astype(np.float64)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("groups", [_huge_ranges, _far_offsets, _small_z, _border_at_zero], ids=lambda f: f.__name__[1:])
def test_codes_where_fp32_distances_round(groups, dtype):
    """The nearest code of every finite group: record for record the 64-bit decision."""
    import hierarchical_sparse_long_b200 as hga
    dt = BF16 if dtype == "bf16" else torch.float32
    rng = np.random.default_rng(17)
    D, n = 128, 24
    x = groups(rng, 2 * n * D)
    k = host(x[:n * D].reshape(n, D, 64).swapaxes(1, 2).reshape(1, 1, n * 64, D), dt)  # a channel of a chunk is a group
    v = host(x[n * D:].reshape(n, 2, 64, 64).swapaxes(1, 2).reshape(1, 1, n * 64, D), dt)  # 64 channels of a token
    hist = torch.zeros(1, 1, n, 72 * D, device="cuda", dtype=torch.uint8)
    hga.hga_pack_history(k, v, n * 64, 1, 1, D, 0, n, hist, n)
    want, kv, vv = ref.pack(f64(k), f64(v))
    got = hist.cpu().numpy()
    assert np.isfinite(kv).any(axis=2).mean() > 0.5  # not all of the grids overflow
    bad = np.argwhere(got != want)
    assert not len(bad), f"{len(bad)} of {want.size} bytes differ, the first at {bad[0]}"


# ------------------------------------------------------------------ attention
class Packed:
    """A packed history of random chunks, its values in 64 bits and a bf16 window or segment."""

    def __init__(self, B, Hq, Hkv, D, topk, nc, n_seg, blocks, seed=0, cap_extra=2, stride_extra=5, routes="random"):
        import hierarchical_sparse_long_b200 as hga
        rng = np.random.default_rng(7 * seed + B + Hq + nc + topk)
        self.shape = (B, Hq, Hkv, D, topk, nc)
        self.cap = nc + cap_extra
        self.stride = n_seg + stride_extra
        self.n_seg, self.blocks = n_seg, blocks
        self.hist = torch.full((B, Hkv, self.cap, 72 * D), 0xFF, device="cuda", dtype=torch.uint8)
        kh, vh = host(keys(rng, B, Hkv, nc * 64, D)), host(rng.standard_normal((B, Hkv, nc * 64, D)))
        if nc:
            hga.hga_pack_history(kh, vh, nc * 64, B, Hkv, D, 0, nc, self.hist, self.cap)
            _, self.kh, self.vh = ref.pack(f64(kh), f64(vh))
        rows = 64 * blocks if n_seg == 64 * blocks else 1
        self.rows = rows
        self.q = host(rng.standard_normal((B, Hq, rows, D)))
        self.k = torch.full((B, Hkv, self.stride, D), float("nan"), device="cuda", dtype=BF16)
        self.v = torch.full_like(self.k, float("nan"))
        self.k[:, :, :n_seg] = host(keys(rng, B, Hkv, n_seg, D))
        self.v[:, :, :n_seg] = host(rng.standard_normal((B, Hkv, n_seg, D)))
        idx = np.full((B, Hkv, blocks, topk), -1, dtype=np.int32)
        for at in np.ndindex(B, Hkv, blocks):
            n = min(topk, nc)
            idx[at][:n] = np.sort(rng.permutation(nc)[:n])
            if routes == "holes":
                idx[at][rng.permutation(topk)[:topk // 2]] = -1
            if routes == "none":
                idx[at] = -1
            if routes == "twice" and n > 1:
                idx[at][1] = idx[at][0]
        self.idx_host, self.idx = idx, torch.from_numpy(idx).cuda()
        self.out = torch.full((B, Hq, rows, D), 7.0, device="cuda", dtype=BF16)
        self.lse = torch.full((B, Hq, rows), 7.0, device="cuda")
        self.p = hga.Params(B, Hq, Hkv, D, topk, rows, nc, seg_head_stride=self.stride, q_block=64 if rows > 1 else 1)

    def run(self, stream=None, out=None, lse=None):
        import hierarchical_sparse_long_b200 as hga
        out, lse = self.out if out is None else out, self.lse if lse is None else lse
        hist = self.hist if self.shape[5] else None
        if self.rows > 1:
            hga.hga_attn_fwd_packed(self.p, self.q, hist, self.cap, self.k, self.v, self.idx, out, lse, stream)
        else:
            hga.hga_attn_decode_packed(self.p, self.q, hist, self.cap, self.k, self.v, self.n_seg, self.idx, out, lse,
                                       stream)
        return out, lse

    def check(self, blocks=None):
        B, Hq, Hkv, D, topk, nc = self.shape
        G, R = Hq // Hkv, 64 if self.rows > 1 else 1
        q, k, v, out, lse = (f64(t) for t in (self.q, self.k, self.v, self.out, self.lse))
        for b, g, blk in np.ndindex(B, Hkv, self.blocks):
            sl = (b, slice(g * G, (g + 1) * G), slice(blk * R, (blk + 1) * R))
            if blocks is not None and blk not in blocks:
                assert np.all(out[sl] == 7.0) and np.all(lse[sl] == 7.0)
                continue
            sel = [j for j in self.idx_host[b, g, blk] if 0 <= j < nc]
            pick = [slice(64 * j, 64 * j + 64) for j in sel]
            n = (blk + 1) * 64 if R > 1 else self.n_seg
            kk = np.concatenate([self.kh[b, g, s] for s in pick] + [k[b, g, :n]])
            vv = np.concatenate([self.vh[b, g, s] for s in pick] + [v[b, g, :n]])
            mask = np.ones((R, len(kk)), dtype=bool)
            if R > 1:
                mask[:, -64:] = np.tril(np.ones((64, 64), dtype=bool))
            o, l, mag, size = ref.attend(q[sl].reshape(G * R, D), kk, vv, np.tile(mask, (G, 1)))
            tol, ltol = ref.attend_tol(o, mag, size, D, len(kk))
            err = abs(out[sl].reshape(G * R, D) - o)
            assert np.all(err <= tol), f"out {b, g, blk}: {err.max():.3e}, {np.max(err / tol):.2f} of its bound"
            err = abs(lse[sl].reshape(-1) - l)
            assert np.all(err <= ltol + 2.0 ** -22 * abs(l)), f"lse {b, g, blk}: {err.max():.3e}"


# (B, Hq, Hkv, D, topk, nc, window, routes)
DECODE = [
    (1, 1, 1, 64, 1, 0, 1, "random"),
    (1, 1, 1, 128, 1, 1, 1, "random"),
    (1, 32, 8, 128, 16, 24, 37, "random"),
    (2, 8, 2, 128, 8, 5, 16, "random"),      # routes padded with -1
    (3, 5, 1, 64, 7, 9, 17, "holes"),
    (2, 16, 2, 64, 40, 60, 130, "holes"),
    (1, 7, 1, 128, 64, 70, 64, "random"),
    (1, 6, 3, 128, 5, 9, 15, "none"),
    (2, 4, 4, 64, 6, 9, 33, "twice"),        # a chunk named twice counts twice, as in hga_attn_decode
    (40, 16, 8, 128, 3, 4, 300, "random"),   # more (batch, KV head) pairs than SMs
    (5, 12, 3, 128, 21, 33, 1, "holes"),
    (1, 8, 1, 128, 64, 64, 2000, "random"),
]


@pytest.mark.parametrize("case", DECODE, ids=str)
def test_decode(case):
    c = Packed(*case[:7], 1, routes=case[7])
    c.run()
    c.check()


# (B, Hq, Hkv, D, topk, nc, blocks, routes)
FWD = [
    (1, 1, 1, 128, 1, 0, 2, "random"),
    (1, 4, 1, 128, 1, 1, 2, "random"),
    (1, 32, 8, 128, 16, 24, 3, "random"),
    (2, 8, 2, 128, 8, 5, 2, "random"),
    (1, 6, 2, 128, 5, 9, 4, "holes"),     # three heads per KV head: one per CTA
    (1, 4, 2, 128, 3, 9, 5, "holes"),     # two
    (2, 8, 1, 128, 7, 12, 2, "random"),   # eight: two CTAs of four
    (1, 4, 1, 128, 64, 70, 2, "random"),
    (1, 8, 2, 128, 6, 9, 3, "none"),
    (1, 4, 1, 128, 6, 9, 2, "twice"),
    (1, 1, 1, 64, 1, 1, 1, "random"),
    (2, 8, 2, 64, 9, 14, 3, "holes"),
    (1, 6, 3, 64, 5, 9, 4, "random"),
    (1, 5, 1, 64, 4, 3, 2, "random"),
    (1, 16, 2, 64, 3, 0, 2, "random"),
]


@pytest.mark.parametrize("case", FWD, ids=str)
def test_forward(case):
    B, Hq, Hkv, D, topk, nc, blocks, routes = case
    c = Packed(B, Hq, Hkv, D, topk, nc, 64 * blocks, blocks, routes=routes)
    c.run()
    c.check()


# Above two CTAs an SM the blocks run in another order, the shortest first on some SMs; CTAs follow
# one another on an SM, and its TMEM is released and taken again.
@pytest.mark.parametrize("case,blocks", [
    ((2, 32, 8, 128, 3, 9, 20, "random"), None),      # 320 CTAs of two halves
    ((3, 16, 8, 64, 2, 5, 15, "holes"), None),        # 360 of one
    ((2, 12, 4, 128, 2, 5, 18, "random"), (2, 17)),   # 360, one head each; the first and the last blocks stay
    ((2, 32, 8, 64, 2, 0, 21, "random"), (0, 19)),    # 304 of two halves, no history
], ids=str)
def test_forward_of_many_blocks(case, blocks):
    B, Hq, Hkv, D, topk, nc, n, routes = case
    G = Hq // Hkv
    c = Packed(B, Hq, Hkv, D, topk, nc, 64 * n, n, routes=routes)
    if blocks:
        c.p.qblock_begin, c.p.qblock_end = blocks
    grid = (blocks[1] - blocks[0] if blocks else n) * B * Hkv * (1 if G % 2 == 0 else G)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert grid >= 2 * sms and grid % sms
    c.run()
    c.check(blocks=range(*blocks) if blocks else None)
    first = c.out.clone(), c.lse.clone()
    for _ in range(3):  # one behind the other: the next call's CTAs wait beside this one's last
        c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])


def test_forward_of_a_block_range():
    c = Packed(1, 8, 2, 128, 4, 9, 320, 5)
    c.p.qblock_begin, c.p.qblock_end = 1, 3
    c.run()
    c.check(blocks=(1, 2))


def test_large_scores():
    """Scores of some hundreds in either direction: the running maximum has to move."""
    for rows in (1, 3):
        c = Packed(1, 8, 2, 128, 12, 20, 64 * rows if rows > 1 else 70, rows, seed=4)
        c.q *= 40
        c.run()
        c.check()


@pytest.mark.parametrize("blocks", [1, 2])
def test_non_finite_chunks_reach_only_their_rows(blocks):
    """A chunk that holds a NaN key makes the rows that route to it NaN, and no others."""
    import hierarchical_sparse_long_b200 as hga
    c = Packed(1, 8, 2, 128, 3, 9, 128 if blocks == 2 else 20, blocks, seed=2)
    bad = int(c.idx_host[0, 0, 0, 0])
    k = torch.full((1, 1, 64, 128), 1.0, device="cuda", dtype=BF16)
    k[0, 0, 5, 7] = float("nan")
    one = torch.zeros(1, 1, 1, 72 * 128, device="cuda", dtype=torch.uint8)
    hga.hga_pack_history(k, k, 64, 1, 1, 128, 0, 1, one, 1)
    c.hist[0, 0, bad] = one[0, 0, 0]
    out, _ = c.run()
    for g, blk in np.ndindex(2, blocks):
        rows = out[0, 4 * g:4 * g + 4, blk * 64:(blk + 1) * 64] if blocks > 1 else out[0, 4 * g:4 * g + 4]
        hit = g == 0 and bad in c.idx_host[0, g, blk]
        assert torch.all(torch.isnan(rows)) if hit else torch.all(torch.isfinite(rows))


def test_bad_routes_are_skipped_and_flagged():
    import hierarchical_sparse_long_b200 as hga
    for rows, n in ((1, 30), (2, 128)):
        c = Packed(1, 8, 2, 128, 6, 9, n, rows, seed=1)
        c.run()
        c.check()
        assert hga.hga_get_device_status() == 0
        c.idx_host[0, 1, 0, 2], c.idx_host[0, 0, 0, 4] = 9, -5
        c.idx.copy_(torch.from_numpy(c.idx_host))
        c.run()
        c.check()
        assert hga.hga_get_device_status() == hga.HGA_DEV_BAD_INDEX


def test_offsets_beyond_32_bits():
    """The last of 250,000 chunks of the second KV head lies 4.6 GB into the history."""
    import hierarchical_sparse_long_b200 as hga
    rng = np.random.default_rng(11)
    cap, n = 250000, 6
    hist = torch.empty(1, 2, cap, 72 * 128, device="cuda", dtype=torch.uint8)
    kh, vh = host(keys(rng, 1, 2, n * 64, 128)), host(rng.standard_normal((1, 2, n * 64, 128)))
    for rows, win in ((1, 10), (2, 128)):
        c = Packed(1, 8, 2, 128, n, n, win, rows)
        hga.hga_pack_history(kh, vh, n * 64, 1, 2, 128, cap - n, n, hist, cap)
        _, c.kh, c.vh = ref.pack(f64(kh), f64(vh))
        small = c.idx_host.copy()
        c.hist, c.cap, c.p.n_hist_chunks = hist, cap, cap
        c.idx = torch.from_numpy(np.where(small >= 0, small + cap - n, -1)).cuda().to(torch.int32)
        c.run()
        c.check()
    k2, v2 = torch.empty_like(kh), torch.empty_like(vh)
    hga.hga_unpack_history(hist, cap, 1, 2, 128, cap - n, n, k2, v2, n * 64)
    assert np.array_equal(f64(k2), c.kh) and np.array_equal(f64(v2), c.vh)


def test_repeated_graph_and_two_streams():
    """Equal inputs give equal bits: again, replayed from a graph on another stream, and with a
    second call under way."""
    for rows, n, batch in ((1, 100, 3), (4, 256, 1)):
        c, other = Packed(batch, 16, 4, 128, 9, 20, n, rows), Packed(batch, 8, 2, 128, 7, 20, n, rows, seed=3)
        out, lse = (t.clone() for t in c.run())
        other.run()
        other.check()
        want = other.out.clone()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            c.run()
        side = torch.cuda.Stream()
        for _ in range(3):
            c.out.fill_(7.0)
            other.out.fill_(7.0)
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                other.run()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(c.out, out) and torch.equal(c.lse, lse) and torch.equal(other.out, want)
        del graph


# ------------------------------------------------------------------ together
def test_projection_to_packed_attention():
    """The operators as a layer uses them: projections normed, rotated and laid out; closed
    chunks detached into the packed history with their summaries; the next segment and then
    single tokens routed over those and attended; the segment's gradients taken back to the
    projections.  Every step is compared with its formula on that step's own inputs."""
    import hierarchical_sparse_long_b200 as hga
    B, Hq, Hkv, D, S, topk = 1, 8, 2, 128, 256, 3
    rng = np.random.default_rng(21)
    row = (Hq + 2 * Hkv) * D
    table = torch.empty(1024, D, device="cuda")
    hga.hga_rope_table(1e6, D, 1024, table)
    wq, wk = host(1 + 0.1 * rng.standard_normal(D)), host(1 + 0.1 * rng.standard_normal(D))

    def project(first, n, k, v):
        x = host(rng.standard_normal((B, n, row)))
        q = torch.empty(B, Hq, n, D, device="cuda", dtype=BF16)
        p = hga.ProjParams(B, Hq, Hkv, D, n, D, kv_head_stride=S, first_pos=first)
        hga.hga_qk_norm_rope(p, x, x[..., Hq * D:], x[..., (Hq + Hkv) * D:], wq, wk, table, None, q, k, v)
        cs = ref.rope_table(1e6, D, 1024)[first:first + n].astype(np.float64)[None, None]
        heads = f64(x).reshape(B, n, -1, D).swapaxes(1, 2)
        y, mag = ref.norm_rope(heads[:, :Hq], f64(wq), cs, D, 1e-6)
        assert np.all(abs(f64(q) - y) <= ref.HALF["bf16"] * abs(y) + 32 * ref.U32 * mag)
        return p, x, q

    kw = torch.empty(B, Hkv, S, D, device="cuda", dtype=BF16)
    vw = torch.empty_like(kw)
    nc = S // 64
    cap = 3 * nc
    hist = torch.zeros(B, Hkv, cap, hga.hga_packed_chunk_bytes(D), device="cuda", dtype=torch.uint8)
    summ = torch.zeros(B, Hkv, cap, D, device="cuda")
    project(0, S, kw, vw)
    hga.hga_pack_history(kw, vw, S, B, Hkv, D, 0, nc, hist, cap, summ, cap)
    _, kh, vh = ref.pack(f64(kw), f64(vw))

    # the next segment
    p, x, q = project(S, S, kw, vw)
    c = Packed(B, Hq, Hkv, D, topk, nc, S, nc, stride_extra=0)
    c.hist, c.cap, c.kh, c.vh, c.q, c.k, c.v = hist, cap, kh, vh, q, kw, vw
    hga.hga_route(c.p, q, summ, cap, c.idx)
    c.idx_host = c.idx.cpu().numpy()
    assert np.all(c.idx_host >= 0)
    out, lse = c.run()
    c.check()

    # its gradients: the backward over the unpacked values of the same chunks
    k2, v2 = torch.empty(B, Hkv, nc * 64, D, device="cuda", dtype=BF16), torch.empty_like(kw)
    hga.hga_unpack_history(hist, cap, B, Hkv, D, 0, nc, k2, v2, nc * 64)
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    hga.hga_attn_fwd(c.p, q, k2, v2, kw, vw, c.idx, out2, lse2)
    hc.compare(hc.f32(out), hc.f32(out2), "bf16", "forward over the unpacked values")
    dout = host(rng.standard_normal((B, Hq, S, D)))
    dq = torch.empty(B, Hq, S, D, device="cuda")
    dk, dv = torch.empty(B, Hkv, S, D, device="cuda"), torch.empty(B, Hkv, S, D, device="cuda")
    ws = torch.empty(hga.hga_attn_bwd_workspace_size(c.p) // 4 + 1, device="cuda")
    hga.hga_attn_bwd(c.p, q, k2, v2, kw, vw, c.idx, out, lse, dout, dq, dk, dv, ws)
    dx = torch.empty_like(x)
    dwq, dwk = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    wsp = torch.empty(hga.hga_qk_norm_rope_workspace_size(p), device="cuda", dtype=torch.uint8)
    hga.hga_qk_norm_rope_bwd(p, x, x[..., Hq * D:], wq, wk, table, None, dq, dk, dv, dx, dx[..., Hq * D:],
                             dx[..., (Hq + Hkv) * D:], dwq, dwk, wsp)
    want = _layer_grad(x, wq, wk, table[S:2 * S], c, dout)
    for got, w, what in ((dx, want[0], "dx"), (dwq, want[1], "dwq"), (dwk, want[2], "dwk")):
        # bf16 q, k, P, dS and dx on the way: a relative error of a few 2^-8 in norm, 8 allowed
        err = np.linalg.norm(f64(got) - w) / np.linalg.norm(w)
        assert err < 8 * ref.HALF["bf16"], f"{what}: {err:.2e}"

    # the segment closes; a token at a time follows
    hga.hga_pack_history(kw, vw, S, B, Hkv, D, nc, nc, hist, cap, summ, cap)
    _, ks, vs = ref.pack(f64(kw), f64(vw))
    kh, vh = np.concatenate([kh, ks], axis=2), np.concatenate([vh, vs], axis=2)
    for t in range(2):
        _, _, q = project(2 * S + t, 1, kw[:, :, t:], vw[:, :, t:])
        c = Packed(B, Hq, Hkv, D, topk, 2 * nc, t + 1, 1, stride_extra=S - t - 1)
        c.rows = 1
        c.hist, c.cap, c.kh, c.vh, c.q, c.k, c.v = hist, cap, kh, vh, q, kw, vw
        hga.hga_route(c.p, q, summ, cap, c.idx)
        c.idx_host = c.idx.cpu().numpy()
        c.run()
        c.check()


def _layer_grad(x, wq, wk, cs, c, dout):
    """Gradients of sum(dout * out) of the segment by torch's differentiation in 64 bits."""
    B, Hq, Hkv, D, topk, nc = c.shape
    x, wq, wk = (t.detach().double().requires_grad_() for t in (x, wq, wk))
    S, G, h = x.shape[1], Hq // Hkv, D // 2
    cos, sin = cs.double()[:, :h], cs.double()[:, h:]

    def rot(y, w):
        n = y * (y.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w
        return torch.cat([n[..., :h] * cos - n[..., h:] * sin, n[..., h:] * cos + n[..., :h] * sin], dim=-1)

    heads = x.view(B, S, Hq + 2 * Hkv, D).transpose(1, 2)
    q, k, v = rot(heads[:, :Hq], wq), rot(heads[:, Hq:Hq + Hkv], wk), heads[:, Hq + Hkv:]
    kh, vh = torch.from_numpy(c.kh).cuda(), torch.from_numpy(c.vh).cuda()
    loss = 0.0
    for g, blk in np.ndindex(Hkv, S // 64):
        sel = torch.cat([torch.arange(64) + 64 * int(j) for j in c.idx_host[0, g, blk]]).cuda()
        n = 64 * (blk + 1)
        kk, vv = torch.cat([kh[0, g][sel], k[0, g, :n]]), torch.cat([vh[0, g][sel], v[0, g, :n]])
        r = slice(64 * blk, n)
        s = q[0, g * G:(g + 1) * G, r] @ kk.T * D ** -0.5
        s[..., -64:] += torch.full((64, 64), -torch.inf, device="cuda", dtype=torch.float64).triu(1)
        loss = loss + (dout[0, g * G:(g + 1) * G, r].double() * (s.softmax(-1) @ vv)).sum()
    loss.backward()
    return f64(x.grad), f64(wq.grad), f64(wk.grad)


def test_readme_example():
    """The README's code runs as printed."""
    import os
    import re
    import hierarchical_sparse_long_b200 as hga
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    names = {}
    for block in re.findall(r"```python\n(.*?)```", text, flags=re.S):
        exec(block, names)
    torch.cuda.synchronize()
    assert hga.hga_get_device_status() == 0
    assert torch.isfinite(names["out"]).all() and torch.isfinite(names["lse"]).all()
    B, Hkv, nc, D = names["B"], names["Hkv"], names["nc"], names["D"]
    want = torch.empty(B, Hkv, nc, D, device="cuda")
    hga.hga_build_summaries(names["k_all"], names["L"], B, Hkv, D, 64, 0, nc, want, nc)
    assert torch.equal(names["summ"][:, :, :nc], want)


@pytest.mark.parametrize("mode", ["stream", "graph"])
def test_calls_behind_one_another(mode):
    """Each kernel takes its place while the previous one drains.  A run of calls in which each
    reads what the one before wrote, and writes what the one before read, gives the bits of the
    same run with the device idle between any two calls."""
    import hierarchical_sparse_long_b200 as hga
    B, Hq, Hkv, D, topk, steps = 2, 12, 3, 128, 3, 4
    rng = np.random.default_rng(31)
    row = (Hq + 2 * Hkv) * D
    x = host(rng.standard_normal((steps, B, 64, row)))
    w = host(1 + 0.1 * rng.standard_normal(D))
    table = torch.empty(512, D, device="cuda")
    hga.hga_rope_table(1e6, D, 512, table)
    dq, dk, dv = (host(rng.standard_normal((B, h, 64, D)), torch.float32) for h in (Hq, Hkv, Hkv))
    buf = lambda *s, t=BF16: torch.zeros(*s, device="cuda", dtype=t)
    q, k, v = buf(B, Hq, 64, D), buf(B, Hkv, 64, D), buf(B, Hkv, 64, D)
    hist = buf(B, Hkv, steps, 72 * D, t=torch.uint8)
    summ, idx = buf(B, Hkv, steps, D, t=torch.float32), buf(B, Hkv, 1, topk, t=torch.int32)
    out, lse = buf(B, Hq, 64, D), buf(B, Hq, 64, t=torch.float32)
    one, lse1 = buf(B, Hq, 1, D), buf(B, Hq, 1, t=torch.float32)
    q1, k2, v2 = buf(B, Hq, 1, D), buf(B, Hkv, 64, D), buf(B, Hkv, 64, D)
    dx, dw = buf(B, 64, row), buf(2, D, t=torch.float32)
    p = hga.ProjParams(B, Hq, Hkv, D, 64, D)
    ws = buf(hga.hga_qk_norm_rope_workspace_size(p), t=torch.uint8)
    seen = buf(steps, B, Hq, 64, D), buf(steps, B, Hq, 1, D), buf(steps, B, 64, row), buf(steps, 2, D, t=torch.float32)

    def run(idle):
        for i in range(steps):
            a = x[i]
            f = hga.Params(B, Hq, Hkv, D, topk, 64, i)
            d = hga.Params(B, Hq, Hkv, D, topk, 1, i + 1, seg_head_stride=64, q_block=1)
            for call in (
                    lambda: hga.hga_qk_norm_rope(p, a, a[..., Hq * D:], a[..., (Hq + Hkv) * D:], w, w, table, None, q,
                                                 k, v),
                    lambda: hga.hga_route(f, q, summ, steps, idx),
                    lambda: hga.hga_attn_fwd_packed(f, q, hist, steps, k, v, idx, out, lse),
                    lambda: hga.hga_pack_history(k, v, 64, B, Hkv, D, i, 1, hist, steps, summ, steps),
                    lambda: hga.hga_unpack_history(hist, steps, B, Hkv, D, i, 1, k2, v2, 64),
                    lambda: q1.copy_(out[:, :, 63:]),
                    lambda: hga.hga_route(d, q1, summ, steps, idx),
                    lambda: hga.hga_attn_decode_packed(d, q1, hist, steps, k2, v2, 33, idx, one, lse1),
                    lambda: hga.hga_qk_norm_rope_bwd(p, a, a[..., Hq * D:], w, w, table, None, dq, dk, dv, dx,
                                                     dx[..., Hq * D:], dx[..., (Hq + Hkv) * D:], dw[0], dw[1], ws),
                    lambda: dq.copy_(q),
                    lambda: [s[i].copy_(t) for s, t in zip(seen, (out, one, dx, dw))]):
                call()
                if idle:
                    torch.cuda.synchronize()

    start = dq.clone()
    run(True)
    want = [s.clone() for s in seen]
    assert all(torch.isfinite(t).all() for t in want)
    graph = torch.cuda.CUDAGraph()
    if mode == "graph":
        with torch.cuda.graph(graph):
            run(False)
    for _ in range(5):
        dq.copy_(start)
        for t in (q, k, v, hist, summ, idx, out, one, q1, k2, v2, dx, dw, *seen):
            t.zero_()
        graph.replay() if mode == "graph" else run(False)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(seen, want))
    del graph


@pytest.mark.parametrize("mode", ["stream", "graph"])
def test_calls_behind_another_streams_event(mode):
    """A call behind an event reads what the event's stream wrote just before it, and a call of that
    stream behind an event of this one writes only what this one has read: projection on one
    stream, records, their values and decode on the other, into the same buffers again and again."""
    import hierarchical_sparse_long_b200 as hga
    B, Hq, Hkv, D, steps, n = 2, 8, 2, 128, 6, 256
    rng = np.random.default_rng(41)
    row = (Hq + 2 * Hkv) * D
    x = host(rng.standard_normal((steps, B, n, row)))
    w = host(1 + 0.1 * rng.standard_normal(D))
    table = torch.empty(n, D, device="cuda")
    hga.hga_rope_table(1e6, D, n, table)
    buf = lambda *s, t=BF16: torch.zeros(*s, device="cuda", dtype=t)
    q, k, v = buf(B, Hq, n, D), buf(B, Hkv, n, D), buf(B, Hkv, n, D)
    k2, v2, hist = buf(steps, B, Hkv, n, D), buf(steps, B, Hkv, n, D), buf(B, Hkv, n // 64, 72 * D, t=torch.uint8)
    q1, idx = buf(B, Hq, 1, D) + 1, torch.arange(n // 64, device="cuda", dtype=torch.int32).expand(B, Hkv, 1, -1).contiguous()
    out, lse = buf(steps, B, Hq, 1, D), buf(steps, B, Hq, 1, t=torch.float32)
    p = hga.ProjParams(B, Hq, Hkv, D, n, D)
    d = hga.Params(B, Hq, Hkv, D, n // 64, 1, n // 64, seg_head_stride=n, q_block=1)
    side = torch.cuda.Stream()

    def run(idle):
        main = torch.cuda.current_stream()
        for i in range(steps):
            side.wait_stream(main)
            a = x[i]
            hga.hga_qk_norm_rope(p, a, a[..., Hq * D:], a[..., (Hq + Hkv) * D:], w, w, table, None, q, k, v, side)
            main.wait_stream(side)
            if idle:
                torch.cuda.synchronize()
            hga.hga_pack_history(k, v, n, B, Hkv, D, 0, n // 64, hist, n // 64)
            hga.hga_unpack_history(hist, n // 64, B, Hkv, D, 0, n // 64, k2[i], v2[i], n)
            hga.hga_attn_decode_packed(d, q1, hist, n // 64, k, v, n, idx, out[i], lse[i])
            if idle:
                torch.cuda.synchronize()

    run(True)
    want = [t.clone() for t in (k2, v2, out, lse)]
    assert all(torch.isfinite(t).all() for t in want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    if mode == "graph":
        with torch.cuda.graph(graph):
            run(False)
    for _ in range(10):
        for t in (q, k, v, k2, v2, hist, out, lse):
            t.zero_()
        graph.replay() if mode == "graph" else run(False)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((k2, v2, out, lse), want))
    del graph
