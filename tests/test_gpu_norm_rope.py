"""GPU parity of hga_qk_norm_rope and its backward against the formulas in 64 bits.

Tolerances count roundings, u = 2^-24 being half a step of fp32.  Forward: the mean square
is a sum of positive terms of at most 2 * 8 products and 4 lane sums with a scaling and the
eps added (22 u, half of it in r), rsqrtf is within 2 ulp (4 u), two products make n (2 u)
and the rotation is two products and a sum (2 u): below 24 u of the magnitudes of the
output's two products, then half a step of the output type.  Backward: dn is two products
and a sum (2 u), g and xh with r's 15 u and a product each, their mean a sum of at most 22 u
and the difference and scaling 3 u more: below 64 u of the magnitudes.  A weight gradient's
term carries 20 u and runs through the sums of one thread (4 heads for each of its tokens)
and of the CTA (at most 32); the rest is summed in 64 bits.
"""
import numpy as np
import pytest
import torch

from tests import hga_cases as hc
from tests import packed_ref as ref

pytestmark = pytest.mark.gpu

# (B, S, Hq, Hkv, D, R, dtype, positions): positions "first" (a null table of positions),
# "far" (given, up to 131,071), "pad" (ragged: -1 behind each sequence's end)
CASES = [
    (1, 1, 1, 1, 64, 64, "bf16", "first"),
    (16, 1, 32, 8, 128, 128, "bf16", "far"),
    (1, 1, 5, 1, 128, 128, "fp32", "far"),
    (2, 67, 8, 2, 128, 128, "bf16", "pad"),
    (3, 130, 6, 3, 64, 32, "fp32", "pad"),
    (1, 333, 7, 5, 128, 64, "bf16", "first"),
    (1, 65, 4, 4, 64, 16, "bf16", "far"),
    (2, 33, 3, 2, 128, 112, "fp32", "pad"),
    (1, 29, 9, 2, 128, 0, "bf16", "first"),
    (1, 700, 32, 8, 128, 128, "bf16", "pad"),
    (1, 40, 4, 1, 64, 0, "fp32", "pad"),
]
EPS = 1e-6
THETA = 1e6


@pytest.fixture(scope="module", autouse=True)
def _built():
    hc.ensure_built()
    assert torch.cuda.is_available()
    yield
    import hierarchical_sparse_long_b200 as hga
    assert hga.hga_get_device_status() == 0


class Case:
    """Inputs of one case: separate projections with padded rows, a window that the new rows end."""

    def __init__(self, B, S, Hq, Hkv, D, R, dtype, kind, seed=0, scale=1.0):
        import hierarchical_sparse_long_b200 as hga
        self.shape = (B, S, Hq, Hkv, D, R)
        rng = np.random.default_rng(1000 * S + 10 * Hq + D + R + seed)
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.dt, self.dtype = dt, dtype
        dev = lambda a, t=dt: torch.from_numpy(np.asarray(a, dtype=np.float32)).cuda().to(t)
        vec = 8
        self.strides = [Hq * D + vec, Hkv * D + 2 * vec, Hkv * D]
        self.x = [dev(scale * rng.standard_normal((B * S, st))) for st in self.strides]
        self.w = [dev(1 + 0.3 * rng.standard_normal(D)) for _ in range(2)]
        self.n_pos = 131072 if kind == "far" else S + 19
        self.first = 11 if kind == "first" else 0
        self.positions = None
        pos = self.first + np.arange(S)[None].repeat(B, 0)
        if kind == "far":
            pos = 131071 - np.arange(B * S).reshape(B, S) * 7
        if kind == "pad":
            n = rng.integers(1, S + 1, (B, 1))
            pos = np.where(np.arange(S)[None] < n, np.arange(S)[None] + 5, -1)
            pos[:, S // 3] = -1  # and a hole inside
        if kind != "first":
            self.positions = torch.from_numpy(pos.astype(np.int32)).cuda()
        self.pos = pos
        self.table = torch.from_numpy(ref.rope_table(THETA, R, self.n_pos)).cuda() if R else None
        self.window = S + 3
        self.q = torch.full((B, Hq, S, D), 7.0, device="cuda", dtype=dt)
        self.k = torch.full((B, Hkv, self.window, D), 7.0, device="cuda", dtype=dt)
        self.v = torch.full((B, Hkv, self.window, D), 7.0, device="cuda", dtype=dt)
        self.d = [torch.from_numpy(rng.standard_normal((B, h, S, D)).astype(np.float32)).cuda()
                  for h in (Hq, Hkv, Hkv)]
        self.p = hga.ProjParams(B, Hq, Hkv, D, S, R, hga.HGA_BF16 if dtype == "bf16" else hga.HGA_FP32, EPS,
                                *self.strides, kv_head_stride=self.window, first_pos=self.first)

    def fwd(self):
        import hierarchical_sparse_long_b200 as hga
        hga.hga_qk_norm_rope(self.p, *self.x, *self.w, self.table, self.positions, self.q, self.k[:, :, 3:],
                             self.v[:, :, 3:])
        return self.q, self.k, self.v

    def bwd(self):
        import hierarchical_sparse_long_b200 as hga
        dx = [torch.full_like(x, 7.0) for x in self.x]
        dw = [torch.full((self.shape[4],), 7.0, device="cuda") for _ in range(2)]
        ws = torch.full((hga.hga_qk_norm_rope_workspace_size(self.p) // 4,), float("nan"), device="cuda")
        hga.hga_qk_norm_rope_bwd(self.p, self.x[0], self.x[1], *self.w, self.table, self.positions, *self.d, *dx,
                                 *dw, ws)
        return dx, dw

    def heads(self, i):
        """Projection i as head rows [B][H][S][D] in float64."""
        B, S, Hq, Hkv, D, _ = self.shape
        h = Hq if i == 0 else Hkv
        return self.x[i][:, :h * D].double().cpu().numpy().reshape(B, S, h, D).swapaxes(1, 2)

    def cs(self):
        R = self.shape[5]
        if R == 0:
            return np.zeros((*self.pos.shape, 0))[:, None]
        return self.table.double().cpu().numpy()[np.maximum(self.pos, 0)][:, None]

    def weight(self, i):
        return self.w[i].double().cpu().numpy()


def within(got, want, tol, what):
    err = np.abs(np.asarray(got, dtype=np.float64) - want)
    assert np.all(err <= tol), f"{what}: error {err.max():.3e}, {np.max(err / np.maximum(tol, 1e-300)):.2f} of its bound"


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    c = Case(*case)
    q, k, v = (t.double().cpu().numpy() for t in c.fwd())
    live = np.broadcast_to((c.pos >= 0)[:, None, :, None], q.shape)
    kl = (c.pos >= 0)[:, None, :, None]
    for got, i in ((q, 0), (k[:, :, 3:], 1)):
        y, mag = ref.norm_rope(c.heads(i), c.weight(i), c.cs(), c.shape[5], EPS)
        y = np.where(kl, y, 7.0)
        within(got, y, ref.HALF[c.dtype] * abs(y) + 24 * ref.U32 * mag, "qk"[i])
    assert np.array_equal(v[:, :, 3:], np.where(kl, c.heads(2), 7.0))
    # rows before the appended ones keep what they held
    assert np.all(k[:, :, :3] == 7.0) and np.all(v[:, :, :3] == 7.0)
    assert live.shape == q.shape


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    B, S, Hq, Hkv, D, R = case[:6]
    c = Case(*case)
    dx, dw = c.bwd()
    live = (c.pos >= 0)[:, None, :, None]
    steps = -(-B * S // 8)  # a thread's tokens are fewer: at least 8 at once
    for i in range(2):
        dy = c.d[i].double().cpu().numpy() * live
        want, mag, row, rmag = ref.norm_rope_bwd(c.heads(i), c.weight(i), c.cs(), R, EPS, dy)
        h = (Hq, Hkv)[i]
        got = dx[i][:, :h * D].double().cpu().numpy().reshape(B, S, h, D).swapaxes(1, 2)
        within(got, want, ref.HALF[c.dtype] * abs(want) + 64 * ref.U32 * mag, f"d{'qk'[i]}")
        assert torch.all(dx[i][:, h * D:] == 7.0)  # the rows' gaps stay
        tot = row.sum(axis=(0, 1, 2))
        tol = ref.U32 * abs(tot) + (20 + 4 * steps + 32) * ref.U32 * rmag.sum(axis=(0, 1, 2))
        within(dw[i].double().cpu().numpy(), tot, tol, f"dw {'qk'[i]}")
    want = c.d[2].double().cpu().numpy() * live
    got = dx[2].double().cpu().numpy().reshape(B, S, Hkv, D).swapaxes(1, 2)
    within(got, want, ref.HALF[c.dtype] * abs(want), "dv")
    dx2, dw2 = c.bwd()  # equal inputs, equal bits
    assert all(torch.equal(a, b) for a, b in zip(dx + dw, dx2 + dw2))


def test_gradient_against_differences():
    """Central differences of sum(dy * y) of the fp32 forward, step 2^-6: the forward's own
    roundings (24 u of values below 8, over 128 outputs) divided by the step stay below 2e-3,
    and the third-order term h^2 / 6 * |f'''| of a normed row below 1e-3."""
    c = Case(1, 2, 2, 1, 64, 32, "fp32", "first")
    dx, dw = c.bwd()
    h = 2.0 ** -6
    rng = np.random.default_rng(5)

    def value():
        q, k, v = c.fwd()
        f = 0.0
        for y, d in ((q, c.d[0]), (k[:, :, 3:], c.d[1]), (v[:, :, 3:], c.d[2])):
            f += float((y.double() * d.double()).sum())
        return f

    for t, g, n in [(c.x[0], dx[0], 128), (c.x[1], dx[1], 64), (c.x[2], dx[2], 64), (c.w[0], dw[0], 64),
                    (c.w[1], dw[1], 64)]:
        for col in rng.integers(0, n, 6):
            at = (1, int(col)) if t.dim() == 2 else (int(col),)
            x0 = float(t[at])
            t[at] = x0 + h
            step_up = float(t[at])
            up = value()
            t[at] = x0 - h
            step_dn = float(t[at])
            dn = value()
            t[at] = x0
            assert abs((up - dn) / (step_up - step_dn) - float(g[at])) < 3e-3


def test_table():
    import hierarchical_sparse_long_b200 as hga
    for rot, n in ((128, 131072), (16, 1000), (64, 1)):
        t = torch.full((n + 1, rot), 7.0, device="cuda")
        hga.hga_rope_table(THETA, rot, n, t[:n])
        want = ref.rope_table(THETA, rot, n).astype(np.float64)
        # angles below 2^17 with a relative error of a few 2^-53 are off by at most 2^-33
        within(t[:n].double().cpu().numpy(), want, 2 * ref.U32 * abs(want) + 2.0 ** -33, "table")
        assert torch.all(t[n:] == 7.0)


def test_positions_outside_the_table_are_flagged_and_skipped():
    import hierarchical_sparse_long_b200 as hga
    c = Case(1, 9, 4, 2, 64, 64, "bf16", "pad")
    good = torch.arange(9, dtype=torch.int32, device="cuda")[None].contiguous()
    c.positions = good.clone()
    c.positions[0, 3] = c.n_pos
    c.positions[0, 5] = -2
    assert hga.hga_get_device_status() == 0
    q, k, v = (t.clone() for t in c.fwd())
    assert hga.hga_get_device_status() == hga.HGA_DEV_BAD_INDEX
    dx, _ = c.bwd()
    assert hga.hga_get_device_status() == hga.HGA_DEV_BAD_INDEX
    for t, off in ((q, 0), (k, 3), (v, 3)):
        for i in (3, 5):
            assert torch.all(t[:, :, off + i] == 7.0)
        assert not torch.any(t[:, :, off] == 7.0)
    assert all(torch.all(d[[3, 5], :128] == 0) for d in dx)


def test_zero_and_extreme_rows():
    c = Case(1, 4, 2, 1, 128, 128, "fp32", "first")
    c.x[0][0] = 0.0      # r = 1 / sqrt(eps): the row stays zero
    c.x[0][1] = 1e-20    # its square underflows: n = x w / sqrt(eps)
    c.x[0][2, :128] = float("nan")
    q, _, _ = c.fwd()
    dx, dw = c.bwd()
    assert torch.all(q[:, :, 0] == 0) and torch.all(torch.isfinite(dx[0][0]))
    y, mag = ref.norm_rope(c.heads(0)[:, :, 1:2], c.weight(0), c.cs()[:, :, 1:2], 128, EPS)
    within(q[:, :, 1:2].double().cpu().numpy(), y, 26 * ref.U32 * mag, "tiny row")
    # a NaN stays in its own head row
    assert torch.all(torch.isnan(q[:, 0, 2])) and torch.all(torch.isfinite(q[:, 1, 2]))
    assert torch.all(torch.isfinite(q[:, :, 3]))


def test_other_stream_and_graph():
    import hierarchical_sparse_long_b200 as hga
    c = Case(2, 50, 8, 2, 128, 128, "bf16", "far")
    want = [t.clone() for t in c.fwd()]
    dx, dw = c.bwd()
    ws = torch.empty(hga.hga_qk_norm_rope_workspace_size(c.p), device="cuda", dtype=torch.uint8)
    dx2 = [torch.full_like(t, 7.0) for t in dx]  # as bwd() fills them: the rows' gaps stay
    dw2 = [torch.zeros_like(t) for t in dw]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.fwd()
        hga.hga_qk_norm_rope_bwd(c.p, c.x[0], c.x[1], *c.w, c.table, c.positions, *c.d, *dx2, *dw2, ws)
    for t in (c.q, c.k, c.v):
        t[:, :, 3:].fill_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.q[:, :, 3:], want[0][:, :, 3:])
    assert torch.equal(c.k[:, :, 3:], want[1][:, :, 3:]) and torch.equal(c.v[:, :, 3:], want[2][:, :, 3:])
    assert all(torch.equal(a, b) for a, b in zip(dx2 + dw2, dx + dw))
