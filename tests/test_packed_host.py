"""Host-side checks of the projection step and of the packed history: the plain references
against their definitions, and every refused argument, on the CPU (a refused call returns
before it touches the device)."""
import ctypes

import numpy as np
import pytest

import hierarchical_sparse_long_b200 as hga
from hierarchical_sparse_long_b200 import binding
from tests import packed_ref as ref

INVALID, UNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def L():
    from hierarchical_sparse_long_b200 import build
    build.build()
    return binding.lib()


FAKE, ODD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)


# ------------------------------------------------------------------ the references
@pytest.mark.parametrize("D", [64, 128])
def test_reference_records_read_back(D):
    """The record's layout, read word by word as the header describes it."""
    rng = np.random.default_rng(D)
    k, v = (ref.to_bf16(rng.standard_normal((1, 1, 64, D))) for _ in range(2))
    rec, kv, vv = ref.pack(k, v)
    r = rec[0, 0, 0]
    assert r.size == 72 * D
    bf = lambda a: float((np.uint32(a) << 16).view(np.float32))
    w, h = r.view(np.uint32), r.view(np.uint16)
    nibble = lambda e: 4 * (e // 2) if e % 2 == 0 else 16 + 4 * (e // 2)
    for t, c in [(0, 0), (63, D - 1), (17, 9), (40, 38), (5, 62)]:
        code = int(w[t * (D // 8) + c // 8]) >> nibble(c % 8) & 15
        s, z = h[16 * D + c], h[17 * D + c]
        assert ref.values(bf(s), bf(z), code) == kv[0, 0, t, c]
        code = int(w[9 * D + c * 8 + t // 8]) >> nibble(t % 8) & 15
        s, z = h[18 * D + 16 * D + c // 64 * 64 + t], h[18 * D + 17 * D + c // 64 * 64 + t]
        assert ref.values(bf(s), bf(z), code) == vv[0, 0, t, c]
    # off by at most half a step, the roundings of z and of the value, and what rounding s lost
    s, z, _ = ref.quant(k.reshape(1, 1, 1, 64, D), 3)
    bound = (0.5 + 15 * 2.0 ** -8) * s + 2.0 ** -8 * abs(z) + 2.0 ** -8 * abs(kv.reshape(1, 1, 1, 64, D))
    assert np.all(abs(k - kv).reshape(1, 1, 1, 64, D) <= bound)


def test_reference_attention_is_softmax():
    rng = np.random.default_rng(0)
    q, k, v = (rng.standard_normal((n, 64)) for n in (3, 11, 11))
    o, lse, _, _ = ref.attend(q, k, v, np.ones((1, 11), dtype=bool))
    e = np.exp(q @ k.T / 8)
    assert np.allclose(o, e @ v / e.sum(1, keepdims=True)) and np.allclose(lse, np.log(e.sum(1)))


# ------------------------------------------------------------------ projection step
def _proj(**kw):
    base = dict(batch=2, n_q_heads=4, n_kv_heads=2, head_dim=128, seq_len=5, rotary_dim=128)
    base.update(kw)
    return hga.ProjParams(**base)


def _fwd(L, p, *, table=FAKE, n_pos=64, positions=FAKE, ptrs=(FAKE,) * 8):
    q, k, v, wq, wk, qo, ko, vo = ptrs
    return L.hga_qk_norm_rope(ctypes.byref(p.c()), q, k, v, wq, wk, table, n_pos, positions, qo, ko, vo, None)


def _bwd(L, p, *, table=FAKE, n_pos=64, positions=FAKE, ptrs=(FAKE,) * 13, ws_bytes=1 << 30):
    q, k, wq, wk, dq, dk, dv, dqi, dki, dvi, dwq, dwk, ws = ptrs
    return L.hga_qk_norm_rope_bwd(ctypes.byref(p.c()), q, k, wq, wk, table, n_pos, positions, dq, dk, dv, dqi, dki,
                                  dvi, dwq, dwk, ws, ws_bytes, None)


BAD_PROJ = [
    (dict(batch=0), INVALID),
    (dict(n_q_heads=0), INVALID),
    (dict(n_kv_heads=-1), INVALID),
    (dict(seq_len=0), INVALID),
    (dict(dtype=2), INVALID),
    (dict(head_dim=96), UNSUPPORTED),
    (dict(rotary_dim=8), INVALID),
    (dict(rotary_dim=144), INVALID),
    (dict(rotary_dim=-16), INVALID),
    (dict(eps=0.0), INVALID),
    (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID),
    (dict(q_token_stride=4 * 128 - 8), INVALID),
    (dict(k_token_stride=2 * 128 + 4), INVALID),  # not a multiple of 16 bytes
    (dict(v_token_stride=0), INVALID),
    (dict(batch=1 << 16, seq_len=1 << 15), UNSUPPORTED),
    (dict(n_q_heads=20000), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD_PROJ, ids=str)
def test_projection_shapes_refused(L, kw, code):
    p = _proj(**kw)
    assert _fwd(L, p) == code and _bwd(L, p) == code
    assert L.hga_qk_norm_rope_workspace_size(ctypes.byref(p.c())) == 0


def test_projection_arguments_refused(L):
    p = _proj()
    assert _fwd(L, _proj(kv_head_stride=4)) == INVALID
    for call, n in ((_fwd, 8), (_bwd, 13)):
        assert call(L, p, table=None) == INVALID
        assert call(L, p, table=ODD) == INVALID
        assert call(L, p, n_pos=0) == INVALID
        # without positions the table has to hold first_pos .. first_pos + S
        assert call(L, _proj(first_pos=60), positions=None) == INVALID
        assert call(L, _proj(first_pos=-1), positions=None) == INVALID
        assert call(L, _proj(first_pos=-1, rotary_dim=0), positions=None) == INVALID
        for i in range(n):
            if call is _bwd and i in (10, 11):  # the weights' gradients are written as single words
                bad = [None]
            else:
                bad = [None, ODD]
            for b in bad:
                assert call(L, p, ptrs=tuple(b if j == i else FAKE for j in range(n))) == INVALID, (call, i)
    need = L.hga_qk_norm_rope_workspace_size(ctypes.byref(p.c()))
    assert need > 0 and _bwd(L, p, ws_bytes=need - 1) == INVALID
    assert L.hga_qk_norm_rope(None, *[FAKE] * 6, 64, *[FAKE] * 4, None) == INVALID


def test_rope_table_refused(L):
    t = lambda theta, rot, n, p=FAKE: L.hga_rope_table(theta, rot, n, p, None)
    for theta in (0.0, -1.0, float("nan"), float("inf")):
        assert t(theta, 64, 4) == INVALID
    for rot in (0, 8, 20, 144):
        assert t(1e4, rot, 4) == INVALID
    assert t(1e4, 64, -1) == INVALID and t(1e4, 64, 1 << 32) == INVALID
    assert t(1e4, 64, 4, None) == INVALID and t(1e4, 64, 4, ODD) == INVALID
    assert t(1e4, 64, 0, None) == 0


# ------------------------------------------------------------------ packed history
def test_record_size(L):
    assert hga.hga_packed_chunk_bytes(64) == 4608 and hga.hga_packed_chunk_bytes(128) == 9216
    assert hga.hga_packed_chunk_bytes(96) == 0


CHUNKS = dict(k=FAKE, v=FAKE, stride=256, batch=2, heads=2, d=128, first=1, n=4, dtype=0, hist=FAKE, cap=5, summ=FAKE,
              scap=5)


def _pack(L, **kw):
    a = {**CHUNKS, **kw}
    return L.hga_pack_history(a["k"], a["v"], a["stride"], a["batch"], a["heads"], a["d"], a["first"], a["n"],
                              a["dtype"], a["hist"], a["cap"], a["summ"], a["scap"], None)


def _unpack(L, **kw):
    a = {**CHUNKS, **kw}
    return L.hga_unpack_history(a["hist"], a["cap"], a["batch"], a["heads"], a["d"], a["first"], a["n"], a["dtype"],
                                a["k"], a["v"], a["stride"], None)


BAD_CHUNKS = [
    (dict(batch=0), INVALID),
    (dict(heads=0), INVALID),
    (dict(d=96), UNSUPPORTED),
    (dict(first=-1), INVALID),
    (dict(n=-1), INVALID),
    (dict(dtype=3), INVALID),
    (dict(cap=4), INVALID),
    (dict(first=0x7FFFFFFF, cap=0x7FFFFFFF), INVALID),  # first + n passes 32 bits
    (dict(stride=255), INVALID),
    (dict(batch=1 << 16, heads=1 << 15), UNSUPPORTED),
    (dict(batch=1 << 10, heads=1 << 10, n=1 << 11, cap=1 << 12, stride=1 << 17, summ=None), UNSUPPORTED),
    (dict(k=None), INVALID),
    (dict(v=ODD), INVALID),
    (dict(hist=None), INVALID),
    (dict(hist=ODD), INVALID),
]


@pytest.mark.parametrize("kw,code", BAD_CHUNKS, ids=str)
def test_pack_and_unpack_refused(L, kw, code):
    assert _pack(L, **kw) == code and _unpack(L, **kw) == code


def test_pack_summaries_refused(L):
    assert _pack(L, scap=4) == INVALID
    assert _pack(L, summ=ODD) == INVALID
    assert _pack(L, n=0, k=None, v=None, hist=None, summ=None) == 0  # nothing to do
    assert _unpack(L, n=0, k=None, v=None, hist=None) == 0


ATTN = dict(batch=1, n_q_heads=4, n_kv_heads=2, head_dim=128, topk=4, seg_len=128, n_hist_chunks=8)


def _attn(L, decode, cap=8, n_local=5, ptrs=(FAKE,) * 7, **kw):
    p = {**ATTN, **(dict(seg_len=1, q_block=1, seg_head_stride=9) if decode else {}), **kw}
    q, hist, k, v, idx, out, lse = ptrs
    c = hga.Params(**p).c()
    if decode:
        return L.hga_attn_decode_packed(ctypes.byref(c), q, hist, cap, k, v, n_local, idx, out, lse, None)
    return L.hga_attn_fwd_packed(ctypes.byref(c), q, hist, cap, k, v, idx, out, lse, None)


@pytest.mark.parametrize("decode", [False, True])
def test_packed_attention_refused(L, decode):
    for kw, code in [(dict(n_q_heads=3), INVALID), (dict(topk=0), INVALID), (dict(topk=65), INVALID),
                     (dict(n_hist_chunks=-1), INVALID), (dict(seg_head_stride=0), INVALID), (dict(dtype=7), INVALID),
                     (dict(head_dim=96), UNSUPPORTED), (dict(chunk=32), UNSUPPORTED), (dict(batch=0), INVALID),
                     (dict(dtype=hga.HGA_FP32), UNSUPPORTED), (dict(n_hist_chunks=9), INVALID)]:
        assert _attn(L, decode, **kw) == code, kw
    for i in range(7):
        for b in [None] + ([ODD] if i in (0, 1, 2, 3, 5) else []):
            assert _attn(L, decode, ptrs=tuple(b if j == i else FAKE for j in range(7))) == INVALID, i
    other = dict(seg_len=64, q_block=64, seg_head_stride=64) if decode else dict(seg_len=1, q_block=1)
    assert _attn(L, decode, **other) == UNSUPPORTED


def test_packed_attention_refused_by_form(L):
    assert _attn(L, True, n_local=0) == INVALID
    assert _attn(L, True, n_local=10) == INVALID            # above the window's stride
    assert _attn(L, True, n_q_heads=18) == UNSUPPORTED      # nine heads per KV head
    assert b"8 query heads" in L.hga_last_error()
    assert _attn(L, True, batch=1 << 15, n_kv_heads=1 << 13, n_q_heads=1 << 13) == UNSUPPORTED
    assert _attn(L, False, seg_len=100) == INVALID
    assert _attn(L, False, qblock_begin=1, qblock_end=3) == INVALID
    assert _attn(L, False, batch=1 << 14, seg_head_stride=1 << 20) == UNSUPPORTED  # rows beyond 32 bits


def test_binding_raises():
    import torch
    t = torch.empty(4096, dtype=torch.uint8)
    p = hga.Params(**{**ATTN, "seg_len": 1, "q_block": 1})
    with pytest.raises(hga.HGAError):  # seven records of a history of eight
        hga.hga_attn_decode_packed(p, t, t, 7, t, t, 1, t, t, t, stream=0)


def test_binding_refuses_mixed_dtypes():
    import torch
    k, hist = torch.empty(64 * 64), torch.empty(4608, dtype=torch.uint8)
    with pytest.raises(hga.HGAError, match="different dtypes"):
        hga.hga_pack_history(k, k.bfloat16(), 64, 1, 1, 64, 0, 1, hist, 1, stream=0)
    with pytest.raises(hga.HGAError, match="different dtypes"):
        hga.hga_unpack_history(hist, 1, 1, 1, 64, 0, 1, k.bfloat16(), k, 64, stream=0)
    with pytest.raises(hga.HGAError, match="unsupported tensor dtype"):
        hga.hga_pack_history(k.half(), k.half(), 64, 1, 1, 64, 0, 1, hist, 1, stream=0)


def test_params_struct_follows_the_fields():
    """Equal fields share one C struct; a changed field is another one."""
    import copy
    import dataclasses
    import pickle
    p = hga.Params(**ATTN)
    struct = lambda q: q.ref()._obj
    assert p.ref() is p.ref() and struct(p).topk == 4 and struct(p).hist_head_stride == 8 * 64
    other, again = copy.copy(p), pickle.loads(pickle.dumps(p))
    p.topk, p.n_hist_chunks = 7, 9
    assert struct(p).topk == 7 and struct(p).hist_head_stride == 9 * 64
    for q in (other, again, copy.deepcopy(other), dataclasses.replace(other)):
        assert q == hga.Params(**ATTN) and struct(q).topk == 4 and struct(q).n_hist_chunks == 8
    setattr(other, "qblock_end", 2)
    assert struct(other).qblock_end == 2 and struct(again).qblock_end == 0
    q = _proj()
    assert struct(q).seq_len == 5
    q.seq_len = 6
    assert struct(q).seq_len == 6 and struct(q).kv_head_stride == 6
    for n in range(1000):  # many shapes: the store of structs stays small
        p.n_hist_chunks = n
        assert struct(p).n_hist_chunks == n
    assert len(hga.Params._refs) <= 256


def test_dependent_kernels_promise_nothing_about_aliasing():
    """A kernel that takes its place before the previous one has ended must not tell the compiler
    that its inputs are constant: loads of const __restrict__ pointers may pass the wait."""
    import os
    from hierarchical_sparse_long_b200 import build
    waiting = 0
    for path in build.sources():
        text = open(path).read()
        if "depend_wait()" in text or "griddepcontrol.wait" in text:
            waiting += 1
            assert "__restrict__" not in text and "__ldg" not in text, os.path.basename(path)
    assert waiting >= 4


def test_binding_refuses_other_types_and_layouts():
    """Every tensor is of the type, and tables and positions of the layout, as which the library
    would read it: anything else gave wrong rows, or rows behind the tensor's end, without an error."""
    import torch
    f32, i32, i64, bf = torch.float32, torch.int32, torch.int64, torch.bfloat16
    B, S, Hq, Hkv, D, R = 2, 5, 4, 2, 64, 32
    p = hga.ProjParams(B, Hq, Hkv, D, S, R)
    row = (Hq + 2 * Hkv) * D
    fwd = dict(q=torch.zeros(B, S, row, dtype=bf), k=torch.zeros(B, S, row, dtype=bf),
               v=torch.zeros(B, S, row, dtype=bf), q_weight=torch.ones(D, dtype=bf), k_weight=torch.ones(D, dtype=bf),
               table=torch.zeros(16, R), positions=torch.zeros(B, S, dtype=i32),
               q_out=torch.zeros(B, Hq, S, D, dtype=bf), k_out=torch.zeros(B, Hkv, S, D, dtype=bf),
               v_out=torch.zeros(B, Hkv, S, D, dtype=bf))
    bwd = dict(q=fwd["q"], k=fwd["k"], q_weight=fwd["q_weight"], k_weight=fwd["k_weight"], table=fwd["table"],
               positions=fwd["positions"], dq=torch.zeros(B, Hq, S, D), dk=torch.zeros(B, Hkv, S, D),
               dv=torch.zeros(B, Hkv, S, D), dq_in=fwd["q"], dk_in=fwd["q"].clone(), dv_in=fwd["q"].clone(),
               dq_weight=torch.zeros(D), dk_weight=torch.zeros(D), workspace=torch.zeros(1 << 20, dtype=torch.uint8))

    def refused(call, args, match, **other):
        with pytest.raises(hga.HGAError, match=match) as e:
            call(*{**args, **other}.values(), stream=0)
        assert e.value.code == INVALID

    for call, args in ((lambda *a, **k: hga.hga_qk_norm_rope(p, *a, **k), fwd),
                       (lambda *a, **k: hga.hga_qk_norm_rope_bwd(p, *a, **k), bwd)):
        for name, t in args.items():
            if name == "workspace":
                continue
            for dt in {f32, bf, i64} - {t.dtype}:
                refused(call, args, f"{name} of {dt}", **{name: t.to(dt)})
        # one row of positions for every sequence, too few, every other one
        for pos in (torch.arange(S, dtype=i32).expand(B, S), torch.zeros(S, dtype=i32),
                    torch.zeros(B, 2 * S, dtype=i32)[:, ::2]):
            refused(call, args, "positions of", positions=pos)
        # rows of another width, cut from wider ones, half a row
        for table in (torch.zeros(16, D), torch.zeros(16, D)[:, :R], torch.zeros(16, R // 2), torch.zeros(R + 1)):
            refused(call, args, "table of", table=table)
    for table in (torch.zeros(7, R), torch.zeros(16, R)[::2], torch.zeros(8, R, dtype=bf)):
        with pytest.raises(hga.HGAError, match="table of"):
            hga.hga_rope_table(1e4, R, 8, table, stream=0)
    k, hist = torch.zeros(64, D, dtype=bf), torch.zeros(72 * D, dtype=torch.uint8)
    with pytest.raises(hga.HGAError, match="summ of torch.bfloat16"):
        hga.hga_pack_history(k, k, 64, 1, 1, D, 0, 1, hist, 1, torch.zeros(D, dtype=bf), 1, stream=0)
    for decode in (False, True):
        n = 1 if decode else 64
        c = hga.Params(1, Hq, Hkv, D, 1, n, 1, q_block=n)
        q, kv = torch.zeros(1, Hq, n, D, dtype=bf), torch.zeros(1, Hkv, n, D, dtype=bf)
        args = dict(q=q, hist=hist, cap=1, k=kv, v=kv.clone(), idx=torch.zeros(1, Hkv, 1, 1, dtype=i32),
                    out=q.clone(), lse=torch.zeros(1, Hq, n))

        def call(q, hist, cap, k, v, idx, out, lse, stream):
            if decode:
                hga.hga_attn_decode_packed(c, q, hist, cap, k, v, 1, idx, out, lse, stream=stream)
            else:
                hga.hga_attn_fwd_packed(c, q, hist, cap, k, v, idx, out, lse, stream=stream)
        for name in ("q", "k", "v", "idx", "out", "lse"):
            for dt in {f32, bf, i64} - {args[name].dtype}:
                refused(call, args, f" of {dt}", **{name: args[name].to(dt)})


def test_params_struct_of_any_number():
    """Fields that are not plain numbers, or lie in another order, give the struct of their values."""
    import torch
    struct = lambda q: q.ref()._obj
    n = torch.tensor(4)
    p = hga.Params(**{**ATTN, "topk": n})
    assert struct(p).topk == 4
    n += 3
    assert struct(p).topk == 7
    assert struct(hga.Params(**{**ATTN, "topk": np.array(5)})).topk == 5
    p = hga.Params(**ATTN)
    p.tag = ["a user's own attribute"]
    assert struct(p).topk == 4
    # topk and seg_len have changed places in the instance, and have each other's usual values
    assert struct(hga.Params(**{**ATTN, "topk": 4, "seg_len": 64})).seg_len == 64
    swapped = hga.Params.__new__(hga.Params)
    names = list(hga.Params(**ATTN).__dict__)
    i, j = names.index("topk"), names.index("seg_len")
    names[i], names[j] = names[j], names[i]
    fields = hga.Params(**{**ATTN, "topk": 64, "seg_len": 4}).__dict__
    for name in names:
        setattr(swapped, name, fields[name])
    assert struct(swapped).topk == 64 and struct(swapped).seg_len == 4


def test_refusals_of_packed_attention_say_why():
    """The library's reason reaches the Python error, and only that call's."""
    import torch
    hist, idx = torch.zeros(72 * 64, dtype=torch.uint8), torch.zeros(1, 1, 1, 1, dtype=torch.int32)

    def call(n, heads, dtype, topk=1):
        p = hga.Params(1, heads, 1, 64, topk, n, 1, q_block=n, dtype=hga.HGA_FP32 if dtype == torch.float32 else hga.HGA_BF16)
        q, kv, lse = torch.zeros(1, heads, n, 64, dtype=dtype), torch.zeros(1, 1, n, 64, dtype=dtype), torch.zeros(1, heads, n)
        with pytest.raises(hga.HGAError) as e:
            if n == 1:
                hga.hga_attn_decode_packed(p, q, hist, 1, kv, kv.clone(), 1, idx, q.clone(), lse, stream=0)
            else:
                hga.hga_attn_fwd_packed(p, q, hist, 1, kv, kv.clone(), idx, q.clone(), lse, stream=0)
        return str(e.value)

    assert "8 query heads" in call(1, 9, torch.bfloat16)
    assert "8 query heads" not in call(1, 1, torch.bfloat16, topk=0)  # another refusal
    assert "bf16 only" in call(64, 1, torch.float32)
    assert "bf16 only" not in call(64, 1, torch.bfloat16, topk=0)
