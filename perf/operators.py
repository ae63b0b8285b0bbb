"""The operators around the packed history, with their plain forms.

``run`` computes one pass of a case: with ``own`` false in elementary torch
operations, with ``own`` true through the package's public calls.  Both take
what ``prepare`` gives.

  qk_norm_rope       projections' rows -> normed, rotated q and k, and v, head-major
  qk_norm_rope_bwd   gradients of the above
  pack_history       closed chunks -> 4-bit records and chunk summaries, and the
                     records' values back
  decode_packed      one new token per sequence over routed 4-bit chunks and its window
  fwd_packed         a segment over routed 4-bit chunks and its causal window

4-bit record of one 64-token chunk of one KV head (72 D bytes):
  K codes   uint32 [64 tokens][D / 8]: word w holds channels 8w .. 8w + 7
  K grid    bf16 s[D], z[D]                  (one pair per channel)
  V codes   uint32 [D channels][8]: word w holds tokens 8w .. 8w + 7
  V grid    bf16 s[D / 64][64], z[D / 64][64] (one pair per token and 64 channels)
Nibble j < 4 of a word is its element 2j, nibble 4 + j its element 2j + 1, and a
code c stands for bf16(s (16 + c) + z), rounded once.
"""
import math

import torch

own = False

CHUNK = 64


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one new token for each of 16 sequences, far into their contexts
        dict(name="norm_rope_token", op="qk_norm_rope", batch=16, seq=1, hq=32, hkv=8, d=128, rot=128,
             dtype="bf16", window=64, pad=False, far=131072),
        # an active segment of the 16K layer
        dict(name="norm_rope_segment", op="qk_norm_rope", batch=1, seq=2048, hq=32, hkv=8, d=128, rot=128,
             dtype="bf16", window=2048, pad=False, far=16384),
        # a padded batch of prompts of odd lengths in fp32, half of each head rotated
        dict(name="norm_rope_ragged_fp32", op="qk_norm_rope", batch=3, seq=257, hq=12, hkv=4, d=64, rot=32,
             dtype="fp32", window=300, pad=True, far=4096),
        # the training step of that 16K segment
        dict(name="norm_rope_bwd_segment", op="qk_norm_rope_bwd", batch=1, seq=2048, hq=32, hkv=8, d=128, rot=128,
             dtype="bf16", window=2048, pad=False, far=16384),
        # a short padded fine-tuning batch in fp32
        dict(name="norm_rope_bwd_ragged_fp32", op="qk_norm_rope_bwd", batch=2, seq=129, hq=6, hkv=2, d=64, rot=64,
             dtype="fp32", window=129, pad=True, far=4096),
        # sixteen sequences each close one chunk while they generate
        dict(name="pack_chunk", op="pack_history", batch=16, chunks=1, hkv=8, d=128, dtype="bf16"),
        # the detached history of a 16K context packed at once
        dict(name="pack_16k", op="pack_history", batch=1, chunks=224, hkv=8, d=128, dtype="bf16"),
        # one sequence generates with a short window
        dict(name="decode_one", op="decode_packed", batch=1, hq=32, hkv=8, d=128, topk=16, nc=224, local=37, holes=0),
        # sixteen sequences at 32K
        dict(name="decode_16", op="decode_packed", batch=16, hq=32, hkv=8, d=128, topk=32, nc=511, local=64, holes=0),
        # many sequences, heads of 64 and an uneven window
        dict(name="decode_d64", op="decode_packed", batch=48, hq=16, hkv=2, d=64, topk=40, nc=200, local=130, holes=3),
        # the last segment of a 16K evaluation
        dict(name="fwd_16k", op="fwd_packed", batch=1, hq=32, hkv=8, d=128, topk=16, nc=224, seq=2048, holes=0),
        # the last segment of a 128K evaluation
        dict(name="fwd_128k", op="fwd_packed", batch=1, hq=32, hkv=8, d=128, topk=32, nc=1984, seq=4096, holes=0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["qk_norm_rope", "qk_norm_rope", "qk_norm_rope_bwd", "pack_history", "decode_packed",
                     "decode_packed", "fwd_packed"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 8])
    d = rng.choice([64, 128])
    if op in ("qk_norm_rope", "qk_norm_rope_bwd"):
        hq = min(32, hkv * group)
        hq -= hq % hkv
        batch = rng.choice([1, 1, 2, 3, 5, 16])
        seq = _log_int(rng, 1, max(1, 2048 // batch))
        return dict(op=op, batch=batch, seq=seq, hq=hq, hkv=hkv, d=d, rot=rng.choice([d, d, d // 2, 16]),
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), window=seq + rng.randrange(0, 70),
                    pad=rng.random() < 0.5 and seq > 1, far=_log_int(rng, seq + 1, 131072))
    if op == "pack_history":
        return dict(op=op, batch=rng.choice([1, 2, 5, 16]), chunks=_log_int(rng, 1, 14), hkv=hkv, d=d,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "decode_packed":
        topk = _log_int(rng, 1, 64)
        return dict(op=op, batch=_log_int(rng, 1, 24), hq=hkv * group, hkv=hkv, d=d, topk=topk,
                    nc=_log_int(rng, 1, 400), local=_log_int(rng, 1, 300), holes=rng.randrange(0, 1 + topk // 4))
    topk = _log_int(rng, 1, 32)
    return dict(op=op, batch=rng.choice([1, 1, 2]), hq=min(32, hkv * group) // hkv * hkv, hkv=hkv, d=128, topk=topk,
                nc=_log_int(rng, 1, 600), seq=64 * _log_int(rng, 1, 24), holes=rng.randrange(0, 1 + topk // 4))


# ---------------------------------------------------------------- inputs
def _dt(case):
    return torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _keys(g, b, h, chunks, d, dtype):
    """N(0, 1) keys with an offset of norm 2 per chunk, [b][h][chunks * 64][d]."""
    off = _randn(g, b, h, chunks, 1, d)
    off = 2 * off / off.norm(dim=-1, keepdim=True)
    return (_randn(g, b, h, chunks, CHUNK, d) + off).reshape(b, h, chunks * CHUNK, d).to(dtype)


def _table(n_pos, rot):
    """cos then sin of pos * 10^(-12 i / rot) (base 10^6), rounded once from 64 bits."""
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    pos = torch.arange(n_pos, device="cuda", dtype=torch.float64)
    ang = pos[:, None] * torch.exp(-math.log(1e6) * 2 * i / rot)[None]
    return torch.cat([ang.cos(), ang.sin()], dim=1).float()


def _positions(case, g):
    b, s, far = case["batch"], case["seq"], case["far"]
    start = torch.randint(0, max(1, far - s), (b, 1), generator=g, device="cuda")
    pos = start + torch.arange(s, device="cuda")[None]
    if case["pad"]:  # sequences of unequal length: the rows behind a sequence's end hold position -1
        n = torch.randint(1, s + 1, (b, 1), generator=g, device="cuda")
        pos = torch.where(torch.arange(s, device="cuda")[None] < n, pos, torch.full_like(pos, -1))
    return pos.to(torch.int32).contiguous()


def _routes(case, g, blocks):
    """Ascending distinct chunks per (b, g, block), -1 where the history is shorter or a hole."""
    b, h, nc, k = case["batch"], case["hkv"], case["nc"], case["topk"]
    n = min(k, nc)
    pick = torch.rand(b, h, blocks, nc, generator=g, device="cuda").topk(n, dim=-1).indices.sort(dim=-1).values
    idx = torch.full((b, h, blocks, k), -1, device="cuda", dtype=torch.int32)
    idx[..., :n] = pick.to(torch.int32)
    for _ in range(case["holes"]):
        at = torch.randint(0, k, (b, h, blocks, 1), generator=g, device="cuda")
        idx.scatter_(-1, at, -1)
    return idx


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case=case)
    if op in ("qk_norm_rope", "qk_norm_rope_bwd"):
        b, s, hq, hkv, d, dt = case["batch"], case["seq"], case["hq"], case["hkv"], case["d"], _dt(case)
        st["qkv"] = _randn(g, b, s, (hq + 2 * hkv) * d, dtype=dt)  # one fused projection, token-major
        st["wq"] = (1 + 0.1 * _randn(g, d)).to(dt)
        st["wk"] = (1 + 0.1 * _randn(g, d)).to(dt)
        st["positions"] = _positions(case, g)
        st["table"] = _table(case["far"], case["rot"])
        if op == "qk_norm_rope":
            w = case["window"]
            st["q"] = _randn(g, b, hq, s, d, dtype=dt)
            st["k"] = _randn(g, b, hkv, w, d, dtype=dt)  # the new rows go behind the window's older ones
            st["v"] = _randn(g, b, hkv, w, d, dtype=dt)
        else:
            st["dq"] = _randn(g, b, hq, s, d)  # fp32, as the attention's backward writes them
            st["dk"] = _randn(g, b, hkv, s, d)
            st["dv"] = _randn(g, b, hkv, s, d)
            st["dqkv"] = torch.empty_like(st["qkv"])
            st["dwq"] = torch.empty(d, device="cuda")
            st["dwk"] = torch.empty(d, device="cuda")
        if own:
            import hierarchical_sparse_long_b200 as hga
            st["p"] = hga.ProjParams(batch=b, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, seq_len=s,
                                     rotary_dim=case["rot"], dtype=hga.HGA_FP32 if dt == torch.float32 else hga.HGA_BF16,
                                     kv_head_stride=case["window"] if op == "qk_norm_rope" else s, eps=1e-6)
            if op == "qk_norm_rope_bwd":
                st["ws"] = torch.empty(hga.hga_qk_norm_rope_workspace_size(st["p"]), device="cuda", dtype=torch.uint8)
    elif op == "pack_history":
        b, n, hkv, d, dt = case["batch"], case["chunks"], case["hkv"], case["d"], _dt(case)
        st["k"] = _keys(g, b, hkv, n, d, dt)
        st["v"] = _randn(g, b, hkv, n * CHUNK, d, dtype=dt)
        st["hist"] = torch.zeros(b, hkv, n, 72 * d, device="cuda", dtype=torch.uint8)
        st["summ"] = torch.empty(b, hkv, n, d, device="cuda")
        st["k2"], st["v2"] = torch.empty_like(st["k"]), torch.empty_like(st["v"])
    else:
        b, hq, hkv, d, nc = case["batch"], case["hq"], case["hkv"], case["d"], case["nc"]
        s = case["seq"] if op == "fwd_packed" else 1
        st["hist"] = torch.empty(b, hkv, nc, 72 * d, device="cuda", dtype=torch.uint8)
        for i in range(b):  # one sequence at a time keeps the bf16 copy small
            st["hist"][i] = _pack(_keys(g, 1, hkv, nc, d, torch.bfloat16),
                                  _randn(g, 1, hkv, nc * CHUNK, d, dtype=torch.bfloat16))[0]
        st["q"] = _randn(g, b, hq, s, d, dtype=torch.bfloat16)
        n = s if op == "fwd_packed" else case["local"]
        st["k"] = _keys(g, b, hkv, -(-n // CHUNK), d, torch.bfloat16)[:, :, :n].contiguous()
        st["v"] = _randn(g, b, hkv, n, d, dtype=torch.bfloat16)
        st["idx"] = _routes(case, g, max(1, s // CHUNK))
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(b, hq, s, device="cuda")
        if own:
            import hierarchical_sparse_long_b200 as hga
            st["p"] = hga.Params(batch=b, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, topk=case["topk"], seg_len=s,
                                 n_hist_chunks=nc, seg_head_stride=n, q_block=64 if op == "fwd_packed" else 1)
    return st


# ---------------------------------------------------------------- plain forms
def _norm_rope(x, w, cos, sin, rot):
    """x [..., heads, d] fp32, cos / sin [..., 1, rot / 2]."""
    n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    a, b = n[..., :rot // 2], n[..., rot // 2:rot]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, n[..., rot:]], dim=-1)


def _norm_rope_grad(x, w, cos, sin, rot, dy):
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    a, b = dy[..., :rot // 2], dy[..., rot // 2:rot]
    dn = torch.cat([a * cos + b * sin, b * cos - a * sin, dy[..., rot:]], dim=-1)
    xh = x * r
    gw = dn * w
    return r * (gw - xh * (gw * xh).mean(-1, keepdim=True)), dn * xh


def _split(case, qkv):
    b, s, hq, hkv, d = case["batch"], case["seq"], case["hq"], case["hkv"], case["d"]
    x = qkv.view(b, s, hq + 2 * hkv, d)
    return x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]


def _plain_norm_rope(st):
    case = st["case"]
    s, rot, w0 = case["seq"], case["rot"], case["window"] - case["seq"]
    q, k, v = _split(case, st["qkv"])
    pos = st["positions"].long()
    keep = (pos >= 0)[:, None, :, None]
    row = st["table"][pos.clamp(min=0)][:, :, None]
    cos, sin = row[..., :rot // 2], row[..., rot // 2:]
    for x, w, dst in ((q, st["wq"], st["q"]), (k, st["wk"], st["k"][:, :, w0:])):
        y = _norm_rope(x.float(), w.float(), cos, sin, rot).transpose(1, 2)
        dst.copy_(torch.where(keep, y.to(dst.dtype), dst))
    dst = st["v"][:, :, w0:]
    dst.copy_(torch.where(keep, v.transpose(1, 2), dst))
    return st["q"], st["k"], st["v"]


def _plain_norm_rope_bwd(st):
    case = st["case"]
    rot = case["rot"]
    q, k, _ = _split(case, st["qkv"])
    pos = st["positions"].long()
    keep = (pos >= 0)[:, :, None, None]
    row = st["table"][pos.clamp(min=0)][:, :, None]
    cos, sin = row[..., :rot // 2], row[..., rot // 2:]
    dx, dw = [], []
    for x, w, dy in ((q, st["wq"], st["dq"]), (k, st["wk"], st["dk"])):
        a, b = _norm_rope_grad(x.float(), w.float(), cos, sin, rot, dy.transpose(1, 2))
        dx.append(torch.where(keep, a, torch.zeros_like(a)))
        # a weight's gradient is a sum over every row: 64 bits
        dw.append(torch.where(keep, b, torch.zeros_like(b)).double().sum(dim=(0, 1, 2)).float())
    dv = st["dv"].transpose(1, 2)
    dx.append(torch.where(keep, dv, torch.zeros_like(dv)))
    st["dqkv"].copy_(torch.cat(dx, dim=2).flatten(2))
    return st["dqkv"], dw[0], dw[1]


def _quant(x, dim):
    """Grid and codes of the groups of x (fp32) along dim."""
    mn, mx = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
    s = ((mx - mn) / 15).bfloat16().float()
    s = torch.where(s < 2.0 ** -100, torch.zeros_like(s), s)
    z = (mn.double() - 16 * s.double()).float().bfloat16().float()
    # which code is nearest is decided in 64 bits
    c = torch.round((x.double() - z) / torch.where(s == 0, torch.ones_like(s), s)) - 16
    c = torch.where(s == 0, torch.zeros_like(c), c).clamp(0, 15)
    return s, z, c.to(torch.int32)


def _words(c):
    """Codes [..., 8] -> int32 words [...] (element 2j in nibble j, 2j + 1 in nibble 4 + j)."""
    sh = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=c.device, dtype=torch.int64)
    w = (c.to(torch.int64) << sh).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _bytes(t):
    return t.contiguous().view(torch.uint8)


def _pack(k, v):
    """k, v [b][h][n * 64][d] -> records [b][h][n][72 d]."""
    b, h, t, d = k.shape
    n = t // CHUNK
    kc = k.float().view(b, h, n, CHUNK, d)
    s, z, c = _quant(kc, 3)
    kw = _words(c.view(b, h, n, CHUNK, d // 8, 8)).view(b, h, n, -1)
    parts = [_bytes(kw), _bytes(s.bfloat16().view(b, h, n, d)), _bytes(z.bfloat16().view(b, h, n, d))]
    vc = v.float().view(b, h, n, CHUNK, d // 64, 64)
    s, z, c = _quant(vc, 5)
    c = c.view(b, h, n, CHUNK, d).transpose(3, 4).reshape(b, h, n, d, 8, 8)
    s, z = (a[..., 0].transpose(3, 4).bfloat16().reshape(b, h, n, -1) for a in (s, z))
    parts += [_bytes(_words(c).view(b, h, n, -1)), _bytes(s), _bytes(z)]
    return torch.cat(parts, dim=-1)


def _codes(w):
    sh = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=w.device, dtype=torch.int32)
    return (w[..., None] >> sh) & 15


def _unpack(rec, d):
    """Records [..., 72 d] -> values of k, v [..., 64, d] (fp32 holding bf16 values)."""
    lead = rec.shape[:-1]
    kw, ks, kz, vw, vs, vz = torch.split(rec, [32 * d, 2 * d, 2 * d, 32 * d, 2 * d, 2 * d], dim=-1)
    f = lambda a: a.contiguous().view(torch.bfloat16).float()
    i = lambda a: a.contiguous().view(torch.int32)
    k = _codes(i(kw).view(*lead, CHUNK, d // 8)).reshape(*lead, CHUNK, d).float()
    k = ((k + 16) * f(ks).unsqueeze(-2) + f(kz).unsqueeze(-2)).bfloat16().float()
    v = _codes(i(vw).view(*lead, d, 8)).reshape(*lead, d // 64, 64, CHUNK).float()
    s, z = (f(a).view(*lead, d // 64, 1, CHUNK) for a in (vs, vz))
    v = ((v + 16) * s + z).bfloat16().float().reshape(*lead, d, CHUNK).transpose(-1, -2)
    return k, v


def _plain_pack(st):
    case = st["case"]
    b, n, hkv, d = case["batch"], case["chunks"], case["hkv"], case["d"]
    st["hist"].copy_(_pack(st["k"], st["v"]))
    st["summ"].copy_(st["k"].float().view(b, hkv, n, CHUNK, d).mean(3))
    k, v = _unpack(st["hist"], d)
    st["k2"].copy_(k.reshape(b, hkv, n * CHUNK, d))
    st["v2"].copy_(v.reshape(b, hkv, n * CHUNK, d))
    return st["summ"], st["k2"], st["v2"]


def _attend(q, keys, vals, mask):
    """q [..., r, d]; keys, vals [..., t, d]; mask [..., r or 1, t] -> out, lse (natural log)."""
    x = (q @ keys.transpose(-1, -2)) / math.sqrt(q.shape[-1])
    x = x.masked_fill(~mask, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    return (p / l) @ vals, (m + l.log())[..., 0]


def _gather(st, blk):
    """Values of block blk's routed chunks [b][h][k * 64][d], and which of them are routed."""
    case = st["case"]
    idx = st["idx"][:, :, blk].long()
    b, h, k = idx.shape
    rec = st["hist"].gather(2, idx.clamp(min=0)[..., None].expand(-1, -1, -1, st["hist"].shape[-1]))
    kk, vv = _unpack(rec, case["d"])
    ok = (idx >= 0)[..., None].expand(-1, -1, -1, CHUNK).reshape(b, h, 1, k * CHUNK)
    return kk.reshape(b, h, k * CHUNK, -1), vv.reshape(b, h, k * CHUNK, -1), ok


def _plain_attn(st):
    case = st["case"]
    b, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["d"]
    grp = hq // hkv
    fwd = case["op"] == "fwd_packed"
    rows = CHUNK if fwd else 1
    for blk in range(st["idx"].shape[2]):
        kh, vh, ok = _gather(st, blk)
        n = (blk + 1) * CHUNK if fwd else case["local"]
        q = st["q"][:, :, blk * rows:(blk + 1) * rows].float().reshape(b, hkv, grp * rows, d)
        loc = torch.ones(1, 1, grp * rows, n, dtype=torch.bool, device="cuda")
        if fwd:
            i = torch.arange(rows, device="cuda").repeat(grp) + blk * CHUNK
            loc = (torch.arange(n, device="cuda")[None] <= i[:, None])[None, None]
        mask = torch.cat([ok.expand(-1, -1, grp * rows, -1), loc.expand(b, hkv, -1, -1)], dim=-1)
        o, l = _attend(q, torch.cat([kh, st["k"][:, :, :n].float()], dim=2),
                       torch.cat([vh, st["v"][:, :, :n].float()], dim=2), mask)
        st["out"][:, :, blk * rows:(blk + 1) * rows] = o.reshape(b, hq, rows, d).to(st["out"].dtype)
        st["lse"][:, :, blk * rows:(blk + 1) * rows] = l.reshape(b, hq, rows)
    return st["out"], st["lse"]


# ---------------------------------------------------------------- one pass
def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"qk_norm_rope": _plain_norm_rope, "qk_norm_rope_bwd": _plain_norm_rope_bwd,
                "pack_history": _plain_pack, "decode_packed": _plain_attn, "fwd_packed": _plain_attn}[op](st)
    import hierarchical_sparse_long_b200 as hga
    if op == "qk_norm_rope":
        d, hq, hkv, w0 = case["d"], case["hq"], case["hkv"], case["window"] - case["seq"]
        x = st["qkv"]
        hga.hga_qk_norm_rope(st["p"], x, x[..., hq * d:], x[..., (hq + hkv) * d:], st["wq"], st["wk"], st["table"],
                             st["positions"], st["q"], st["k"][:, :, w0:], st["v"][:, :, w0:])
        return st["q"], st["k"], st["v"]
    if op == "qk_norm_rope_bwd":
        d, hq, hkv = case["d"], case["hq"], case["hkv"]
        x, dx = st["qkv"], st["dqkv"]
        hga.hga_qk_norm_rope_bwd(st["p"], x, x[..., hq * d:], st["wq"], st["wk"], st["table"], st["positions"],
                                 st["dq"], st["dk"], st["dv"], dx, dx[..., hq * d:], dx[..., (hq + hkv) * d:],
                                 st["dwq"], st["dwk"], st["ws"])
        return dx, st["dwq"], st["dwk"]
    if op == "pack_history":
        b, n, hkv, d = case["batch"], case["chunks"], case["hkv"], case["d"]
        hga.hga_pack_history(st["k"], st["v"], n * CHUNK, b, hkv, d, 0, n, st["hist"], n, st["summ"], n)
        hga.hga_unpack_history(st["hist"], n, b, hkv, d, 0, n, st["k2"], st["v2"], n * CHUNK)
        return st["summ"], st["k2"], st["v2"]
    if op == "decode_packed":
        hga.hga_attn_decode_packed(st["p"], st["q"], st["hist"], case["nc"], st["k"], st["v"], case["local"],
                                   st["idx"], st["out"], st["lse"])
    else:
        hga.hga_attn_fwd_packed(st["p"], st["q"], st["hist"], case["nc"], st["k"], st["v"], st["idx"], st["out"],
                                st["lse"])
    return st["out"], st["lse"]


def work(case):
    op, hkv, d, b = case["op"], case["hkv"], case["d"], case["batch"]
    e = 4 if case.get("dtype") == "fp32" else 2
    if op in ("qk_norm_rope", "qk_norm_rope_bwd"):
        tok, hq = b * case["seq"], case["hq"]
        plan = tok * (4 * case["rot"] + 4) + 2 * d * e
        if op == "qk_norm_rope":
            # squares and their sum 2, two scalings 2, rotation 3 per element of q and k
            return dict(bytes=2 * tok * (hq + 2 * hkv) * d * e + plan, flops=7 * tok * (hq + hkv) * d)
        return dict(bytes=tok * ((hq + hkv) * d * e + (hq + 2 * hkv) * d * (4 + e)) + plan + 8 * d,
                    flops=14 * tok * (hq + hkv) * d)
    if op == "pack_history":
        n = b * hkv * case["chunks"]
        # K and V in, records and summaries out; records in, K and V out
        return dict(bytes=n * (4 * CHUNK * d * e + 2 * 72 * d + 4 * d), flops=n * CHUNK * d * 2 * 8)
    hq, k = case["hq"], min(case["topk"], case["nc"])
    if op == "decode_packed":
        return dict(bytes=b * hkv * (k * 72 * d + case["local"] * 4 * d + 4 * case["topk"]) + b * hq * (4 * d + 4),
                    flops=4 * d * b * hq * (k * CHUNK + case["local"]))
    s = case["seq"]
    routed = min(case["nc"], k * (s // CHUNK))  # distinct chunks a head can route to
    return dict(bytes=b * hkv * (routed * 72 * d + 4 * s * d + 4 * case["topk"] * (s // CHUNK)) + b * hq * s * (4 * d + 4),
                flops=4 * d * b * hq * (s * k * CHUNK + s * (s + 1) // 2))


# ---------------------------------------------------------------- from the definitions, in 64 bits
def _to_bf16(x):
    """float64 -> the nearest bf16 value, ties to even, in one rounding (normal range)."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(torch.ldexp(m, torch.full_like(e, 8))), e - 8)


def _exact_grid(x, dim):
    """Values that the 4-bit record stands for, from float64 x of bf16 or fp32 values."""
    lo, hi = x.min(dim, keepdim=True).values, x.max(dim, keepdim=True).values
    # the definition divides in 32 bits before it rounds to bf16
    s = _to_bf16(((hi - lo).float() / 15).double())
    s = s * (s >= 2.0 ** -100)
    z = _to_bf16((lo - 16 * s).float().double())
    code = torch.round((x - z) / s.masked_fill(s == 0, 1)).clamp(16, 31)
    return _to_bf16(torch.where(s == 0, z.expand_as(x), s * code + z))


def _exact_values(rec, d):
    """Records [n][72 d] -> k, v [n][64][d] in float64, byte by byte."""
    n = rec.shape[0]
    r = rec.long()
    half = lambda a: (a[:, 0::2] + 256 * a[:, 1::2])
    bf = lambda a: (half(a) << 16).to(torch.int32).view(torch.float32).double()
    # byte y of a word holds nibbles 2y and 2y + 1: elements 0 2 | 4 6 | 1 3 | 5 7
    order = torch.tensor([0, 4, 1, 5, 2, 6, 3, 7], device=rec.device)
    nib = lambda a, rows: torch.stack([a & 15, a >> 4], dim=-1).view(n, rows, -1, 8)[..., order].reshape(n, rows, -1)
    k = nib(r[:, :32 * d], CHUNK) + 16
    k = _to_bf16(k * bf(r[:, 32 * d:34 * d])[:, None] + bf(r[:, 34 * d:36 * d])[:, None])
    r = r[:, 36 * d:]
    v = nib(r[:, :32 * d], d) + 16
    s, z = (bf(a).view(n, d // 64, 1, CHUNK).expand(-1, -1, 64, -1).reshape(n, d, CHUNK)
            for a in (r[:, 32 * d:34 * d], r[:, 34 * d:]))
    return k, _to_bf16(v * s + z).transpose(1, 2)


def _exact_norm_rope(case, st):
    b, s, hq, hkv, d, rot = (case[n] for n in ("batch", "seq", "hq", "hkv", "d", "rot"))
    x = st["qkv"].double().view(b, s, hq + 2 * hkv, d).permute(0, 2, 1, 3)  # [b][head][s][d]
    w = torch.ones(hq + 2 * hkv, 1, d, dtype=torch.float64, device="cuda")
    w[:hq], w[hq:hq + hkv] = st["wq"].double(), st["wk"].double()
    pos = st["positions"].long()
    live = pos >= 0
    ang = st["table"].double()[pos.clamp(min=0)][:, None]  # [b][1][s][rot]
    # the rotation as a complex product of the pairs (i, i + rot / 2)
    turn = torch.complex(ang[..., :rot // 2], ang[..., rot // 2:])
    r = (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    return x, w, r, turn, live


def exact(case, seed):
    st = prepare(case, seed)
    op, d = case["op"], case["d"]
    if op == "qk_norm_rope":
        hq, hkv, rot, w0 = case["hq"], case["hkv"], case["rot"], case["window"] - case["seq"]
        x, w, r, turn, live = _exact_norm_rope(case, st)
        n = x * r * w
        y = torch.view_as_real(torch.complex(n[..., :rot // 2], n[..., rot // 2:rot]) * turn)
        y = torch.cat([y[..., 0], y[..., 1], n[..., rot:]], dim=-1)
        at = live[:, None, :, None]
        q = torch.where(at, y[:, :hq], st["q"].double())
        k, v = st["k"].double(), st["v"].double()
        k[:, :, w0:] = torch.where(at, y[:, hq:hq + hkv], k[:, :, w0:])
        v[:, :, w0:] = torch.where(at, x[:, hq + hkv:], v[:, :, w0:])
        return q, k, v
    if op == "qk_norm_rope_bwd":
        b, s, hq, hkv, rot = (case[n] for n in ("batch", "seq", "hq", "hkv", "rot"))
        x, w, r, turn, live = _exact_norm_rope(case, st)
        x, w, r = x[:, :hq + hkv], w[:hq + hkv], r[:, :hq + hkv]
        at = live[:, None, :, None]
        dy = torch.cat([st["dq"], st["dk"]], dim=1).double() * at
        dn = torch.view_as_real(torch.complex(dy[..., :rot // 2], dy[..., rot // 2:rot]) * turn.conj())
        dn = torch.cat([dn[..., 0], dn[..., 1], dy[..., rot:]], dim=-1)
        # d/dx of x r(x): r I - r^3 x x^T / d
        g = dn * w
        dx = r * g - r ** 3 * x * (g * x).sum(-1, keepdim=True) / d
        dx = torch.cat([dx, st["dv"].double() * at], dim=1)
        dw = (dn * x * r).sum(dim=(0, 2))
        return dx.permute(0, 2, 1, 3).reshape(b, s, -1), dw[:hq].sum(0), dw[hq:].sum(0)
    if op == "pack_history":
        b, n, hkv = case["batch"], case["chunks"], case["hkv"]
        k = st["k"].double().view(b, hkv, n, CHUNK, d)
        v = st["v"].double().view(b, hkv, n * CHUNK, d // 64, 64)
        return (k.sum(3) / CHUNK, _exact_grid(k, 3).view(b, hkv, n * CHUNK, d),
                _exact_grid(v, 4).view(b, hkv, n * CHUNK, d))
    b, hq, hkv = case["batch"], case["hq"], case["hkv"]
    fwd = op == "fwd_packed"
    rows, grp = (CHUNK if fwd else 1), hq // hkv
    out = torch.empty(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["lse"].shape, dtype=torch.float64, device="cuda")
    for i in range(b):
        for h in range(hkv):
            for blk in range(st["idx"].shape[2]):
                idx = st["idx"][i, h, blk].long()
                kk, vv = _exact_values(st["hist"][i, h][idx[idx >= 0]], d)
                n = (blk + 1) * CHUNK if fwd else case["local"]
                kk = torch.cat([kk.reshape(-1, d), st["k"][i, h, :n].double()])
                vv = torch.cat([vv.reshape(-1, d), st["v"][i, h, :n].double()])
                q = st["q"][i, h * grp:(h + 1) * grp, blk * rows:(blk + 1) * rows].double()
                x = torch.einsum("grd,td->grt", q, kk) * d ** -0.5
                if fwd:  # row r of the block does not see its last 63 - r tokens
                    x[..., -CHUNK:] += torch.full((rows, CHUNK), -math.inf, dtype=torch.float64,
                                                  device="cuda").triu(1)
                l = torch.logsumexp(x, dim=-1)
                sl = (i, slice(h * grp, (h + 1) * grp), slice(blk * rows, (blk + 1) * rows))
                out[sl] = torch.einsum("grt,td->grd", torch.exp(x - l[..., None]), vv)
                lse[sl] = l
    return out, lse
