"""Cases of the operators around a main cache held in 4 bits: the norm of queries and keys with their rotary positions in one
pass, the entries that are packed into the cache, the rows that are read back from it, and the sparse attention over it.

Sizes are those of the package's workloads (64 heads of 192 / 128 over one KV head, 512 selected entries, a 128-token window,
blocks of 8 entries with 64-dim indexer keys, 8,192 to 32,768 entries a sequence) and, in drawn cases, generic ones.

An entry's key and value lie side by side: of every 16 dims, 16 codes of 4 bits (a sign, two bits of exponent, one of mantissa:
0, 0.5, 1, 1.5, 2, 3, 4, 6) and one scale of 8 bits (four of exponent, three of mantissa, up to 448); the key's groups
first, all codes before all scales, dim 2i in a byte's low bits, padded to 16 bytes. The value is code x scale x 2^exp."""
import math
import types

import torch

own = False

ROPE_BASE = 10000.0
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def _norm(name, **kw):
    c = dict(op="norm", rows=8, heads=64, dim=192, rot=64, off=128, dtype="bf16", interleaved=False, yarn=False, far=131072,
             center=False, each=False, fused=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def _append(name, **kw):
    c = dict(op="append", seqs=64, new=1, entries=32768, k_dim=192, v_dim=128, idx_dim=64, block=8, k_exp=-2, v_exp=0, dtype="bf16")
    c.update(kw)
    return dict(c, name=name) if name else c


def _rows(name, **kw):
    c = dict(op="rows", seqs=64, tokens=1, rows=512, entries=8192, k_dim=192, v_dim=128, k_exp=-2, v_exp=0, dtype="bf16")
    c.update(kw)
    return dict(c, name=name) if name else c


def _attn(name, **kw):
    c = dict(op="attn", seqs=1, tokens=1, entries=32768, topk=512, swa=128, heads=64, k_dim=192, v_dim=128, k_exp=-2, v_exp=0,
             holes=False, dtype="bf16")
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # queries and keys of one sequence's 8 drafted tokens, out of one projection: latency
        _norm("norm_draft_8", fused=True),
        # a prompt's queries and keys, positions up to 1M under YaRN, interleaved pairs: bandwidth
        _norm("norm_prompt_8192_yarn", rows=8192, interleaved=True, yarn=True, far=1048576),
        # an odd prompt in fp32, whole heads turned, layer norm with gains of each head
        _norm("norm_prompt_4097_f32", rows=4097, heads=16, dim=128, rot=128, off=0, dtype="f32", center=True, each=True),
        # one new entry of each of 64 sequences: a decode step's latency
        _append("append_64x1"),
        # prompts of 16 sequences packed behind what their caches hold already: bandwidth
        _append("append_16x8191", seqs=16, new=8191, entries=16384),
        # the rows that 64 queries selected
        _rows("rows_64x512"),
        # 16 whole caches read back
        _rows("rows_16x8192", seqs=16, rows=8192),
        # one query: latency
        _attn("attn_1"),
        # one token of each of 64 sequences of 128K tokens
        _attn("attn_64x1", seqs=64),
        # one token of each of 256 sequences of 32K tokens, some of whose selections are short
        _attn("attn_256x1", seqs=256, entries=8192, holes=True),
        # 32 tokens of each of 32 sequences
        _attn("attn_32x32", seqs=32, tokens=32, entries=8192),
        # fp32 queries and windows of other sizes
        _attn("attn_20x1_f32", seqs=20, entries=5000, topk=300, swa=50, heads=16, k_dim=100, v_dim=72, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "append", "append", "rows", "attn", "attn", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dims = rng.choice([(192, 128), (192, 128), (128, 128), (64, 64), (100, 72), (40, 24)])
    exps = dict(k_exp=rng.choice([-4, -2, -2, 0, 3]), v_exp=rng.choice([-3, 0, 0, 2]))
    if op == "norm":
        dim = rng.choice([64, 128, 192, 192, 256, 96, 40, 512])
        rot = rng.choice([r for r in (0, 8, 32, 64, 64, 128, dim) if r <= dim])
        heads = rng.choice([1, 8, 16, 48, 64, 64, 128])
        rows = _log(rng, 1, max(2, 8192 * 64 * 192 // (2 * heads * dim)))
        return _norm(None, rows=min(rows, 16384), heads=heads, dim=dim, rot=rot, off=rng.choice([0, dim - rot]), dtype=dtype,
                     interleaved=rng.random() < 0.5, yarn=rng.random() < 0.4, far=_log(rng, 100, 2000000),
                     center=rng.random() < 0.3, each=rng.random() < 0.3, fused=rng.random() < 0.5)
    if op == "append":
        seqs = _log(rng, 1, 64)
        new = _log(rng, 1, max(2, 65536 // seqs))
        return _append(None, seqs=seqs, new=new, entries=new + _log(rng, 8, 8192), k_dim=dims[0], v_dim=dims[1],
                       idx_dim=rng.choice([64, 64, 32]), block=rng.choice([8, 8, 4, 16]), dtype=dtype, **exps)
    if op == "rows":
        seqs = _log(rng, 1, 64)
        tokens = rng.choice([1, 1, 1, 3, 8])
        return _rows(None, seqs=seqs, tokens=tokens, rows=_log(rng, 1, max(2, 65536 // (seqs * tokens))),
                     entries=_log(rng, 16, 16384), k_dim=dims[0], v_dim=dims[1], dtype=dtype, **exps)
    tokens = rng.choice([1, 1, 1, 1, 2, 5, 16, 32])
    seqs = _log(rng, 1, max(1, min(256, 768 // tokens)))
    kw = dict(seqs=seqs, tokens=tokens, entries=_log(rng, 48, max(64, min(32768, (1 << 23) // (seqs * tokens)))),
              topk=rng.choice([512, 512, 512, 256, 99, 700]), swa=rng.choice([128, 128, 64, 37, 0]), holes=rng.random() < 0.5, **exps)
    if rng.random() < 0.3:  # other head counts, dims and the fp32 type
        kw.update(heads=rng.choice([4, 16, 40]), k_dim=dims[0], v_dim=dims[1], dtype=dtype, seqs=max(1, min(seqs, 96 // tokens)))
    return _attn(None, **kw)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 29)
    return g


def _randn(g, shape, dtype, mul=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * mul).to(dtype)


def _randint(g, lo, hi, shape):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)


def _selection(g, S, T, N, K, holes):
    """Selected entries [S * T, K], ascending, -1 behind: the tokens of a sequence are neighbours, so three quarters of their
    selections are the same entries; the others are each token's own. With holes, some select fewer, some nothing."""
    nv = _randint(g, max(1, (3 * N) // 4), N + 1, (S,))
    out = torch.arange(N, device="cuda", dtype=torch.int32)[None, :] >= nv[:, None]
    k = min(K, N)
    shared = (3 * k) // 4
    common = torch.rand((S, N), generator=g, device="cuda").masked_fill(out, -1.0)
    if shared:
        common.scatter_(1, common.topk(shared, dim=1).indices, 2.0)
    r = torch.rand((S, T, N), generator=g, device="cuda")
    r = torch.where((common == 2.0)[:, None, :], torch.full_like(r, 2.0), r).masked_fill(out[:, None, :], -1.0)
    top = r.topk(k, dim=2)
    ids = torch.where(top.values < 0, torch.full_like(top.indices, N), top.indices)
    if holes:
        short = torch.rand((S, T), generator=g, device="cuda") < 0.3
        n = torch.where(short, _randint(g, 0, k + 1, (S, T)), k)
        ids = ids.masked_fill(torch.arange(k, device="cuda") >= n[:, :, None], N)
    ids = ids.sort(dim=2).values
    idx = torch.full((S * T, K), -1, device="cuda", dtype=torch.int32)
    idx[:, :k] = torch.where(ids == N, torch.full_like(ids, -1), ids).reshape(S * T, k).to(torch.int32)
    return idx


def _shape(case, batch, **kw):
    d = dict(batch=batch, n_entries=case["entries"], idx_heads=8, idx_dim=64, block=8, pool_blocks=0, topk=512, q_heads=64,
             k_dim=case["k_dim"], v_dim=case["v_dim"], swa=128, scale=0.0, relu=1, dtype=case["dtype"], tokens=case.get("tokens", 1))
    d.update(kw)
    return types.SimpleNamespace(**d)


def _freqs(case):
    """Radians a position, per pair (float64), and the magnitude: base ** (-2 i / rot), under YaRN between that and that / factor."""
    rot = case["rot"]
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    f = ROPE_BASE ** (-2.0 * i / max(1, rot))
    if not case["yarn"]:
        return f, 1.0
    factor, orig = 32.0, 32768.0
    edge = lambda turns: rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(ROPE_BASE))  # noqa: E731
    lo, hi = max(0.0, math.floor(edge(32.0))), min(rot - 1.0, math.ceil(edge(1.0)))
    keep = 1.0 - torch.clamp((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
    return f / factor * (1.0 - keep) + f * keep, 0.1 * math.log(factor) + 1.0


def _entry_bytes(case):
    return -(-9 * (-(-case["k_dim"] // 16) + -(-case["v_dim"] // 16)) // 16) * 16


def _keys_values(g, case, shape):
    """Keys and values as they leave their projection: some dims are larger than the others, and 2^exp is about their size."""
    dt = DTYPES[case["dtype"]]
    dims = lambda d: 0.5 + torch.rand((d,), generator=g, device="cuda").square() * 2.0  # noqa: E731
    k = (_randn(g, (*shape, case["k_dim"]), torch.float32) * dims(case["k_dim"]) * 2.0 ** case["k_exp"]).to(dt)
    v = (_randn(g, (*shape, case["v_dim"]), torch.float32) * dims(case["v_dim"]) * 2.0 ** case["v_exp"]).to(dt)
    return k, v


def prepare(case, seed):
    g, dt, op = _gen(seed), DTYPES[case["dtype"]], case["op"]
    s = types.SimpleNamespace(case=case, call=None)
    if op == "norm":
        n, h, d = case["rows"], case["heads"], case["dim"]
        if case["fused"]:  # queries and keys are parts of one projection's rows
            whole = _randn(g, (n, (h + 1) * d), dt, 1.5)
            s.x = [whole[:, :h * d].unflatten(1, (h, d)), whole[:, h * d:].unflatten(1, (1, d))]
        else:
            s.x = [_randn(g, (n, h, d), dt, 1.5), _randn(g, (n, 1, d), dt, 0.7)]
        if case["center"]:
            s.x[0].add_(0.25)
        s.gain = [1.0 + 0.3 * torch.randn((h, d) if case["each"] else (d,), generator=g, device="cuda"),
                  1.0 + 0.3 * torch.randn((d,), generator=g, device="cuda")]
        s.out = [torch.empty((n, x.shape[1], d), device="cuda", dtype=dt) for x in s.x]
        s.pos = _randint(g, 0, case["far"], (n,))
        s.freq, s.mag = _freqs(case)
        s.eps = 1e-6
    elif op == "append":
        S, N, M = case["seqs"], case["entries"], case["new"]
        s.shape = _shape(case, S, idx_dim=case["idx_dim"], block=case["block"])
        s.k_new, s.v_new = _keys_values(g, case, (S, M))
        s.x_new = _randint(g, -4, 5, (S, M, case["idx_dim"])).to(dt)
        s.n_new = torch.where(torch.rand((S,), generator=g, device="cuda") < 0.75, M, _randint(g, 0, M + 1, (S,))).to(torch.int32)
        s.start = (torch.rand((S,), generator=g, device="cuda") * (N - M + 1)).to(torch.int32).clamp(max=N - M)
        s.n_valid = s.start.clone()
        s.kv = torch.zeros((S, N, _entry_bytes(case)), device="cuda", dtype=torch.uint8)
        s.k_idx = _randint(g, -4, 5, (S, N, case["idx_dim"])).to(dt)
        s.kb = torch.zeros((S, -(-N // case["block"]), case["idx_dim"]), device="cuda", dtype=dt)
        at = torch.arange(M, device="cuda", dtype=torch.int32)
        s.idx = torch.where(at < s.n_new[:, None], s.start[:, None] + at, -1).to(torch.int32).contiguous()
        s.out = [torch.empty((S, M, case["k_dim"]), device="cuda", dtype=dt), torch.empty((S, M, case["v_dim"]), device="cuda", dtype=dt)]
    else:
        S, T, N = case["seqs"], case["tokens"], case["entries"]
        B = S * T
        s.kv = torch.empty((S, N, _entry_bytes(case)), device="cuda", dtype=torch.uint8)
        step = max(1, (1 << 19) // N)
        for i in range(0, S, step):
            k, v = _keys_values(g, case, (min(step, S - i), N))
            s.kv[i:i + step] = _pack(case, k, v)
        if op == "rows":
            s.shape = _shape(case, B)
            R = case["rows"]
            if R >= N:  # the whole cache, in order
                row = torch.arange(R, device="cuda", dtype=torch.int32)
                s.idx = torch.where(row < N, row, -1).to(torch.int32).expand(B, R).contiguous()
            else:
                s.idx = _randint(g, -1, N, (B, R)).sort(dim=1, descending=True).values.contiguous()
            s.out = [torch.empty((B, R, case["k_dim"]), device="cuda", dtype=dt), torch.empty((B, R, case["v_dim"]), device="cuda", dtype=dt)]
        else:
            W, H, dk = case["swa"], case["heads"], case["k_dim"]
            s.shape = _shape(case, B, topk=case["topk"], swa=W, q_heads=H)
            s.scale = 1.0 / math.sqrt(dk)
            s.idx = _selection(g, S, T, N, case["topk"], case["holes"])
            # queries as large as makes some logits stand out, whatever the keys' size
            s.q = _randn(g, (B, H, dk), dt, 1.2 * 2.0 ** -case["k_exp"])
            s.k_swa, s.v_swa = _keys_values(g, case, (B, W))
            s.n_swa = torch.where(torch.rand((B,), generator=g, device="cuda") < 0.75, W, _randint(g, 0, W + 1, (B,))).to(torch.int32)
            s.out = torch.empty((B, H, case["v_dim"]), device="cuda", dtype=dt)
            s.lse = torch.empty((B, H), device="cuda", dtype=torch.float32)
    if own:  # the marshalled call that a decode loop keeps, as it keeps a layer group's
        s.call = _call(s, case)
    return s


# ------------------------------------------------------------------ the framework's calls

def _call(s, case):
    from sparse_attention_decode_index_gb300 import csa2
    if case["op"] == "norm":
        turned = case["rot"] > 0
        return csa2.NormRopeCall([(x, o, w, case["off"]) for x, o, w in zip(s.x, s.out, s.gain)], s.pos if turned else None,
                                 s.freq if turned else None, mag=s.mag, eps=s.eps, norm="layer" if case["center"] else "rms",
                                 interleaved=case["interleaved"])
    s.ws = csa2.workspace(s.shape)
    exps = dict(k_exp=case["k_exp"], v_exp=case["v_exp"])
    if case["op"] == "attn":
        return csa2.Kv4AttnCall(s.shape, s.q, s.kv, s.idx, s.k_swa, s.v_swa, s.n_swa, s.out, s.ws, lse=s.lse, **exps)
    rows = csa2.Kv4RowsCall(s.shape, s.kv, s.idx, s.out[0], s.out[1], s.ws, **exps)
    if case["op"] == "rows":
        return rows
    append = csa2.Kv4AppendCall(s.shape, s.n_new, s.k_new, s.v_new, s.x_new, s.kv, s.k_idx, s.kb, s.n_valid, s.ws, **exps)
    return lambda: (append(), rows())


# ------------------------------------------------------------------ plain forms

_MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)  # between neighbouring codes; a tie goes to the even one
_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _pow2(e):
    """2^e in fp32 for whole numbers e [...] of -126 to 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _codes(x, exp):
    """x [..., d] as codes [..., groups, 16] (0 to 15) and the scales' bytes [..., groups]."""
    d = x.shape[-1]
    t = torch.nn.functional.pad(x.float() * 2.0 ** -exp, (0, -d % 16)).unflatten(-1, (-1, 16))
    top = t.abs().amax(-1)
    want = (top.double() / 6.0).clamp(2.0 ** -9, 448.0)
    e = torch.frexp(want).exponent.clamp(min=-5) - 1  # floor of the logarithm, -6 for the subnormal ones
    m = torch.round(want * _pow2(3 - e)).to(torch.int32)  # 8 to 16 values (fewer where subnormal), ties to even
    byte = (e + 6) * 8 + m  # a mantissa of 16 values carries into the exponent
    s = m * _pow2(e - 3)
    c = torch.zeros(t.shape, device=t.device, dtype=torch.uint8)
    for i, mid in enumerate(_MIDS):
        edge = (mid * s)[..., None]
        c += (t.abs() >= edge) if i % 2 else (t.abs() > edge)
    c += (t < 0) * (c > 0) * torch.tensor(8, device=t.device, dtype=torch.uint8)
    bad = ~torch.isfinite(top)
    return c.masked_fill(bad[..., None], 0), byte.to(torch.uint8).masked_fill(bad, 127)


def _pack(case, k, v):
    """Packed entries [..., bytes] of keys and values."""
    parts = [_codes(k, case["k_exp"]), _codes(v, case["v_exp"])]
    codes = torch.cat([c for c, _ in parts], -2).flatten(-2)
    scales = torch.cat([b for _, b in parts], -1)
    flat = torch.cat((codes[..., 0::2] | (codes[..., 1::2] << 4), scales), -1)
    return torch.nn.functional.pad(flat, (0, _entry_bytes(case) - flat.shape[-1]))


def _unpack(case, entries):
    """Keys and values (fp32) of packed entries [..., bytes]."""
    gk, gv = -(-case["k_dim"] // 16), -(-case["v_dim"] // 16)
    g = gk + gv
    b = entries[..., :8 * g].to(torch.int32)
    codes = torch.stack((b & 15, b >> 4), -1).flatten(-2).unflatten(-1, (g, 16))
    level = torch.tensor(_LEVELS + tuple(-x for x in _LEVELS), device=b.device)[codes]
    byte = entries[..., 8 * g:9 * g].to(torch.int32)
    e, m = byte >> 3, byte & 7
    s = torch.where(e == 0, m * 2.0 ** -9, (m + 8) * _pow2(e - 10))
    s = s.masked_fill(byte == 127, math.nan)
    x = level * s[..., None]
    k = x[..., :gk, :].flatten(-2)[..., :case["k_dim"]] * 2.0 ** case["k_exp"]
    return k, x[..., gk:, :].flatten(-2)[..., :case["v_dim"]] * 2.0 ** case["v_exp"]


def _plain_norm(s, case):
    rot, off, half = case["rot"], case["off"], case["rot"] // 2
    if rot:
        a = s.pos.double()[:, None] * s.freq[None, :]
        cos, sin = (a.cos() * s.mag).float()[:, None, :], (a.sin() * s.mag).float()[:, None, :]
    for x, out, gain in zip(s.x, s.out, s.gain):
        y = x.float()
        if case["center"]:
            y = y - y.mean(-1, keepdim=True)
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s.eps) * gain
        if rot:
            r = y[..., off:off + rot]
            if case["interleaved"]:
                u, v = r[..., 0::2], r[..., 1::2]
                r = torch.stack((u * cos - v * sin, v * cos + u * sin), -1).flatten(-2)
            else:
                u, v = r[..., :half], r[..., half:]
                r = torch.cat((u * cos - v * sin, v * cos + u * sin), -1)
            y = torch.cat((y[..., :off], r, y[..., off + rot:]), -1)
        out.copy_(y)
    return s.out


def _gather(s, case, idx):
    """Packed entries [B, R, bytes] of each query's sequence, row 0 where idx is -1."""
    seq = torch.arange(idx.shape[0], device="cuda") // case.get("tokens", 1)
    return s.kv[seq[:, None], idx.clamp(min=0).long()]


def _plain_rows(s, case):
    gone = (s.idx < 0)[:, :, None]
    for out, x in zip(s.out, _unpack(case, _gather(s, case, s.idx))):
        out.copy_(x.masked_fill(gone, 0.0))
    return s.out


def _plain_append(s, case):
    S, N, blk = case["seqs"], case["entries"], case["block"]
    seq, at = (s.idx >= 0).nonzero(as_tuple=True)
    row = s.idx[seq, at].long()
    s.kv[seq, row] = _pack(case, s.k_new[seq, at], s.v_new[seq, at])
    s.k_idx[seq, row] = s.x_new[seq, at]
    s.n_valid.copy_(s.start + s.n_new)
    e = torch.arange(s.kb.shape[1] * blk, device="cuda")
    live = (e < s.n_valid[:, None])[..., None]
    x = torch.nn.functional.pad(s.k_idx.float(), (0, 0, 0, e.shape[0] - N)).masked_fill(~live, 0.0)
    mean = x.unflatten(1, (-1, blk)).sum(2) / live.unflatten(1, (-1, blk)).sum(2).clamp(min=1)
    j = torch.arange(s.kb.shape[1], device="cuda")
    touched = (j >= (s.start // blk)[:, None]) & (j * blk < s.n_valid[:, None]) & (s.n_new > 0)[:, None]
    s.kb.copy_(torch.where(touched[..., None], mean.round().to(s.kb.dtype), s.kb))
    return _plain_rows(s, case)


def _plain_attn(s, case):
    W = case["swa"]
    k, v = _unpack(case, _gather(s, case, s.idx))
    mask = torch.cat((s.idx >= 0, torch.arange(W, device="cuda") < s.n_swa[:, None]), 1)
    k, v = torch.cat((k, s.k_swa.float()), 1), torch.cat((v, s.v_swa.float()), 1)
    x = (s.q.float() @ k.transpose(1, 2) * s.scale).masked_fill(~mask[:, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    base = top.masked_fill(top == -math.inf, 0.0)
    p = (x - base).exp()
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / total.clamp(min=1e-38)
    return [o.to(s.q.dtype), (base + total.log()).squeeze(-1)]


def run(s):
    case = s.case
    if case["op"] == "append":  # the step before is put back, so that each pass appends the same entries
        s.n_valid.copy_(s.start)
    if own:
        s.call()
        if case["op"] == "attn":
            return [s.out, s.lse]
    else:
        got = {"norm": _plain_norm, "append": _plain_append, "rows": _plain_rows, "attn": _plain_attn}[case["op"]](s, case)
        if case["op"] == "attn":
            return got
    return [*s.out, s.k_idx, s.kb, s.n_valid] if case["op"] == "append" else s.out


# ------------------------------------------------------------------ what a pass cannot do without

def _union(S, T, N, K):
    """Expected distinct rows that T neighbours of each sequence select (see _selection)."""
    n = 0.875 * N
    k = min(K, n)
    shared = 0.75 * k
    return S * (shared + (n - shared) * (1.0 - (1.0 - (k - shared) / max(1.0, n - shared)) ** T))


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        n = case["rows"] * (case["heads"] + 1)
        gains = ((case["heads"] if case["each"] else 1) + 1) * case["dim"] * 4
        return {"bytes": 2 * n * case["dim"] * e + 4 * case["rows"] + gains, "flops": n * (4 * case["dim"] + 3 * case["rot"])}
    dk, dv, entry = case["k_dim"], case["v_dim"], _entry_bytes(case)
    if case["op"] == "append":  # and its rows read back
        n = case["seqs"] * case["new"] * (1.0 if case["new"] == 1 else 0.875)
        x = case["idx_dim"] * e
        return {"bytes": n * (2 * (dk + dv) * e + 2 * entry + 2 * x + x / case["block"]) + case["seqs"] * 12,
                "flops": n * 4 * (dk + dv)}
    S, T, N = case["seqs"], case["tokens"], case["entries"]
    B = S * T
    if case["op"] == "rows":
        R = case["rows"]
        n = S * N * (1.0 - (1.0 - 1.0 / N) ** (T * R)) if R < N else S * N
        return {"bytes": n * entry + B * R * ((dk + dv) * e + 4), "flops": B * R * (dk + dv)}
    H, K, W = case["heads"], case["topk"], case["swa"]
    k = min(K, 0.875 * N) * (0.85 if case["holes"] else 1.0)
    return {"bytes": B * H * (dk * e + dv * e + 4) + _union(S, T, N, k) * entry + B * 0.875 * W * (dk + dv) * e + B * K * 4,
            "flops": 2 * B * H * (k + 0.875 * W) * (dk + dv)}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _exact_norm(s, case):
    got = []
    f = s.freq.tolist()
    pos = s.pos.double()
    for x, gain in zip(s.x, s.gain):
        z = x.double()
        if case["center"]:
            z = z - z.sum(-1, keepdim=True) / case["dim"]
        z = gain.double() * z / torch.sqrt((z * z).sum(-1, keepdim=True) / case["dim"] + s.eps)
        y = z.clone()
        for i in range(case["rot"] // 2):
            p, q = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + case["rot"] // 2)
            p, q = p + case["off"], q + case["off"]
            w = torch.polar(torch.ones_like(pos), pos * f[i]) * s.mag
            w = torch.complex(z[..., p], z[..., q]) * w[:, None]
            y[..., p], y[..., q] = w.real, w.imag
        got.append(y)
    return got


def _nearest(x, table):
    """The entry of an ascending table (of an even count) nearest to x, at a tie the one of even index, as its index."""
    i = torch.searchsorted(table, x).clamp(1, table.numel() - 1)
    lo, hi = x - table[i - 1], table[i] - x
    return torch.where((lo < hi) | ((lo == hi) & ((i - 1) % 2 == 0)), i - 1, i)


def _stored(x, exp):
    """The 64-bit values that x [..., d] is stored as."""
    d = x.shape[-1]
    x = torch.nn.functional.pad(x.double() / 2.0 ** exp, (0, -d % 16)).unflatten(-1, (-1, 16))
    values = [m / 512 for m in range(8)] + [(8 + m) / 8 * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    scales = torch.tensor(values[:127], device=x.device, dtype=torch.float64)
    s = scales[_nearest(x.abs().amax(-1) / 6.0, scales).clamp(min=1)][..., None]
    levels = torch.tensor(_LEVELS, device=x.device, dtype=torch.float64)
    y = levels[_nearest(x.abs() / s, levels)] * s * torch.sign(x)
    return (y * 2.0 ** exp).flatten(-2)[..., :d]


def _exact_append(s, case):
    S, blk = case["seqs"], case["block"]
    live = (s.idx >= 0)[:, :, None]
    rows = [_stored(x, e).masked_fill(~live, 0.0) for x, e in ((s.k_new, case["k_exp"]), (s.v_new, case["v_exp"]))]
    kb = torch.zeros(s.kb.shape, device="cuda", dtype=torch.float64)
    for i in range(S):
        n0, m = int(s.start[i]), int(s.n_new[i])
        if m == 0:
            continue
        lo = n0 // blk * blk
        x = torch.cat((s.k_idx[i, lo:n0], s.x_new[i, :m])).double()
        for part, j in ((x[:len(x) // blk * blk].view(-1, blk, x.shape[1]), lo // blk), (x[len(x) // blk * blk:][None], (n0 + m) // blk)):
            if part.shape[0] and part.shape[1]:
                kb[i, j:j + part.shape[0]] = part.mean(1).round()
    return [*rows, None, kb, None]


def _exact_entries(case, entries):
    """Keys and values of packed entries [n, bytes], in 64 bits."""
    gk, gv = -(-case["k_dim"] // 16), -(-case["v_dim"] // 16)
    two = torch.tensor([2.0 ** i for i in range(-7, 9)], device="cuda", dtype=torch.float64)
    raw = entries.long()
    c = torch.stack((raw[:, :8 * (gk + gv)] % 16, raw[:, :8 * (gk + gv)] // 16), 2).flatten(1)
    ce, cm = c % 8 // 2, (c % 2).double() / 2
    x = torch.where(ce > 0, (1 + cm) * two[ce + 6], cm) * (1.0 - 2.0 * (c // 8))
    b = raw[:, 8 * (gk + gv):9 * (gk + gv)]
    e, m = b // 8, (b % 8).double() / 8
    x = x * torch.where(e > 0, (1 + m) * two[e], m / 64).repeat_interleave(16, 1)
    return x[:, :case["k_dim"]] * 2.0 ** case["k_exp"], x[:, 16 * gk:16 * gk + case["v_dim"]] * 2.0 ** case["v_exp"]


def _exact_rows(s, case):
    B, R = s.idx.shape
    out = [torch.zeros((B, R, case[d]), device="cuda", dtype=torch.float64) for d in ("k_dim", "v_dim")]
    for b in range(B):
        at = (s.idx[b] >= 0).nonzero().flatten()
        for o, x in zip(out, _exact_entries(case, s.kv[b // case["tokens"]][s.idx[b][at].long()])):
            o[b, at] = x
    return out


def _exact_attn(s, case):
    B, H = s.q.shape[:2]
    out = torch.zeros((B, H, case["v_dim"]), device="cuda", dtype=torch.float64)
    lse = torch.full((B, H), -math.inf, device="cuda", dtype=torch.float64)
    fills, idx, T = s.n_swa.tolist(), s.idx.cpu(), case["tokens"]
    for i in range(case["seqs"]):
        mine = idx[i * T:(i + 1) * T]
        ids = mine[mine >= 0].unique()
        keys, values = _exact_entries(case, s.kv[i][ids.cuda().long()])
        for b in range(i * T, (i + 1) * T):
            at = torch.searchsorted(ids, idx[b][idx[b] >= 0]).cuda()
            k = torch.cat((keys[at], s.k_swa[b, :fills[b]].double()))
            v = torch.cat((values[at], s.v_swa[b, :fills[b]].double()))
            if len(k) == 0:
                continue
            x = s.q[b].double() @ k.T / math.sqrt(case["k_dim"])
            lse[b] = torch.logsumexp(x, 1)
            out[b] = torch.exp(x - lse[b][:, None]) @ v
    return [out, lse]


def exact(case, seed):
    s = prepare(dict(case), seed)
    return {"norm": _exact_norm, "append": _exact_append, "rows": _exact_rows, "attn": _exact_attn}[case["op"]](s, case)
