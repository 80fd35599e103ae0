"""Cases of the operators around drafted tokens on the CSA2 caches: rotary positions, attention of a drafted tree, the
attention weights of accepted queries, the commit of an accepted path and eviction by accumulated weight.

Sizes are those of the package's workloads (64 heads of 192 / 128 over one KV head, 512 selected entries, a 128-token window,
blocks of 8 entries with 64-dim indexer keys, 8,192 to 262,144 entries a sequence) and, in drawn cases, generic ones."""
import math
import types

import torch

own = False

ROPE_BASE = 10000.0
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def _rope(name, **kw):
    c = dict(op="rope", rows=8, heads=64, dim=192, rot=64, off=128, dtype="bf16", interleaved=False, inverse=False, yarn=False,
             far=131072)
    c.update(kw)
    return dict(c, name=name) if name else c


def _tree(name, **kw):
    c = dict(op="tree", seqs=1, tokens=8, chain=False, ragged=False, entries=32768, topk=512, swa=128, heads=64, k_dim=192,
             v_dim=128, dtype="bf16")
    c.update(kw)
    return dict(c, name=name) if name else c


def _weights(name, **kw):
    c = dict(op="weights", seqs=1, tokens=1, entries=32768, topk=512, swa=128, heads=64, k_dim=192, v_dim=128, dtype="bf16")
    c.update(kw)
    return dict(c, name=name) if name else c


def _commit(name, **kw):
    c = dict(op="commit", seqs=1, tokens=8, layers=4, entries=32768, topk=512, swa=128, k_dim=192, v_dim=128, dtype="bf16")
    c.update(kw)
    return dict(c, name=name) if name else c


def _evict(name, **kw):
    c = dict(op="evict", seqs=1, entries=262144, keep=196608, sink=16, recent=1024, k_dim=192, v_dim=128, idx_dim=64, block=8,
             dtype="bf16")
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # queries and keys of one sequence's 8 drafted tokens: latency
        _rope("rope_draft_8"),
        # a prompt's queries and keys, positions up to 1M under YaRN, interleaved pairs: bandwidth
        _rope("rope_prompt_8192_yarn", rows=8192, interleaved=True, yarn=True, far=1048576),
        # a chain of 8 drafted tokens of one sequence: latency
        _tree("tree_1x8_chain", chain=True),
        # one token of each of 64 sequences, nothing drafted behind it: the form for single tokens
        _tree("tree_64x1", seqs=64, tokens=1),
        # trees of 16 drafted tokens, sequences with fewer live tokens among them
        _tree("tree_16x16", seqs=16, tokens=16, ragged=True),
        # the largest verification step: 32 sequences, trees of 32 tokens, 32K context
        _tree("tree_32x32", seqs=32, tokens=32, entries=8192),
        # one accepted query: latency
        _weights("weights_1x1"),
        # four accepted queries of each of 64 sequences
        _weights("weights_64x4", seqs=64, tokens=4, entries=8192),
        # one sequence's accepted path into 4 layers' windows
        _commit("commit_1x8"),
        # 64 sequences, 20 layers: a decoder group's windows and the weights of its accepted queries
        _commit("commit_64x16", seqs=64, tokens=16, layers=20, entries=8192),
        # one sequence of 1M tokens gives a quarter of its entries back
        _evict("evict_1x262144"),
        # 64 sequences of 32K tokens, some of them below the trigger, odd counts
        _evict("evict_64x8192", seqs=64, entries=8192, keep=6145, recent=256),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "tree", "tree", "tree", "weights", "commit", "evict"])
    if op == "rope":
        dim = rng.choice([64, 128, 192, 192, 96, 40])
        rot = rng.choice([r for r in (8, 16, 32, 64, 64, 128, dim) if r <= dim])
        heads = rng.choice([1, 8, 48, 64, 64, 128])
        rows = _log(rng, 1, max(2, 8192 * 64 * 192 // (2 * heads * dim)))
        return _rope(None, rows=min(rows, 16384), heads=heads, dim=dim, rot=rot, off=rng.choice([0, dim - rot]),
                     dtype=rng.choice(["bf16", "bf16", "f32"]), interleaved=rng.random() < 0.5, inverse=rng.random() < 0.3,
                     yarn=rng.random() < 0.4, far=_log(rng, 100, 2000000))
    if op in ("tree", "weights"):
        most = 64 if op == "tree" else 16
        tokens = _log(rng, 1, most)
        seqs = _log(rng, 1, max(1, min(64, 512 // tokens)))
        entries = _log(rng, 48, max(64, min(32768, (1 << 25) // (seqs * tokens * 4))))
        kw = dict(seqs=seqs, tokens=tokens, entries=entries, topk=rng.choice([512, 512, 512, 256, 99]),
                  swa=rng.choice([128, 128, 64, 37]))
        if rng.random() < 0.3:  # other head counts, dims and the fp32 type
            kw.update(heads=rng.choice([4, 16, 40]), k_dim=rng.choice([16, 64, 128, 100]), v_dim=rng.choice([16, 64, 128, 72]),
                      dtype=rng.choice(["bf16", "f32"]), seqs=max(1, min(seqs, 128 // tokens)))
        if op == "tree":
            kw.update(chain=rng.random() < 0.3, ragged=rng.random() < 0.5)
            return _tree(None, **kw)
        return _weights(None, **kw)
    if op == "commit":
        tokens = _log(rng, 1, 64)
        seqs = _log(rng, 1, max(1, min(64, 1024 // tokens)))
        return _commit(None, seqs=seqs, tokens=tokens, layers=rng.randint(1, 16), entries=_log(rng, 512, 32768),
                       topk=rng.choice([512, 256, 99]), swa=rng.choice([128, 64, 37]), dtype=rng.choice(["bf16", "bf16", "f32"]))
    seqs = _log(rng, 1, 48)
    entries = _log(rng, 128, max(256, 384 * 1024 // seqs))
    entries = min(262144, entries - entries % rng.choice([1, 8]))
    keep = rng.randint(max(8, entries // 4), entries - 1)
    return _evict(None, seqs=seqs, entries=entries, keep=keep, sink=rng.randint(0, 4), recent=rng.randint(0, keep // 2),
                  k_dim=rng.choice([192, 192, 64]), v_dim=rng.choice([128, 128, 72]), dtype=rng.choice(["bf16", "bf16", "f32"]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    return g


def _randn(g, shape, dtype, div=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) / div).to(dtype)


def _randint(g, lo, hi, shape):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)


def _selection(g, case):
    """Selected entries [seqs * tokens, topk], ascending, -1 behind: the drafted tokens of a sequence are neighbours, so three
    quarters of their selections are the same entries; the others are each token's own."""
    S, T, N, K = case["seqs"], case["tokens"], case["entries"], case["topk"]
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
    ids = torch.where(top.values < 0, torch.full_like(top.indices, N), top.indices).sort(dim=2).values
    idx = torch.full((S * T, K), -1, device="cuda", dtype=torch.int32)
    idx[:, :k] = torch.where(ids == N, torch.full_like(ids, -1), ids).reshape(S * T, k).to(torch.int32)
    return idx, nv


def _parents(g, S, T, chain):
    """Each drafted token's parent (an earlier token; -1 for the first): a chain, or a tree that grows near its newest tokens."""
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    if chain:
        return (t - 1).expand(S, T).contiguous()
    back = 1 + (torch.rand((S, T), generator=g, device="cuda").square() * torch.clamp(t, max=6)).to(torch.int32)
    return torch.clamp(t - back, min=0).masked_fill(t == 0, -1).to(torch.int32).contiguous()


def _paths(parent, g):
    """A path from the first token to a random one, as token ids [S, T] (0 behind) and its lengths [S]."""
    S, T = parent.shape
    par = parent.tolist()
    ends = _randint(g, 0, T, (S,)).tolist()
    rows, lens = [], []
    for s in range(S):
        p, t = [], ends[s]
        while t >= 0:
            p.append(t)
            t = par[s][t]
        rows.append(p[::-1] + [0] * (T - len(p)))
        lens.append(len(p))
    i32 = dict(device="cuda", dtype=torch.int32)
    return torch.tensor(rows, **i32), torch.tensor(lens, **i32)


def _shape(case, batch, **kw):
    d = dict(batch=batch, n_entries=case["entries"], idx_heads=8, idx_dim=64, block=8, pool_blocks=0, topk=512, q_heads=64, k_dim=192,
             v_dim=128, swa=128, scale=0.0, relu=1, dtype=case["dtype"], tokens=1)
    d.update(kw)
    return types.SimpleNamespace(**d)


def _freqs(case):
    """Radians a position, per pair (float64), and the magnitude: base ** (-2 i / rot), under YaRN between that and that / factor."""
    rot = case["rot"]
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    f = ROPE_BASE ** (-2.0 * i / rot)
    if not case["yarn"]:
        return f, 1.0
    factor, orig = 32.0, 32768.0
    edge = lambda turns: rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(ROPE_BASE))  # noqa: E731
    lo, hi = max(0.0, math.floor(edge(32.0))), min(rot - 1.0, math.ceil(edge(1.0)))
    keep = 1.0 - torch.clamp((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
    return f / factor * (1.0 - keep) + f * keep, 0.1 * math.log(factor) + 1.0


def prepare(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    s = types.SimpleNamespace(case=case, call=None)
    if case["op"] == "rope":
        n, h, d = case["rows"], case["heads"], case["dim"]
        s.x = [_randn(g, (n, h, d), dt), _randn(g, (n, 1, d), dt)]
        s.out = [torch.empty_like(x) for x in s.x]
        s.pos = _randint(g, 0, case["far"], (n,))
        s.freq, s.mag = _freqs(case)
    elif case["op"] in ("tree", "weights"):
        S, T, N, W, H = case["seqs"], case["tokens"], case["entries"], case["swa"], case["heads"]
        B, dk, dv = S * T, case["k_dim"], case["v_dim"]
        s.shape = _shape(case, B, topk=case["topk"], swa=W, q_heads=H, k_dim=dk, v_dim=dv, tokens=T)
        s.scale = 1.0 / math.sqrt(dk)
        s.k_main = _randn(g, (S, N, dk), dt, math.sqrt(dk) / 4)
        s.idx, _ = _selection(g, case)
        s.q = _randn(g, (B, H, dk), dt)
        if case["op"] == "tree":
            s.v_main = _randn(g, (S, N, dv), dt)
            s.k_swa, s.v_swa = _randn(g, (S, W, dk), dt, math.sqrt(dk) / 4), _randn(g, (S, W, dv), dt)
            s.k_draft, s.v_draft = _randn(g, (S, T, dk), dt, math.sqrt(dk) / 4), _randn(g, (S, T, dv), dt)
            s.n_swa = torch.where(torch.rand((S,), generator=g, device="cuda") < 0.75, W, _randint(g, 0, W + 1, (S,))).to(torch.int32)
            s.swa_head = torch.where(s.n_swa == W, _randint(g, 0, W, (S,)), s.n_swa).to(torch.int32)
            s.parent = _parents(g, S, T, case["chain"])
            s.n_draft = _randint(g, 1, T + 1, (S,)) if case["ragged"] else None
            s.out = torch.empty((B, H, dv), device="cuda", dtype=dt)
            s.lse = torch.empty((B, H), device="cuda", dtype=torch.float32)
        else:
            # what the attention left behind: the log-sum-exp over the selected entries and about as much again
            s.lse = torch.randn((B, H), generator=g, device="cuda") * 0.1 + math.log(2.0 * case["topk"])
            s.out = torch.empty((B, case["topk"]), device="cuda", dtype=torch.float32)
    elif case["op"] == "commit":
        S, T, N, W, K, L = case["seqs"], case["tokens"], case["entries"], case["swa"], case["topk"], case["layers"]
        s.shape = _shape(case, S * T, topk=K, swa=W, k_dim=case["k_dim"], v_dim=case["v_dim"], tokens=T)
        s.k_draft, s.v_draft = _randn(g, (L, S, T, case["k_dim"]), dt), _randn(g, (L, S, T, case["v_dim"]), dt)
        s.k_swa, s.v_swa = _randn(g, (L, S, W, case["k_dim"]), dt), _randn(g, (L, S, W, case["v_dim"]), dt)
        # a group's layers attend with the indices of every fourth of them
        sel = [_selection(g, case)[0] for _ in range(-(-L // 4))]
        s.idx = torch.stack([sel[i // 4] for i in range(L)])
        s.weights = torch.rand((L, S * T, K), generator=g, device="cuda").square().masked_fill(s.idx < 0, 0.0)
        s.path, s.n_path = _paths(_parents(g, S, T, False), g)
        # the heads, the fill counts and the accumulated weights in one buffer, so that one copy puts a step back
        s.start = torch.empty(S * N + S, device="cuda", dtype=torch.int64)
        s.start[:S * N] = (torch.rand(S * N, generator=g, device="cuda").double() * 2 ** 36).to(torch.int64)
        counts = s.start[S * N:].view(torch.int32)
        counts[S:] = torch.where(torch.rand((S,), generator=g, device="cuda") < 0.75, W, _randint(g, 0, W + 1, (S,)))
        counts[:S] = torch.where(counts[S:] == W, _randint(g, 0, W, (S,)), counts[S:])
        s.now = s.start.clone()
        s.mass = s.now[:S * N].view(S, N)
        s.swa_head, s.n_swa = s.now[S * N:].view(torch.int32)[:S], s.now[S * N:].view(torch.int32)[S:]
    else:
        S, N = case["seqs"], case["entries"]
        nb = -(-N // case["block"])
        s.shape = _shape(case, S, idx_dim=case["idx_dim"], block=case["block"], k_dim=case["k_dim"], v_dim=case["v_dim"])
        s.k_main, s.v_main = _randn(g, (S, N, case["k_dim"]), dt), _randn(g, (S, N, case["v_dim"]), dt)
        s.k_idx = _randint(g, -4, 5, (S, N, case["idx_dim"])).to(dt)
        full = torch.rand((S,), generator=g, device="cuda") < 0.8
        full[0] = True
        s.n_valid = torch.where(full, _randint(g, case["keep"] + 1, N + 1, (S,)), _randint(g, 1, case["keep"] + 1, (S,))).to(torch.int32)
        # a few entries draw most of the weight, many none at all
        u = torch.rand((S, N), generator=g, device="cuda").double()
        s.mass = torch.where(u < 0.1, torch.zeros_like(u), u.pow(8) * 2 ** 40).to(torch.int64)
        s.out = [torch.zeros_like(t) for t in (s.k_main, s.v_main, s.k_idx, s.mass, s.n_valid)]
        s.kb = torch.zeros((S, nb, case["idx_dim"]), device="cuda", dtype=dt)
        s.kept = torch.empty((S, N), device="cuda", dtype=torch.int32)
    if own:  # the marshalled call that a decode loop keeps, as it keeps a layer group's
        s.call = _call(s, case)
    return s


# ------------------------------------------------------------------ the framework's calls

def _call(s, case):
    from sparse_attention_decode_index_gb300 import csa2
    if case["op"] == "rope":
        return csa2.RopeCall([(x, o, case["off"]) for x, o in zip(s.x, s.out)], s.pos, s.freq, mag=s.mag,
                             interleaved=case["interleaved"], inverse=case["inverse"])
    s.ws = csa2.workspace(s.shape)
    if case["op"] == "tree":
        return csa2.TreeAttnCall(s.shape, s.q, s.k_main, s.v_main, s.idx, s.k_swa, s.v_swa, s.n_swa, s.k_draft, s.v_draft, s.out,
                                 s.ws, swa_head=s.swa_head, parent=s.parent, n_draft=s.n_draft, lse=s.lse)
    if case["op"] == "weights":
        return csa2.AttnWeightsCall(s.shape, s.q, s.k_main, s.idx, s.lse, s.out, s.ws)
    if case["op"] == "commit":
        slots = [(s.k_draft[i], s.v_draft[i], s.k_swa[i], s.v_swa[i], s.idx[i], s.weights[i]) for i in range(case["layers"])]
        return csa2.TreeCommitCall(s.shape, slots, s.path, s.n_path, s.swa_head, s.n_swa, s.ws, mass=s.mass)
    return csa2.KvEvictCall(s.shape, case["keep"], case["keep"], case["sink"], case["recent"], s.k_main, s.v_main, s.k_idx, s.mass,
                            s.n_valid, s.kept, s.ws, kb=s.kb, out=s.out)


# ------------------------------------------------------------------ plain forms

def _plain_rope(s, case):
    rot, off, half = case["rot"], case["off"], case["rot"] // 2
    a = s.pos.double()[:, None] * s.freq[None, :]
    m = 1.0 / s.mag if case["inverse"] else s.mag
    cos = (a.cos() * m).float()[:, None, :]
    sin = (a.sin() * (-m if case["inverse"] else m)).float()[:, None, :]

    def turn(x, out):
        r = x[..., off:off + rot].float()
        out.copy_(x)
        if case["interleaved"]:
            u, v = r[..., 0::2], r[..., 1::2]
            out[..., off:off + rot] = torch.stack((u * cos - v * sin, v * cos + u * sin), -1).flatten(-2).to(x.dtype)
        else:
            u, v = r[..., :half], r[..., half:]
            out[..., off:off + rot] = torch.cat((u * cos - v * sin, v * cos + u * sin), -1).to(x.dtype)
        return out

    return [turn(s.x[0], s.out[0]), turn(s.x[1], s.out[1])]


def _closure(parent):
    """[S, T, T]: 1 where the second token is the first one itself or an ancestor of it."""
    S, T = parent.shape
    a = (parent.long()[:, :, None] == torch.arange(T, device="cuda")).float() + torch.eye(T, device="cuda")
    for _ in range(max(1, (T - 1).bit_length())):  # each product doubles the reach
        a = (a @ a).clamp(max=1.0)
    return a


def _gather(cache, idx, T):
    """Rows idx [S * T, K] of cache [S, N, d], -1 read as row 0, in fp32."""
    seq = torch.arange(idx.shape[0], device="cuda") // T
    return cache[seq[:, None], idx.clamp(min=0).long()].float()


def _plain_tree(s, case):
    S, T, W = case["seqs"], case["tokens"], case["swa"]
    B = S * T
    anc = _closure(s.parent)
    depth = anc.sum(-1)  # keys among the draft: itself and its ancestors
    near = (anc > 0) & (depth[:, :, None] - depth[:, None, :] < W)
    row = torch.arange(W, device="cuda")
    newest = torch.where(s.n_swa == W, s.swa_head - 1, s.n_swa - 1)
    age = (newest[:, None] - row) % W  # 0 for the newest row of the window
    age = torch.where((s.n_swa == W)[:, None], age, newest[:, None] - row)
    in_window = (age[:, None, :] >= 0) & (age[:, None, :] + depth[:, :, None] < W) & (row < s.n_swa[:, None])[:, None, :]
    live = torch.ones((S, T), dtype=torch.bool, device="cuda")
    if s.n_draft is not None:
        live = torch.arange(T, device="cuda") < s.n_draft[:, None]
    mask = torch.cat((s.idx >= 0, in_window.reshape(B, W), near.reshape(B, T)), 1) & live.reshape(B, 1)
    each = lambda x: x.float()[:, None].expand(S, T, *x.shape[1:]).reshape(B, *x.shape[1:])  # noqa: E731
    k = torch.cat((_gather(s.k_main, s.idx, T), each(s.k_swa), each(s.k_draft)), 1)
    v = torch.cat((_gather(s.v_main, s.idx, T), each(s.v_swa), each(s.v_draft)), 1)
    x = (s.q.float() @ k.transpose(1, 2) * s.scale).masked_fill(~mask[:, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    base = top.masked_fill(top == -math.inf, 0.0)
    p = (x - base).exp()
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / total.clamp(min=1e-38)
    return [o.to(s.q.dtype), (base + total.log()).squeeze(-1)]


def _plain_weights(s, case):
    k = _gather(s.k_main, s.idx, case["tokens"])
    p = (s.q.float() @ k.transpose(1, 2) * s.scale - s.lse[:, :, None]).exp()
    return p.sum(1).masked_fill(s.idx < 0, 0.0)


def _plain_commit(s, case):
    L, S, T, W, N = case["layers"], case["seqs"], case["tokens"], case["swa"], case["entries"]
    s.now.copy_(s.start)
    j = torch.arange(T, device="cuda")
    taken = j < s.n_path[:, None]
    last = taken & (j >= s.n_path[:, None] - W)
    seq, at = last.nonzero(as_tuple=True)
    row = (s.swa_head[seq] + at) % W
    tok = s.path[seq, at].long()
    s.k_swa[:, seq, row.long()] = s.k_draft[:, seq, tok]
    s.v_swa[:, seq, row.long()] = s.v_draft[:, seq, tok]
    seq, at = taken.nonzero(as_tuple=True)
    b = seq * T + s.path[seq, at].long()
    idx, w = s.idx[:, b].long(), s.weights[:, b]
    units = torch.round(w.double() * 2 ** 32).to(torch.int64).masked_fill(idx < 0, 0)
    s.mass.view(-1).index_add_(0, (seq[None, :, None] * N + idx.clamp(min=0)).reshape(-1), units.reshape(-1))
    s.swa_head.copy_((s.swa_head + s.n_path) % W)
    s.n_swa.copy_((s.n_swa + s.n_path).clamp(max=W))
    return [s.k_swa, s.v_swa, s.mass, s.swa_head, s.n_swa]


def _plain_evict(s, case):
    S, N, keep, blk = case["seqs"], case["entries"], case["keep"], case["block"]
    e = torch.arange(N, device="cuda")
    nv = s.n_valid.long()
    evict = nv > keep
    safe = (e < case["sink"]) | (e >= nv[:, None] - case["recent"])
    rank = torch.where(safe, torch.full_like(s.mass, 2 ** 62), s.mass).masked_fill(e >= nv[:, None], -1)
    order = rank.sort(dim=1, descending=True, stable=True).indices
    chosen = torch.zeros((S, N), dtype=torch.bool, device="cuda").scatter_(1, order[:, :keep], True)
    chosen = torch.where(evict[:, None], chosen, torch.ones_like(chosen)) & (e < nv[:, None])
    n = chosen.sum(1)
    kept = torch.where(chosen, e, N).sort(dim=1).values
    seq, slot = (kept < N).nonzero(as_tuple=True)
    old = kept[seq, slot]
    k, v, x, mass, count = s.out
    k[seq, slot], v[seq, slot], x[seq, slot] = s.k_main[seq, old], s.v_main[seq, old], s.k_idx[seq, old]
    mass.zero_()
    mass[seq, slot] = s.mass[seq, old]
    count.copy_(n)
    s.kept.copy_(kept.masked_fill(kept == N, -1))
    nb = s.kb.shape[1]
    rows = torch.zeros((S, nb * blk, case["idx_dim"]), device="cuda")
    rows[seq, slot] = s.k_idx[seq, old].float()
    members = (n[:, None] - torch.arange(nb, device="cuda") * blk).clamp(1, blk)
    s.kb.copy_((rows.view(S, nb, blk, -1).sum(2) / members[:, :, None]).round())
    return [k, v, x, mass, count, s.kept, s.kb]


def run(s):
    case = s.case
    if own:
        if case["op"] == "commit":  # the step before is put back, so that each pass commits the same path
            s.now.copy_(s.start)
        s.call()
        return {"rope": lambda: s.out, "tree": lambda: [s.out, s.lse], "weights": lambda: s.out,
                "commit": lambda: [s.k_swa, s.v_swa, s.mass, s.swa_head, s.n_swa],
                "evict": lambda: [*s.out, s.kept, s.kb]}[case["op"]]()
    return {"rope": _plain_rope, "tree": _plain_tree, "weights": _plain_weights, "commit": _plain_commit,
            "evict": _plain_evict}[case["op"]](s, case)


# ------------------------------------------------------------------ what a pass cannot do without

def _union(S, T, N, K):
    """Expected distinct rows that T neighbours of each sequence select (see _selection)."""
    n = 0.875 * N
    k = min(K, n)
    shared = 0.75 * k
    return S * (shared + (n - shared) * (1.0 - (1.0 - (k - shared) / max(1.0, n - shared)) ** T))


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rope":
        n = case["rows"] * (case["heads"] + 1)
        return {"bytes": 2 * n * case["dim"] * e + 4 * case["rows"], "flops": 3 * n * case["rot"]}
    if case["op"] == "evict":
        row = (case["k_dim"] + case["v_dim"] + case["idx_dim"]) * e + 8
        S, N, keep = case["seqs"], case["entries"], case["keep"]
        full = 1 + 0.8 * (S - 1)
        kept = full * keep + (S - full) * (keep + 1) / 2
        nb = -(-N // case["block"])
        return {"bytes": 2 * kept * row + (full * 0.5 * (N - keep) + S * N) * 8 + S * N * 4 + S * nb * case["idx_dim"] * e,
                "flops": kept * case["idx_dim"]}
    S, T, N, K, W = case["seqs"], case["tokens"], case["entries"], case["topk"], case["swa"]
    B, dk, dv = S * T, case["k_dim"], case["v_dim"]
    if case["op"] == "commit":
        taken = 1 + math.log(T) / math.log(2.0)  # about as deep as a random token lies
        return {"bytes": S * taken * case["layers"] * (2 * (dk + dv) * e + 8 * K) + _union(S, 1, N, K) * 16,
                "flops": S * taken * case["layers"] * K}
    H = case["heads"]
    rows = _union(S, T, N, K)
    if case["op"] == "weights":
        return {"bytes": B * H * (dk * e + 4) + rows * dk * e + B * K * 8, "flops": 2 * B * H * min(K, 0.875 * N) * dk}
    live = 0.5 * B + 0.5 * S if case["ragged"] else B
    return {"bytes": live * H * dk * e + B * H * (dv * e + 4) + (rows + S * 0.9 * W + S * T) * (dk + dv) * e + live * K * 4,
            "flops": 2 * live * H * (min(K, 0.875 * N) + 0.9 * W) * (dk + dv)}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _exact_rope(s, case):
    got = []
    f = s.freq.tolist()
    pos = s.pos.double()
    for x in s.x:
        y = x.double().clone()
        for i in range(case["rot"] // 2):
            p, q = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + case["rot"] // 2)
            p, q = p + case["off"], q + case["off"]
            z = torch.polar(torch.ones_like(pos), pos * f[i])
            z = z.conj() / s.mag if case["inverse"] else z * s.mag
            w = torch.complex(x[..., p].double(), x[..., q].double()) * z[:, None]
            y[..., p], y[..., q] = w.real, w.imag
        got.append(y)
    return got


def _exact_tree(s, case):
    S, T, W, H = case["seqs"], case["tokens"], case["swa"], case["heads"]
    out = torch.zeros((S * T, H, case["v_dim"]), device="cuda", dtype=torch.float64)
    lse = torch.full((S * T, H), -math.inf, device="cuda", dtype=torch.float64)
    par, heads, fills, idx = s.parent.tolist(), s.swa_head.tolist(), s.n_swa.tolist(), s.idx.cpu()
    for i in range(S):
        live = T if s.n_draft is None else int(s.n_draft[i])
        order = [(heads[i] - 1 - a) % W for a in range(W)] if fills[i] == W else list(range(fills[i] - 1, -1, -1))
        for t in range(live):
            chain, c = [], t
            while c >= 0:
                chain.append(c)
                c = par[i][c]
            ring = order[:max(0, W - len(chain))]
            chain = chain[:W]
            b = i * T + t
            sel = idx[b][idx[b] >= 0].long().cuda()
            k = torch.cat((s.k_main[i][sel], s.k_swa[i][ring], s.k_draft[i][chain])).double()
            v = torch.cat((s.v_main[i][sel], s.v_swa[i][ring], s.v_draft[i][chain])).double()
            x = s.q[b].double() @ k.T / math.sqrt(case["k_dim"])
            lse[b] = torch.logsumexp(x, 1)
            out[b] = torch.exp(x - lse[b][:, None]) @ v
    return [out, lse]


def _exact_weights(s, case):
    w = torch.zeros(s.idx.shape, device="cuda", dtype=torch.float64)
    for b in range(s.idx.shape[0]):
        at = (s.idx[b] >= 0).nonzero().flatten()
        k = s.k_main[b // case["tokens"]][s.idx[b][at].long()].double()
        x = s.q[b].double() @ k.T / math.sqrt(case["k_dim"])
        w[b, at] = torch.exp(x - s.lse[b].double()[:, None]).sum(0)
    return w


def _exact_evict(s, case):
    """The block keys alone are computed numbers; everything else is moved."""
    S, blk = case["seqs"], case["block"]
    kb = torch.zeros(s.kb.shape, device="cuda", dtype=torch.float64)
    for i in range(S):
        n = int(s.n_valid[i])
        ids = list(range(n))
        if n > case["keep"]:
            mass = s.mass[i].tolist()
            middle = range(case["sink"], n - case["recent"])
            best = sorted(middle, key=lambda e: (-mass[e], e))[:case["keep"] - case["sink"] - case["recent"]]
            ids = sorted({*range(min(case["sink"], n)), *range(max(0, n - case["recent"]), n), *best})
        x = s.k_idx[i][torch.tensor(ids, device="cuda")].double()
        whole = len(ids) // blk
        kb[i, :whole] = x[:whole * blk].view(whole, blk, -1).mean(1).round()
        if len(ids) % blk:
            kb[i, whole] = x[whole * blk:].mean(0).round()
    return [None, None, None, None, None, None, kb]


def exact(case, seed):
    s = prepare(dict(case), seed)
    if case["op"] == "commit":
        return None
    return {"rope": _exact_rope, "tree": _exact_tree, "weights": _exact_weights, "evict": _exact_evict}[case["op"]](s, case)
