"""The operators around drafted tokens (csa2_rope, csa2_tree_attn, csa2_attn_weights, csa2_tree_commit, csa2_kv_evict)
on the GPU against plain 64-bit definitions, alone and as a serving step runs them together."""
import types

import numpy as np
import pytest

from tests import draft_reference as R
from tests.gpu_helpers import assert_no_device_error, lib_ready, need_gpu, torch

pytestmark = pytest.mark.gpu

BAD_INDEX, BAD_COUNT, BAD_WEIGHT = 1, 2, 16
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a rounding step, relative
EPS32 = 2.0 ** -23


@pytest.fixture(scope="module")
def csa2():
    need_gpu()
    return lib_ready()


def shape(batch, **kw):
    d = dict(batch=batch, n_entries=64, idx_heads=8, idx_dim=64, block=8, pool_blocks=0, topk=512, q_heads=64, k_dim=192,
             v_dim=128, swa=128, scale=0.0, relu=1, dtype="bf16", tokens=1)
    d.update(kw)
    return types.SimpleNamespace(**d)


def randn(g, size, dtype, div=1.0):
    return (torch.randn(size, generator=g) / div).to(dtype).cuda()


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def f64(t):
    return t.detach().cpu().double().numpy()


# ------------------------------------------------------------------ rotary positions

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rows,heads,dim,rot,off,inverse", [
    (1, 1, 2, 2, 0, False), (3, 64, 192, 64, 128, False), (5, 8, 64, 64, 0, True), (17, 3, 40, 8, 32, False),
    (2, 5, 10, 6, 3, True), (700, 4, 96, 16, 0, False), (4, 128, 1024, 1024, 0, False), (9, 2, 24, 12, 8, True),
    # vectors of 8 bytes; small rows, many a block
    (33, 5, 64, 8, 56, False), (6, 3, 36, 24, 4, False), (3000, 1, 40, 40, 0, True), (5000, 1, 64, 8, 0, False), (2000, 2, 12, 4, 8, True)])
def test_rope_matches_definition(csa2, dtype, inter, rows, heads, dim, rot, off, inverse):
    g = torch.Generator().manual_seed(rows * 31 + dim)
    x = randn(g, (rows, heads, dim), dtype)
    k = randn(g, (rows, dim), dtype)
    pos = torch.randint(0, 2 ** 20, (rows,), generator=g, dtype=torch.int32)
    pos[0] = 2 ** 31 - 1
    if rows > 2:
        pos[1], pos[2] = -12345, 0
    freqs, mag = csa2.rope_freqs(rot, 10000.0, scaling="yarn", factor=8.0, orig_ctx=4096)
    out, ko = torch.full_like(x, 7.0), torch.full_like(k, 7.0)
    csa2.rope([(x, out, off), (k, ko, off)], pos.cuda(), freqs, mag=mag, interleaved=inter, inverse=inverse)
    t = pos.numpy().astype(np.longdouble)[:, None] * freqs.cpu().numpy().astype(np.longdouble)[None]
    m = 1.0 / mag if inverse else mag
    c, s = np.cos(t) * m, np.sin(t) * (-m if inverse else m)
    for src, dst in ((x, out), (k[:, None], ko[:, None])):
        want = f64(src)
        r = want[..., off:off + rot].copy()
        a, b = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :rot // 2], r[..., rot // 2:])
        u, v = a * c[:, None] - b * s[:, None], b * c[:, None] + a * s[:, None]
        turned = np.empty_like(r)
        if inter:
            turned[..., 0::2], turned[..., 1::2] = u, v
        else:
            turned[..., :rot // 2], turned[..., rot // 2:] = u, v
        want[..., off:off + rot] = turned
        # the angle: 2^-52 of it from the frequency's rounding, 2^-25 turns in fp32; cos and sin 2 ulp; three roundings
        angle = np.abs(t).max() * 2.0 ** -51 + 2 * np.pi * 2.0 ** -25
        tol = (np.abs(a) + np.abs(b)) * m * (float(angle) + 2.5 * EPS32)
        tol = np.concatenate([tol, tol], -1) if not inter else np.repeat(tol, 2, -1)
        err = np.abs(f64(dst) - want)
        lim = np.zeros_like(want)
        lim[..., off:off + rot] = tol.astype(np.float64) + HALF[dtype] * np.abs(turned) * 1.01
        assert np.all(err <= lim), float((err - lim).max())


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("base,scaling,factor", [(10000.0, "plain", 1.0), (1e8, "plain", 1.0), (10000.0, "yarn", 40.0), (500000.0, "linear", 8.0)])
def test_rope_angles_of_every_position(csa2, base, scaling, factor, inter):
    """cos and sin of each position to its own bound: a frequency is rounded to 2^-52 of it and to 2^-65 turns, the reduced angle
    to fp32 (2^-26 turns); their own errors are 2 steps, and two products are rounded."""
    rot = 64
    pos = np.array([0, 1, -1, 2, 7, 100, -4095, 32767, 10 ** 5, 2 ** 20, -(2 ** 24) - 1, 10 ** 9, 2 ** 31 - 1, -2 ** 31])
    freqs, mag = csa2.rope_freqs(rot, base, scaling=scaling, factor=factor, orig_ctx=4096)
    x = torch.zeros((len(pos), rot), device="cuda")
    x[:, slice(0, None, 2) if inter else slice(0, rot // 2)] = 1.0          # pairs (1, 0): cos and sin come out
    out = torch.empty_like(x)
    csa2.rope([(x, out, 0)], i32(pos), freqs, mag=mag, interleaved=inter)
    t = pos.astype(np.longdouble)[:, None] * freqs.cpu().numpy().astype(np.longdouble)[None]
    off = np.abs(t) * 2.0 ** -52 + np.abs(pos)[:, None] * 2 * np.pi * 2.0 ** -65 + 2 * np.pi * 2.0 ** -26
    got = f64(out)
    c, s = (got[:, 0::2], got[:, 1::2]) if inter else (got[:, :rot // 2], got[:, rot // 2:])
    for have, want, other in ((c, np.cos(t), np.sin(t)), (s, np.sin(t), np.cos(t))):
        lim = mag * (off * (np.abs(other) + off) + 3.1 * EPS32 * np.abs(want))
        assert np.all(np.abs(have - want * mag) <= lim), float((np.abs(have - want * mag) - lim).max())


def test_rope_of_the_most_rows(csa2):
    """2^31 - 1 rows of one pair, in place (17 GB): the first, the last and some between."""
    rows = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    x = torch.zeros((rows, 2), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1.0
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    freqs = torch.tensor([0.5], dtype=torch.float64, device="cuda")
    csa2.rope([(x, x, 0)], pos, freqs)
    at = np.concatenate([np.arange(200), rows // 3 + np.arange(200), rows - 200 + np.arange(200)])
    got = f64(x[torch.as_tensor(at, device="cuda")])
    t = at.astype(np.longdouble) * 0.5
    # half a step of bf16, and the angle: 2^-52 of it and 2^-26 turns
    assert np.abs(got - np.stack([np.cos(t), np.sin(t)], 1)).max() <= 2.0 ** -8 * 0.5 + 2.0 ** 30 * 2.0 ** -52 + 1e-6


@pytest.mark.parametrize("dtype,dim,rot,off", [(torch.bfloat16, 192, 64, 128), (torch.float32, 20, 6, 5)])
def test_rope_in_place_equals_out_of_place_and_turns_back(csa2, dtype, dim, rot, off):
    g = torch.Generator().manual_seed(3)
    x = randn(g, (33, 16, dim), dtype)
    pos = torch.randint(0, 100000, (33,), generator=g, dtype=torch.int32).cuda()
    freqs, _ = csa2.rope_freqs(rot, 500000.0, scaling="ntk", factor=4.0)
    out, y = torch.empty_like(x), x.clone()
    csa2.rope([(x, out, off)], pos, freqs, mag=1.25)
    csa2.rope([(y, y, off)], pos, freqs, mag=1.25)
    assert torch.equal(out, y)
    csa2.rope([(y, y, off)], pos, freqs, mag=1.25, inverse=True)
    # two roundings to the type, each half a step of values up to 1.25 (|a| + |b|), and fp32 arithmetic
    lim = 3 * HALF[dtype] * float(x.abs().max()) * 2 * 1.25 + 1e-5
    assert float((y.float() - x.float()).abs().max()) <= lim
    assert torch.equal(y[..., :off], x[..., :off]) and torch.equal(y[..., off + rot:], x[..., off + rot:])


def test_rope_unaligned_tensors_and_offsets(csa2):
    g = torch.Generator().manual_seed(5)
    freqs, _ = csa2.rope_freqs(16)
    pos = i32(np.arange(6) * 1000)
    whole = randn(g, (6 * 8 * 32 + 1,), torch.bfloat16)
    x = whole[1:].view(6, 8, 32)                       # two bytes behind a 16-byte boundary
    a, b = torch.empty_like(x), torch.empty(6 * 8 * 32, dtype=torch.bfloat16, device="cuda").view(6, 8, 32)
    csa2.rope([(x, a, 16)], pos, freqs)
    csa2.rope([(x.clone(), b, 16)], pos, freqs)
    assert torch.equal(a, b)


# ------------------------------------------------------------------ tree attention

def make_parents(rng, S, T, roots=1):
    p = np.full((S, T), -1)
    for s in range(S):
        for t in range(min(roots, T), T):
            p[s, t] = rng.integers(max(0, t - 5), t)
    return p


def tree_inputs(sh, seed, fill=None, holes=0.0, roots=1, spread=4.0):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    dt = torch.float32 if sh.dtype == "f32" else torch.bfloat16
    B, T, N, W, K = sh.batch, sh.tokens, sh.n_entries, sh.swa, sh.topk
    S = B // T
    d = types.SimpleNamespace(dt=dt)
    d.q = randn(g, (B, sh.q_heads, sh.k_dim), dt)
    d.k_main, d.v_main = randn(g, (S, N, sh.k_dim), dt, np.sqrt(sh.k_dim) / spread), randn(g, (S, N, sh.v_dim), dt)
    d.k_swa, d.v_swa = randn(g, (S, W, sh.k_dim), dt, np.sqrt(sh.k_dim) / spread), randn(g, (S, W, sh.v_dim), dt)
    d.k_draft, d.v_draft = randn(g, (S, T, sh.k_dim), dt, np.sqrt(sh.k_dim) / spread), randn(g, (S, T, sh.v_dim), dt)
    idx = np.full((B, K), -1)
    for b in range(B):
        n = min(K, N) if holes == 0.0 else int(rng.integers(0, min(K, N) + 1))
        idx[b, :n] = np.sort(rng.choice(N, n, replace=False))
    d.idx = i32(idx)
    n_swa = rng.integers(0, W + 1, S) if fill is None else np.full(S, fill)
    d.n_swa = i32(n_swa)
    d.head = i32(np.where(n_swa == W, rng.integers(0, W, S), n_swa))
    d.parent = i32(make_parents(rng, S, T, roots))
    d.out = torch.full((B, sh.q_heads, sh.v_dim), 9.0, dtype=dt, device="cuda")
    d.lse = torch.full((B, sh.q_heads), 9.0, device="cuda")
    return d


def run_tree(csa2, sh, d, n_draft=None, parent="own", head="own"):
    sh, idx = padded(sh, d)
    ws = csa2.workspace(sh)
    p = d.parent if isinstance(parent, str) else parent
    h = d.head if isinstance(head, str) else head
    csa2.tree_attn(sh, d.q, d.k_main, d.v_main, idx, d.k_swa, d.v_swa, d.n_swa, d.k_draft, d.v_draft, d.out, ws,
                   swa_head=h, parent=p, n_draft=n_draft, lse=d.lse)
    return ws


def check_tree(sh, d, n_draft=None, parent=None, head=None):
    S = sh.batch // sh.tokens
    par = d.parent.cpu().numpy() if parent is None else parent
    hd = d.head.cpu().numpy() if head is None else head
    scale = sh.scale if sh.scale > 0 else 1.0 / np.sqrt(sh.k_dim)
    out, lse, absum, dot = R.tree_attention(f64(d.q), f64(d.k_main), f64(d.v_main), d.idx.cpu().numpy(), f64(d.k_swa),
                                            f64(d.v_swa), d.n_swa.cpu().numpy(), f64(d.k_draft), f64(d.v_draft), par,
                                            None if n_draft is None else n_draft.cpu().numpy(), hd, scale, sh.tokens)
    assert par.shape == (S, sh.tokens)
    got, gl = f64(d.out), f64(d.lse)
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(gl), empty)
    assert np.all(got[empty] == 0.0)
    # a logit: k_dim products summed in fp32, each addition half a step of at most the sum of |q k|
    logit = dot * (sh.k_dim + 4) * 2.0 ** -24
    # exp and log within 4 steps of a value up to |lse|, the sum of up to 1024 terms in fp32
    tol = 2 * logit + 8 * EPS32 * (1.0 + np.abs(lse[~empty])) + 64 * 2.0 ** -24
    assert np.all(np.abs(gl[~empty] - lse[~empty]) <= tol), float(np.abs(gl[~empty] - lse[~empty]).max())
    # a weight: twice the logit's error (itself and the sum), bf16: half a step of rounding; the output's own rounding
    rel = 4 * logit + 64 * EPS32 + (HALF[torch.bfloat16] if d.dt == torch.bfloat16 else 0.0) + sh.swa * 2.0 ** -24 + 512 * 2.0 ** -24
    lim = absum * rel * 1.01 + HALF[d.dt] * np.abs(out) * 1.01 + 1e-30
    err = np.abs(got - out)
    assert np.all(err <= lim), (float(err.max()), float((err - lim).max()))


FAST = dict(q_heads=64, k_dim=192, v_dim=128, dtype="bf16")

# Queries of a case by kernel: up to 384 slots a query's tokens are attended on the tensor cores by plan, alone (up to an SM
# each) or in pairs; with more slots few queries have a cluster of CTAs each, to which lists are padded here with -1.  Any
# other shape of bf16 rows in whole 8-byte pieces is of kind rows, the rest generic.
KINDS = {"clusters": (dict(FAST, pad=440), 1), "alone": (FAST, 1), "pairs": (FAST, 0), "rows": (dict(q_heads=20, k_dim=100, v_dim=72, dtype="bf16"), 1),
         "generic": (dict(q_heads=5, k_dim=24, v_dim=8, dtype="f32"), 1)}


def of_kind(kind, seqs, tokens, slots=100):
    """(shape arguments, sequences): enough of them for the kernel."""
    kw, few = KINDS[kind]
    ctas = -(-slots // 160)
    return kw, seqs if few else -(-(266 // ctas + 2) // tokens)


def padded(sh, d):
    """The shape and the lists of a call: sh.pad slots, -1 behind the list, where the shape has it."""
    pad = getattr(sh, "pad", 0)
    if not pad:
        return sh, d.idx
    more = torch.full((d.idx.shape[0], pad - sh.topk), -1, dtype=torch.int32, device="cuda")
    return types.SimpleNamespace(**{**vars(sh), "topk": pad}), torch.cat([d.idx, more], 1)


@pytest.mark.parametrize("S,T,N,K,W,roots,holes", [
    (1, 1, 40, 1, 1, 1, 0.0), (1, 8, 600, 512, 128, 1, 0.0), (3, 7, 700, 512, 128, 2, 1.0), (2, 33, 300, 99, 37, 1, 1.0),
    (1, 128, 64, 40, 128, 3, 0.0), (5, 2, 513, 512, 4, 1, 0.0), (65, 1, 96, 64, 16, 1, 1.0), (2, 64, 1024, 512, 8, 1, 0.0),
    (20, 16, 600, 512, 128, 2, 1.0), (1, 3, 1200, 1000, 24, 1, 0.0),
    # pairs of tokens on the tensor cores: odd token counts, one token, full and short lists, the longest ones
    (10, 7, 700, 512, 128, 1, 0.0), (67, 1, 513, 512, 128, 1, 1.0), (3, 33, 900, 512, 64, 3, 0.0), (1, 128, 700, 512, 128, 1, 1.0),
    (70, 1, 600, 512, 128, 1, 0.0), (1, 1, 300, 256, 128, 1, 0.0), (4, 9, 200, 99, 37, 2, 1.0), (19, 8, 700, 512, 128, 1, 0.0), (1, 1, 9, 1, 1, 1, 0.0),
    (51, 3, 700, 512, 128, 1, 1.0), (1, 60, 700, 512, 128, 1, 0.0), (2, 30, 700, 512, 128, 2, 1.0), (20, 2, 1100, 1000, 24, 1, 0.0), (90, 3, 30, 9, 7, 1, 1.0), (160, 2, 64, 40, 1, 1, 0.0)])
def test_tree_attention_fast_path(csa2, S, T, N, K, W, roots, holes):
    sh = shape(S * T, tokens=T, n_entries=N, topk=K, swa=W, **FAST)
    d = tree_inputs(sh, S * 1000 + T, holes=holes, roots=roots)
    ws = run_tree(csa2, sh, d)
    assert_no_device_error(csa2, ws)
    check_tree(sh, d)


@pytest.mark.parametrize("H,dk,dv,dtype", [(4, 16, 16, "f32"), (1, 1, 1, "f32"), (16, 64, 72, "bf16"), (40, 100, 33, "f32"),
                                           (9, 192, 128, "bf16"), (3, 1024, 1024, "bf16"), (64, 192, 128, "f32")])
@pytest.mark.parametrize("S,T,N,K,W", [(2, 5, 50, 33, 7), (1, 1, 9, 3, 4)])
def test_tree_attention_any_shape(csa2, H, dk, dv, dtype, S, T, N, K, W):
    sh = shape(S * T, tokens=T, n_entries=N, topk=K, swa=W, q_heads=H, k_dim=dk, v_dim=dv, dtype=dtype)
    d = tree_inputs(sh, H * 7 + T, holes=1.0)
    ws = run_tree(csa2, sh, d)
    assert_no_device_error(csa2, ws)
    check_tree(sh, d)


@pytest.mark.parametrize("H,dk,dv,dtype,S,T,N,K,W", [
    # bf16 rows in whole 8-byte pieces: few and many CTAs, part tiles of heads, slots and dims, the largest
    (4, 128, 128, "bf16", 2, 10, 600, 512, 128), (40, 100, 64, "bf16", 7, 18, 700, 512, 64), (17, 4, 4, "bf16", 3, 7, 90, 31, 17),
    (1, 20, 132, "bf16", 1, 1, 5, 1, 1), (33, 72, 16, "bf16", 10, 11, 65, 40, 9), (16, 1024, 1024, "bf16", 1, 2, 1500, 900, 124),
    (8, 192, 128, "bf16", 1, 128, 300, 99, 37),
    # the generic kernel: bf16 rows that are not, many CTAs of fp32, part fours of V dims
    (5, 18, 128, "bf16", 2, 9, 80, 33, 8), (5, 64, 7, "bf16", 30, 7, 80, 33, 8), (40, 100, 128, "f32", 4, 12, 600, 512, 37),
    (9, 130, 130, "f32", 3, 2, 1500, 900, 124), (12, 1024, 1024, "f32", 1, 2, 90, 65, 3), (3, 33, 260, "f32", 64, 1, 50, 13, 5)])
def test_tree_attention_other_shapes_by_kernel(csa2, H, dk, dv, dtype, S, T, N, K, W):
    sh = shape(S * T, tokens=T, n_entries=N, topk=K, swa=W, q_heads=H, k_dim=dk, v_dim=dv, dtype=dtype)
    d = tree_inputs(sh, H * 7 + T, holes=1.0)
    ws = run_tree(csa2, sh, d)
    assert_no_device_error(csa2, ws)
    check_tree(sh, d)


@pytest.mark.parametrize("off", [1, 2, 4])
def test_tree_attention_of_rows_at_any_address(csa2, off):
    """Caches that start `off` elements into an allocation: at 2, 4 and 8 bytes the kernels of each width."""
    sh = shape(6, tokens=3, n_entries=60, topk=33, swa=7, q_heads=6, k_dim=20, v_dim=12, dtype="bf16")
    d = tree_inputs(sh, 21, holes=1.0)
    for n in ("q", "k_main", "v_main", "k_swa", "v_swa", "k_draft", "v_draft"):
        t = getattr(d, n)
        moved = torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")[off:].view(t.shape)
        setattr(d, n, moved.copy_(t))
    ws = run_tree(csa2, sh, d)
    assert_no_device_error(csa2, ws)
    check_tree(sh, d)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("fill", [0, 1, 15, 16])
def test_tree_window_edges_and_chains(csa2, kind, fill):
    """Windows that are empty, filling and full, chains longer than the window, no parents and no heads given."""
    T = 24
    kw, S = of_kind(kind, 2, T)
    sh = shape(S * T, tokens=T, n_entries=80, topk=20, swa=16, **kw)
    d = tree_inputs(sh, 50 + fill, fill=fill)
    chain = np.tile(np.arange(T) - 1, (S, 1))
    run_tree(csa2, sh, d, parent=None)
    check_tree(sh, d, parent=chain)
    run_tree(csa2, sh, d, parent=i32(chain), head=None)
    check_tree(sh, d, parent=chain, head=np.zeros(S, dtype=int))


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("T,W", [(128, 128), (127, 40), (65, 70), (33, 1), (2, 3)])
def test_tree_paths_of_every_length(csa2, kind, T, W):
    """A chain given by its parents, one long branch with leaves, and parents that are not earlier tokens in its middle."""
    kw, S = of_kind(kind, 1, T)
    S = max(S, 3)
    sh = shape(S * T, tokens=T, n_entries=60, topk=12, swa=W, **{**kw, "pad": 440 if kind == "clusters" else 0})
    d = tree_inputs(sh, T)
    par = np.tile(np.arange(T) - 1, (S, 1))
    par[1] = np.where(np.arange(T) % 3 == 2, np.arange(T) - 2, np.arange(T) - 1)
    bad = T // 2
    given = par.copy()
    given[2, bad] = bad + 5                                # recorded, and a root
    par[2, bad] = -1
    d.parent.copy_(i32(given))
    ws = run_tree(csa2, sh, d)
    assert csa2.read_device_error(ws) == (-5, BAD_INDEX)
    check_tree(sh, d, parent=par)
    d.parent.copy_(i32(par))
    assert_no_device_error(csa2, run_tree(csa2, sh, d))
    check_tree(sh, d)


@pytest.mark.parametrize("kind,T,W", [(k, *x) for k, longest in (("clusters", 88), ("alone", 128), ("pairs", 128), ("rows", 128), ("generic", 128))
                                      for x in ((longest, 128), (longest - 1, 40), (65, 70), (33, 1), (2, 3))])
def test_tree_long_paths_in_the_kernel_of_each_kind(csa2, kind, T, W):
    """A chain given by its parents, a long branch with leaves and a parent that is not an earlier token, each alone in a call,
    in the kernel that is named: so few queries that every one has a cluster or an SM, or so many that they go in pairs.
    Clusters take 385 slots and more (three CTAs a query: up to 88 queries of 152 SMs), as one launch; plan and attention are two."""
    kw, _ = KINDS[kind]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    S = -(-(sms + 1) // T) if kind == "pairs" else 1
    assert kind != "clusters" or 8 * T * 3 <= 14 * sms
    sh = shape(S * T, tokens=T, n_entries=60, topk=12, swa=W, **{**kw, "pad": 400 - W if kind == "clusters" else 0})
    d = tree_inputs(sh, T)
    chain = np.arange(T) - 1
    branch = np.where(np.arange(T) % 3 == 2, np.arange(T) - 2, np.arange(T) - 1)
    cut = chain.copy()
    cut[T // 2] = -1
    for given, means in ((chain, chain), (branch, branch), (np.where(cut == chain, chain, T // 2 + 5), cut)):
        d.parent.copy_(i32(np.tile(given, (S, 1))))
        before = csa2.launch_count()
        ws = run_tree(csa2, sh, d)
        assert csa2.launch_count() - before == (2 if kind in ("alone", "pairs") else 1)
        if given is means:
            assert_no_device_error(csa2, ws)
        else:
            assert csa2.read_device_error(ws) == (-5, BAD_INDEX)
        check_tree(sh, d, parent=np.tile(means, (S, 1)))


@pytest.mark.parametrize("kind", list(KINDS))
def test_tree_rows_without_keys_and_dead_tokens(csa2, kind):
    T = 6
    kw, S = of_kind(kind, 3, T)
    sh = shape(S * T, tokens=T, n_entries=70, topk=40, swa=9, **kw)
    d = tree_inputs(sh, 77, holes=1.0)
    live = [(6, 1, 4)[s % 3] for s in range(S)]
    n_draft = i32(live)
    # what a dead token or an unused row holds must not matter
    nan = float("nan")
    n_swa, idx = d.n_swa.tolist(), d.idx.cpu()
    for s, n in enumerate(live):
        d.k_draft[s, n:], d.v_draft[s, n:] = nan, nan
        idx[s * T + n:(s + 1) * T] = -1
        d.k_swa[s, n_swa[s]:], d.v_swa[s, n_swa[s]:] = nan, nan
        free = sorted(set(range(70)) - set(idx[s * T:(s + 1) * T].flatten().tolist()))
        d.k_main[s, free], d.v_main[s, free] = nan, float("inf")
    d.idx.copy_(idx)
    dead = torch.arange(T, device="cuda") >= n_draft[:, None]
    d.q.view(S, T, sh.q_heads, -1)[dead] = nan
    ws = run_tree(csa2, sh, d, n_draft=n_draft)
    assert_no_device_error(csa2, ws)
    check_tree(sh, d, n_draft=n_draft)
    assert torch.isinf(d.lse.view(S, T, -1)[dead]).all() and (d.out.view(S, T, sh.q_heads, -1)[dead] == 0).all()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")])
def test_tree_values_of_one_token_stay_with_it(csa2, kind, what):
    """A value row that is not finite reaches the tokens that attend it and no others: a selected entry of one token, the
    drafted row of another."""
    T = 4
    kw, S = of_kind(kind, 2, T)
    sh = shape(S * T, tokens=T, n_entries=90, topk=20, swa=8, **kw)
    d = tree_inputs(sh, 5)
    d.parent.copy_(i32([[-1, 0, 0, 2]] * S))
    rng = np.random.default_rng(0)
    idx = np.stack([np.sort(rng.choice(80, 20, replace=False)) for _ in range(S * T)]).reshape(S, T, 20)
    idx[:, 1, 19] = 85                                     # token 1 alone selects entry 85
    d.idx.copy_(i32(idx.reshape(S * T, 20)))
    run_tree(csa2, sh, d)
    clean, lse = d.out.clone(), d.lse.clone()
    d.v_main[:, 85, 3] = what
    d.v_draft[:, 2, 1] = what                              # token 2 and its child 3
    run_tree(csa2, sh, d)
    out, was = d.out.view(S, T, sh.q_heads, -1), clean.view(S, T, sh.q_heads, -1)
    assert torch.equal(d.lse, lse)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[:, 1, :, 3] = True
    want[:, 2:, :, 1] = True
    assert torch.equal(bad, want)
    rest = out.masked_fill(want, 0).float() - was.masked_fill(want, 0).float()
    # Beside such a row an output may be computed again with unrounded weights: a weight's rounding moves a weighted mean
    # of the values by at most half a step of the largest, and both outputs are rounded once.
    most = max(float(x[x.isfinite()].abs().max()) for x in (d.v_main, d.v_swa, d.v_draft))
    lim = 3 * HALF[d.dt] * most + 1e-5
    assert float(rest.abs().max()) <= lim


@pytest.mark.parametrize("kind", list(KINDS))
def test_tree_scores_that_are_not_finite(csa2, kind):
    """A NaN key makes its tokens' heads NaN, as the definition does, and leaves the others alone."""
    T = 2
    kw, S = of_kind(kind, 2, T)
    sh = shape(S * T, tokens=T, n_entries=90, topk=20, swa=8, **kw)
    d = tree_inputs(sh, 6)
    idx = np.tile(np.arange(20), (S * T, 1)).reshape(S, T, 20)
    idx[:, 1, 19] = 85
    d.idx.copy_(i32(idx.reshape(S * T, 20)))
    d.k_main[:, 85] = float("nan")
    run_tree(csa2, sh, d)
    assert torch.isfinite(d.out.view(S, T, -1)[:, 0]).all() and torch.isfinite(d.lse.view(S, T, -1)[:, 0]).all()
    assert torch.isnan(d.out.view(S, T, -1)[:, 1]).all() and torch.isnan(d.lse.view(S, T, -1)[:, 1]).all()


@pytest.mark.parametrize("kind", list(KINDS))
def test_tree_scores_that_are_all_nan_make_lse_nan(csa2, kind):
    """A live token whose query is NaN, and a stretch of the window whose keys are: out and lse are NaN, as the definition has
    them, though no key or no key of a cluster's CTA scores a number.  -inf stays the lse of tokens that attend nothing."""
    T, W = 2, 8
    kw, S = of_kind(kind, 2, T)
    sh = shape(S * T, tokens=T, n_entries=90, topk=20, swa=W, **kw)
    d = tree_inputs(sh, 8, fill=W)
    d.parent.copy_(i32([[-1, -1]] * S))
    d.head.copy_(i32([0] * S))                             # newest committed row: W - 1
    q = d.q.clone()
    d.q.view(S, T, -1)[:, 1] = float("nan")
    assert_no_device_error(csa2, run_tree(csa2, sh, d))
    out, lse = d.out.view(S, T, -1), d.lse.view(S, T, -1)
    assert torch.isfinite(out[:, 0]).all() and torch.isfinite(lse[:, 0]).all()
    assert torch.isnan(out[:, 1]).all() and torch.isnan(lse[:, 1]).all()
    # Window slots are dealt to a cluster's CTAs in order, ceil(8 / CTAs) each, and the listed entries all lie with its first
    # CTA of three: slots 3 to 5 are all the keys that the second has.
    d.q.copy_(q)
    d.k_swa[:, W - 5:W - 2] = float("nan")
    assert_no_device_error(csa2, run_tree(csa2, sh, d))
    assert torch.isnan(d.out).all() and torch.isnan(d.lse).all()
    # and the weights of such a query say so
    weights = torch.empty((S * T, sh.topk), device="cuda")
    csa2.attn_weights(sh, d.q, d.k_main, d.idx, d.lse, weights, csa2.workspace(sh))
    assert torch.isnan(weights).all()
    n_draft = i32([0] * S)
    assert_no_device_error(csa2, run_tree(csa2, sh, d, n_draft=n_draft))
    assert (d.out == 0).all() and (d.lse == -float("inf")).all()


def test_tree_queries_that_are_nan_take_no_longer(csa2):
    """Rows whose scores are NaN are NaN and not computed again key by key: the call takes what it takes for numbers (best of
    five each, and a wide margin: key by key it was 240 times as long), beside one such query and with all."""
    S, T = 32, 16
    sh = shape(S * T, tokens=T, n_entries=2048, topk=512, swa=128, **FAST)
    d = tree_inputs(sh, 3)
    ws = csa2.workspace(sh)
    call = csa2.TreeAttnCall(sh, d.q, d.k_main, d.v_main, d.idx, d.k_swa, d.v_swa, d.n_swa, d.k_draft, d.v_draft, d.out, ws,
                             swa_head=d.head, parent=d.parent, lse=d.lse)

    def best():
        times = []
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            call()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    clean, out = best(), d.out.clone()
    assert torch.isfinite(out).all()
    d.q[7] = float("nan")
    one = best()
    assert torch.isnan(d.out[7]).all() and torch.isnan(d.lse[7]).all()
    rest = torch.arange(S * T, device="cuda") != 7
    assert torch.equal(d.out[rest], out[rest])
    d.q.fill_(float("nan"))
    most = best()
    assert torch.isnan(d.out).all() and torch.isnan(d.lse).all()
    assert_no_device_error(csa2, ws)
    assert max(one, most) <= 10 * clean, (clean, one, most)


@pytest.mark.parametrize("kind", list(KINDS))
def test_tree_bad_inputs_are_recorded(csa2, kind):
    T = 4
    kw, S = of_kind(kind, 2, T)
    sh = shape(S * T, tokens=T, n_entries=70, topk=10, swa=6, **kw)
    d = tree_inputs(sh, 9, fill=6)
    d.idx[3, 2] = 70                                       # an entry behind the cache
    ws = run_tree(csa2, sh, d)
    assert csa2.read_device_error(ws) == (-5, BAD_INDEX)
    check_tree(sh, d)
    d.idx[3, 2] = -7
    d.parent[1] = i32([-1, 1, 5, -9])                      # not earlier tokens: roots
    ws = run_tree(csa2, sh, d)
    assert csa2.read_device_error(ws) == (-5, BAD_INDEX)
    check_tree(sh, d)
    d.parent[1] = i32([-1, 0, 0, 1])
    d.n_swa[0] = 99                                        # clamped to the window
    d.head[1] = 6                                          # clamped to its last row
    ws = run_tree(csa2, sh, d)
    assert csa2.read_device_error(ws) == (-5, BAD_COUNT)
    d.n_swa[0], d.head[1] = 6, 5
    check_tree(sh, d)


@pytest.mark.parametrize("kind", ["clusters", "alone", "pairs"])
def test_tree_repeated_entries_count_each_time(csa2, kind):
    """The same index twice, and lists that do not ascend: as in csa2_sparse_attn."""
    kw, S = of_kind(kind, 2, 4)
    sh = shape(S * 4, tokens=4, n_entries=64, topk=48, swa=8, **kw)
    d = tree_inputs(sh, 13)
    rng = np.random.default_rng(4)
    d.idx.copy_(i32(rng.integers(-1, 64, (S * 4, 48))))
    ws = run_tree(csa2, sh, d)
    assert_no_device_error(csa2, ws)
    check_tree(sh, d)


@pytest.mark.parametrize("S,T", [(2, 6), (17, 4), (70, 1)])
def test_tree_large_logits(csa2, S, T):
    sh = shape(S * T, tokens=T, n_entries=600, topk=512, swa=128, **FAST)
    d = tree_inputs(sh, 21, spread=400.0)
    ws = run_tree(csa2, sh, d)
    assert_no_device_error(csa2, ws)
    assert torch.isfinite(d.out).all() and torch.isfinite(d.lse).all()
    out, lse, _, dot = R.tree_attention(f64(d.q), f64(d.k_main), f64(d.v_main), d.idx.cpu().numpy(), f64(d.k_swa), f64(d.v_swa),
                                        d.n_swa.cpu().numpy(), f64(d.k_draft), f64(d.v_draft), d.parent.cpu().numpy(), None,
                                        d.head.cpu().numpy(), 1 / np.sqrt(192), T)
    assert np.abs(f64(d.lse) - lse).max() <= dot * 196 * 2.0 ** -24 + 8 * EPS32 * np.abs(lse).max()


def test_chain_equals_steps_of_append_and_attention(csa2):
    """A chain of T drafted tokens gives what T steps of swa_append and sparse_attn give."""
    S, T, W = 3, 6, 8
    sh = shape(S * T, tokens=T, n_entries=200, topk=64, swa=W, **FAST)
    one = shape(S, n_entries=200, topk=64, swa=W, **FAST)
    d = tree_inputs(sh, 31, fill=5)
    run_tree(csa2, sh, d, parent=None)
    ws = csa2.workspace(one)
    ks, vs, head, n = d.k_swa.clone(), d.v_swa.clone(), d.head.clone(), d.n_swa.clone()
    pick = lambda x, t: x.view(S, T, *x.shape[1:])[:, t].contiguous()  # noqa: E731
    for t in range(T):
        csa2.swa_append(one, [(d.k_draft[:, t].contiguous(), d.v_draft[:, t].contiguous(), ks, vs)], head, n, ws)
        out = torch.empty((S, 64, 128), device="cuda")
        lse = torch.empty((S, 64), device="cuda")
        csa2.sparse_attn(one, pick(d.q, t), d.k_main, d.v_main, pick(d.idx, t), ks, vs, n, out, ws, lse=lse)
        # the same keys in another order: a bf16 rounding of each weight on both sides, then of the output
        assert float((pick(d.lse, t) - lse).abs().max()) <= 2e-5
        lim = 2.0 ** -8 * (2 * float(d.v_main.abs().max()) + out.abs()) + 1e-5
        assert bool(((pick(d.out, t).float() - out).abs() <= lim).all())
    # and committing the whole chain leaves the windows that the steps left
    kt, vt, ht, nt = d.k_swa.clone(), d.v_swa.clone(), d.head.clone(), d.n_swa.clone()
    path = i32(np.tile(np.arange(T), (S, 1)))
    csa2.tree_commit(sh, [(d.k_draft, d.v_draft, kt, vt, None, None)], path, i32([T] * S), ht, nt, None)
    assert torch.equal(kt, ks) and torch.equal(vt, vs) and torch.equal(ht, head) and torch.equal(nt, n)


@pytest.mark.parametrize("kind", list(KINDS))
def test_tree_and_weights_of_caches_beyond_32_bit_offsets(csa2, kind):
    """Rows that lie beyond 2^32 bytes of K and of V: bit for bit what the same rows give in a cache of 90 entries."""
    S, T = (2, 80) if kind == "pairs" else (1, 4)
    kw = KINDS[kind][0]
    sh = shape(S * T, tokens=T, n_entries=90, topk=20, swa=8, **kw)
    d = tree_inputs(sh, 3, holes=1.0)
    N = 2 ** 32 // (sh.v_dim * (4 if sh.dtype == "f32" else 2)) + 1000
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    lse = torch.full((S * T, sh.q_heads), 4.0, device="cuda")
    w = [torch.empty((S * T, 20), device="cuda") for _ in range(2)]
    assert_no_device_error(csa2, run_tree(csa2, sh, d))
    csa2.attn_weights(sh, d.q, d.k_main, d.idx, lse, w[0], csa2.workspace(sh))
    out, out_lse = d.out.clone(), d.lse.clone()
    check_tree(sh, d)
    far = torch.arange(90, device="cuda") * ((N - 1) // 89)
    for n in ("k_main", "v_main"):
        t = getattr(d, n)
        big = torch.zeros((S, N, t.shape[-1]), dtype=t.dtype, device="cuda")
        big[:, far] = t
        setattr(d, n, big)
    d.idx = torch.where(d.idx < 0, d.idx, far.int()[d.idx.clamp(min=0).long()])
    sh.n_entries = N
    d.out.fill_(9.0)
    ws = run_tree(csa2, sh, d)
    csa2.attn_weights(sh, d.q, d.k_main, d.idx, lse, w[1], ws)
    assert_no_device_error(csa2, ws)
    assert torch.equal(d.out, out) and torch.equal(d.lse, out_lse) and torch.equal(w[0], w[1])


# ------------------------------------------------------------------ attention weights

SHAPES = [(64, 192, "bf16"), (5, 24, "f32"), (16, 64, "bf16"), (1, 1, "f32"), (12, 1024, "bf16")]


@pytest.mark.parametrize("H,dk,dtype,S,T,N,K", [
    (*x, *y) for x in SHAPES for y in [(1, 1, 5, 1), (2, 3, 300, 130), (1, 2, 700, 512)]] + [
    (17, 4, "bf16", 3, 5, 90, 65), (40, 100, "bf16", 8, 16, 600, 256), (5, 18, "bf16", 2, 3, 300, 130),
    (40, 100, "f32", 8, 16, 600, 256)] + [
    # the fast shape in batches that fill the GPU: a tile or several a query, part tiles, more queries than CTAs
    (64, 192, "bf16", *y) for y in [(70, 1, 300, 130), (16, 5, 700, 512), (200, 1, 40, 9), (33, 9, 300, 128), (3, 50, 1100, 1000)]])
def test_attention_weights(csa2, H, dk, dtype, S, T, N, K):
    sh = shape(S * T, tokens=T, n_entries=N, topk=K, swa=4, q_heads=H, k_dim=dk, v_dim=16, dtype=dtype)
    d = tree_inputs(sh, 5 + H, holes=1.0)
    g = torch.Generator().manual_seed(1)
    lse = (torch.randn((S * T, H), generator=g) * 0.1 + np.log(K + 1.0)).cuda()
    lse[0, 0] = float("-inf")
    w = torch.full((S * T, K), 9.0, device="cuda")
    ws = csa2.workspace(sh)
    csa2.attn_weights(sh, d.q, d.k_main, d.idx, lse, w, ws)
    assert_no_device_error(csa2, ws)
    scale = 1 / np.sqrt(dk)
    want = R.attention_weights(f64(d.q), f64(d.k_main), d.idx.cpu().numpy(), f64(lse), scale, T)
    dot = float((np.abs(f64(d.q)).max(0).max(0) @ np.abs(f64(d.k_main)).reshape(-1, dk).max(0))) * scale
    # logits' fp32 sums, lse * log2(e) and the exponential's argument rounded, the heads added up
    rel = dot * (dk + 4) * 2.0 ** -24 + 16 * EPS32 * (4 + np.log(K + 1.0)) + H * 2.0 ** -24
    assert np.all(np.abs(f64(w) - want) <= want * rel + 1e-30)
    live = i32(np.arange(S * T) % 3 > 0)
    d.q[live == 0] = float("nan")
    d.idx[live == 0] = N
    w2 = torch.full_like(w, 9.0)
    csa2.attn_weights(sh, d.q, d.k_main, d.idx, lse, w2, ws, live=live)
    assert_no_device_error(csa2, ws)
    assert (w2[live == 0] == 0).all() and torch.equal(w2[live == 1], w[live == 1])


@pytest.mark.parametrize("H,dk,dtype,B", [(64, 192, "bf16", 3), (64, 192, "bf16", 200), (20, 100, "bf16", 3), (5, 18, "bf16", 3),
                                          (5, 24, "f32", 3)])
def test_heads_that_attended_nothing_add_nothing_whatever_they_hold(csa2, H, dk, dtype, B):
    """A head whose lse is -inf adds nothing though its query is NaN or infinite, nor though the row is; the heads beside
    it are not touched.  An lse of +inf, a score being so, stays the definition's NaN."""
    sh = shape(B, n_entries=200, topk=130, swa=4, q_heads=H, k_dim=dk, v_dim=16, dtype=dtype)
    d = tree_inputs(sh, 9)
    lse = torch.full((B, H), 6.0, device="cuda")
    lse[:, 1], lse[1] = float("-inf"), float("-inf")
    d.k_main[1, int(d.idx[1, 0])] = float("inf")           # of a query whose heads all are
    ws = csa2.workspace(sh)
    w = [torch.empty((B, 130), device="cuda") for _ in range(3)]
    q = d.q.clone()
    q[:, 1], q[1] = 0, 0
    csa2.attn_weights(sh, q, d.k_main, d.idx, lse, w[0], ws)
    q[:, 1, ::2], q[:, 1, 1::2], q[1] = float("nan"), float("inf"), float("-inf")
    csa2.attn_weights(sh, q, d.k_main, d.idx, lse, w[1], ws)
    assert_no_device_error(csa2, ws)
    assert torch.isfinite(w[1]).all() and torch.equal(w[0], w[1]) and (w[1][1] == 0).all() and (w[1][0] > 0).any()
    lse[0, 0], q[0, 0] = float("inf"), 0
    q[0, 0, 0] = 1.0
    d.k_main[0, int(d.idx[0, 0]), 0] = float("inf")
    csa2.attn_weights(sh, q, d.k_main, d.idx, lse, w[2], ws)
    assert torch.isnan(w[2][0, 0])


@pytest.mark.parametrize("B", [4, 90])
def test_attention_weights_of_a_whole_row_sum_to_the_heads(csa2, B):
    """With the window empty and one token, an attention's weights add up to the head count, less the token's own."""
    sh = shape(B, n_entries=600, topk=512, swa=128, **FAST)
    d = tree_inputs(sh, 8, fill=0)
    ws = run_tree(csa2, sh, d)
    w = torch.empty((B, 512), device="cuda")
    csa2.attn_weights(sh, d.q, d.k_main, d.idx, d.lse, w, ws)
    own = torch.exp((d.q.double() * d.k_draft.double()).sum(-1) / np.sqrt(192) - d.lse.double()).sum(1)
    assert float((w.double().sum(1) + own - 64).abs().max()) <= 64 * 1e-4
    d.idx[2, 5] = 600
    csa2.attn_weights(sh, d.q, d.k_main, d.idx, d.lse, w, ws)
    assert csa2.read_device_error(ws) == (-5, BAD_INDEX) and float(w[2, 5]) == 0.0


# ------------------------------------------------------------------ commit

def commit_inputs(S, T, L, N, K, W, dk, dv, dtype, seed):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    sh = shape(S * T, tokens=T, n_entries=N, topk=K, swa=W, k_dim=dk, v_dim=dv, dtype=dtype)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    d = types.SimpleNamespace(sh=sh)
    d.kd, d.vd = randn(g, (L, S, T, dk), dt), randn(g, (L, S, T, dv), dt)
    d.ks, d.vs = randn(g, (L, S, W, dk), dt), randn(g, (L, S, W, dv), dt)
    d.idx = i32(rng.integers(-1, N, (L, S * T, K)))         # unsorted, entries repeated
    d.w = torch.rand((L, S * T, K), generator=g).cuda()
    d.path = i32(np.stack([rng.permutation(T) for _ in range(S)]))
    d.n_path = i32(rng.integers(0, T + 1, S))
    n_swa = rng.integers(0, W + 1, S)
    d.n_swa, d.head = i32(n_swa), i32(np.where(n_swa == W, rng.integers(0, W, S), n_swa % W))
    d.mass = torch.randint(0, 2 ** 40, (S, N), generator=g).cuda()
    return d


def commit_reference(d, L, S, T, W, N):
    ks, vs, mass = d.ks.cpu().clone(), d.vs.cpu().clone(), d.mass.cpu().numpy().copy()
    head, n = d.head.cpu().numpy().copy(), d.n_swa.cpu().numpy().copy()
    idx, w = d.idx.cpu().numpy(), d.w.cpu().numpy()
    for s in range(S):
        for i in range(int(d.n_path[s])):
            t = int(d.path[s, i])
            if not 0 <= t < T:
                break
            for l in range(L):
                ks[l, s, head[s]], vs[l, s, head[s]] = d.kd[l, s, t].cpu(), d.vd[l, s, t].cpu()
                for j in range(idx.shape[2]):
                    e, x = idx[l, s * T + t, j], float(w[l, s * T + t, j])
                    if 0 <= e < N and 0 <= x <= 2 ** 20:
                        mass[s, e] += int(np.rint(np.float64(x) * 2.0 ** 32))
            head[s] = (head[s] + 1) % W
            n[s] = min(n[s] + 1, W)
    return ks, vs, mass, head, n


@pytest.mark.parametrize("S,T,L,N,K,W,dk,dv,dtype", [
    (1, 1, 1, 9, 3, 1, 192, 128, "bf16"), (4, 8, 4, 200, 64, 16, 192, 128, "bf16"), (3, 20, 11, 50, 30, 7, 24, 12, "f32"),
    (2, 128, 2, 40, 5, 37, 5, 3, "bf16"), (7, 3, 64, 33, 4, 8, 8, 8, "bf16")])
def test_tree_commit(csa2, S, T, L, N, K, W, dk, dv, dtype):
    d = commit_inputs(S, T, L, N, K, W, dk, dv, dtype, S * 10 + T)
    want = commit_reference(d, L, S, T, W, N)
    ws = csa2.workspace(d.sh)
    slots = [(d.kd[l], d.vd[l], d.ks[l], d.vs[l], d.idx[l], d.w[l]) for l in range(L)]
    csa2.tree_commit(d.sh, slots, d.path, d.n_path, d.head, d.n_swa, ws, mass=d.mass)
    assert_no_device_error(csa2, ws)
    for got, ref in zip((d.ks, d.vs, d.mass, d.head, d.n_swa), want):
        assert torch.equal(got.cpu(), torch.as_tensor(ref))


def test_tree_commit_bad_inputs(csa2):
    S, T, L, N, K, W = 3, 4, 2, 20, 6, 5
    d = commit_inputs(S, T, L, N, K, W, 16, 8, "bf16", 3)
    d.n_path.copy_(i32([4, 4, 3]))
    d.path[1, 2] = 4                                       # ends the path behind two tokens
    d.w[0, 0, 0], d.w[0, 0, 1], d.w[1, 0, 2] = float("nan"), -1.0, float("inf")
    d.idx[0, 0, :3] = 1
    d.idx[1, 0, 2], d.idx[1, 0, 3] = 1, N
    want = commit_reference(d, L, S, T, W, N)
    ws = csa2.workspace(d.sh)
    slots = [(d.kd[l], d.vd[l], d.ks[l], d.vs[l], d.idx[l], d.w[l]) for l in range(L)]
    csa2.tree_commit(d.sh, slots, d.path, d.n_path, d.head, d.n_swa, ws, mass=d.mass)
    assert csa2.read_device_error(ws) == (-5, BAD_INDEX | BAD_WEIGHT)
    for got, ref in zip((d.ks, d.vs, d.mass, d.head, d.n_swa), want):
        assert torch.equal(got.cpu(), torch.as_tensor(ref))
    # counts out of range are clamped; no mass, no weights, no workspace
    d.n_path[0], d.head[1], d.n_swa[2] = -3, 77, -1
    head, n, m = d.head.clone(), d.n_swa.clone(), d.mass.clone()
    csa2.read_static_device_error()
    csa2.tree_commit(d.sh, [x[:4] + (None, None) for x in slots], d.path, d.n_path, d.head, d.n_swa, None)
    assert csa2.read_static_device_error() == (-5, BAD_INDEX | BAD_COUNT)
    assert int(d.head[0]) == int(head[0]) and int(d.n_swa[0]) == int(n[0])
    assert int(d.head[1]) == (W - 1 + 2) % W and int(d.n_swa[2]) == 3 and torch.equal(m, d.mass)


def test_tree_commit_of_a_token_twice(csa2):
    """A path that names a token more than once pushes its rows and adds its weights each time; windows shorter than it."""
    S, T, L, N, K, W = 3, 9, 5, 300, 64, 4
    d = commit_inputs(S, T, L, N, K, W, 32, 16, "bf16", 4)
    d.path.copy_(i32([[2] * 9, [0, 1, 0, 1, 0, 1, 0, 1, 0], [8, 8, 7, 7, 8, 0, 0, 1, 1]]))
    d.n_path.copy_(i32([9, 8, 7]))
    want = commit_reference(d, L, S, T, W, N)
    ws = csa2.workspace(d.sh)
    csa2.tree_commit(d.sh, [(d.kd[l], d.vd[l], d.ks[l], d.vs[l], d.idx[l], d.w[l]) for l in range(L)], d.path, d.n_path, d.head,
                     d.n_swa, ws, mass=d.mass)
    assert_no_device_error(csa2, ws)
    for got, ref in zip((d.ks, d.vs, d.mass, d.head, d.n_swa), want):
        assert torch.equal(got.cpu(), torch.as_tensor(ref))


def test_tree_commit_rounds_weights_once(csa2):
    """Weights that end at, below and between the halves of 2^-32, whole and large ones, and entries selected twice by a
    token: rint(w 2^32) each, in integers (w 2^32 is exact in 64 bits)."""
    S, T, L, N, K, W = 1, 3, 11, 40, 32, 4
    d = commit_inputs(S, T, L, N, K, W, 16, 8, "bf16", 8)
    d.n_path.fill_(3)
    vals = [2.0 ** -33, 3 * 2.0 ** -33, 2.0 ** -33 * 1.0001, 2.0 ** -32, 1e-40, 0.0, 0.99999994, 1.0, 1.5, 63.999996, 64.00001,
            1000.3, 2.0 ** 20, 1048575.94, 2.0 ** -9 * 1.2345, 5 * 2.0 ** -33]
    d.w.copy_(torch.tensor(vals).repeat(d.w.numel() // len(vals)).view(d.w.shape))
    d.idx[:, :, 5:9] = d.idx[:, :, 4:5]                     # the same entry five times
    d.idx[3:, :, :] = d.idx[2:3]                            # layers that share a list
    want = commit_reference(d, L, S, T, W, N)
    ws = csa2.workspace(d.sh)
    csa2.tree_commit(d.sh, [(d.kd[l], d.vd[l], d.ks[l], d.vs[l], d.idx[l], d.w[l]) for l in range(L)], d.path, d.n_path, d.head,
                     d.n_swa, ws, mass=d.mass)
    assert_no_device_error(csa2, ws)
    assert torch.equal(d.mass.cpu(), torch.as_tensor(want[2]))


def test_tree_commit_saturates_the_mass(csa2):
    """A mass ends at 2^63 - 1 and does not wrap: sums that end below, at and beyond it, by one weight and by many, from
    masses that are great, small and below zero, and the eviction that follows keeps such an entry."""
    S, T, L, N, K, W = 2, 128, 9, 12, 10, 4
    d = commit_inputs(S, T, L, N, K, W, 16, 8, "bf16", 12)
    most, unit = 2 ** 63 - 1, 2 ** 32
    d.n_path.copy_(i32([1, 128]))
    d.path.copy_(i32(np.tile(np.arange(T), (S, 1))))
    d.idx.copy_(torch.arange(K, dtype=torch.int32, device="cuda").expand_as(d.idx))
    d.w.fill_(1.0)                                         # 9 units in sequence 0, 1,152 in sequence 1
    d.w[:, T:, 7] = 2.0 ** 20                              # 1,152 * 2^52: past 2^62, not 2^63
    d.w[:, T:, 8] = 2.0 ** 20
    for s, n in ((0, 9), (1, 1152)):
        d.mass[s] = torch.tensor([most, most - n * unit, most - n * unit + 1, most - n * unit - 1, most - unit, -2 ** 63, -5, 0,
                                  2 ** 62, 3, most, 0])
    before = d.mass.cpu().numpy().copy()
    ws = csa2.workspace(d.sh)
    csa2.tree_commit(d.sh, [(d.kd[l], d.vd[l], d.ks[l], d.vs[l], d.idx[l], d.w[l]) for l in range(L)], d.path, d.n_path, d.head,
                     d.n_swa, ws, mass=d.mass)
    assert_no_device_error(csa2, ws)
    for s, n in ((0, 9), (1, 1152)):
        add = [n * unit] * K + [0, 0]
        if s == 1:
            add[7] = add[8] = n * 2 ** 52
        assert d.mass[s].tolist() == [min(int(b) + a, most) for b, a in zip(before[s], add)], s
    sh = shape(S, n_entries=N, k_dim=16, v_dim=8, idx_dim=8)
    k, v, x = (torch.zeros((S, N, z), dtype=torch.bfloat16, device="cuda") for z in (16, 8, 8))
    kept, n_valid = torch.empty((S, N), dtype=torch.int32, device="cuda"), i32([N, N])
    mass = d.mass.cpu().numpy()
    csa2.kv_evict(sh, 4, 4, 0, 0, k, v, x, d.mass, n_valid, kept, None)
    for s in range(S):
        assert kept[s, :4].tolist() == R.evict(N, 4, 4, 0, 0, mass[s])
        assert 0 in kept[s, :4].tolist()                   # the greatest before the commit still is


# ------------------------------------------------------------------ eviction

def evict_inputs(S, N, dk, dv, dI, block, dtype, seed, kind, n_valid=None):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    d = types.SimpleNamespace(sh=shape(S, n_entries=N, k_dim=dk, v_dim=dv, idx_dim=dI, block=block, dtype=dtype))
    d.k, d.v, d.x = randn(g, (S, N, dk), dt), randn(g, (S, N, dv), dt), randn(g, (S, N, dI), dt, 0.25)
    m = {"spread": lambda: rng.integers(0, 2 ** 40, (S, N)), "ties": lambda: rng.integers(0, 4, (S, N)),
         "equal": lambda: np.full((S, N), 5), "zero": lambda: np.zeros((S, N), dtype=np.int64),
         "wide": lambda: rng.integers(-2 ** 63, 2 ** 63 - 1, (S, N)),
         "rising": lambda: np.tile(np.arange(N), (S, 1)), "falling": lambda: np.tile(-np.arange(N), (S, 1)),
         "offset": lambda: 2 ** 40 + rng.integers(0, 1000, (S, N)), "below": lambda: -2 ** 62 + rng.integers(0, 2 ** 50, (S, N)),
         "edges": lambda: rng.choice(np.array([-2 ** 63, 2 ** 63 - 1, -1, 0, 1, 2, 3, 4, 5, 7, 8, 2 ** 31, 2 ** 32 - 1, 2 ** 32, 2 ** 62,
                                               2 ** 62 - 1, 3 * 2 ** 61, -2 ** 62], dtype=np.int64), (S, N))}[kind]()
    d.mass = torch.as_tensor(np.asarray(m, dtype=np.int64)).cuda()
    d.n = i32(rng.integers(0, N + 1, S) if n_valid is None else n_valid)
    return d


def check_evict(d, before, got, kept, kb, args, rounded=True, untouched=None):
    """`before`, `got`: (k, v, x, mass, n) host copies; untouched: what rows behind the last hold."""
    trigger, keep, sink, recent = args
    N, block = d.sh.n_entries, d.sh.block
    for s in range(d.sh.batch):
        n = int(before[4][s])
        ids = R.evict(n, trigger, keep, sink, recent, before[3][s].numpy())
        assert int(got[4][s]) == len(ids)
        assert kept[s].tolist() == ids + [-1] * (N - len(ids)), s
        for a, b in zip(got[:4], before[:4]):
            assert torch.equal(a[s, :len(ids)], b[s][ids]), s
        if n > trigger or untouched is not None:
            assert not got[3][s, len(ids):].any()
        if untouched is not None:
            for a, u in zip(got[:3], untouched):
                assert torch.equal(a[s, len(ids):], u[s, len(ids):])
        if kb is not None and (n > trigger or untouched is not None):
            want = R.block_means(before[2][s][ids].double().numpy() if ids else np.zeros((0, d.sh.idx_dim)), len(ids), block, rounded)
            mean = f64(kb[s])
            assert np.abs(mean[len(want):]).max(initial=0.0) == 0.0
            tol = 0.0 if rounded else (HALF[kb.dtype] + 8 * EPS32) * np.abs(want) + 8 * EPS32
            if rounded:                                    # a mean within fp32 rounding of a half may go either way
                raw = R.block_means(before[2][s][ids].double().numpy() if ids else np.zeros((0, d.sh.idx_dim)), len(ids), block, False)
                near = np.abs(np.abs(raw - np.floor(raw)) - 0.5) < 1e-5
                assert np.all((mean[:len(want)] == want) | near)
            else:
                assert np.all(np.abs(mean[:len(want)] - want) <= tol)


def host(*ts):
    return tuple(t.cpu().clone() for t in ts)


CASES = [(3, 40, 30, 2, 5, "spread"), (1, 9, 1, 0, 0, "ties"), (4, 700, 512, 16, 100, "ties"), (2, 129, 128, 0, 0, "equal"),
         (2, 5000, 777, 0, 0, "wide"), (1, 30000, 20000, 16, 1024, "spread"), (2, 600, 100, 60, 40, "spread"),
         (3, 300, 299, 0, 1, "zero"), (2, 300, 200, 3, 0, "rising"), (2, 300, 200, 0, 3, "falling"), (1, 20001, 19000, 1, 1, "zero"),
         (2, 3000, 1500, 5, 7, "offset"), (1, 40000, 33333, 2, 3, "offset"), (2, 2000, 900, 0, 0, "edges"), (1, 40000, 11111, 2, 3, "edges"),
         (3, 1500, 40, 0, 0, "edges"), (1, 9000, 8000, 0, 9, "below"), (2, 100, 60, 30, 30, "spread")]


@pytest.mark.parametrize("S,N,keep,sink,recent,kind", CASES)
@pytest.mark.parametrize("in_place", [False, True])
def test_kv_evict(csa2, S, N, keep, sink, recent, kind, in_place):
    d = evict_inputs(S, N, 192, 128, 64, 8, "bf16", N + S, kind, n_valid=[N] + list(np.random.default_rng(N).integers(0, N + 1, S - 1)))
    run_evict(csa2, d, (keep, keep, sink, recent), in_place)


def run_evict(csa2, d, args, in_place, rounded=True, with_kb=True):
    S, N = d.sh.batch, d.sh.n_entries
    nb = -(-N // d.sh.block)
    before = host(d.k, d.v, d.x, d.mass, d.n)
    kept = torch.full((S, N), 99, dtype=torch.int32, device="cuda")
    kb = torch.full((S, nb, d.sh.idx_dim), 99.0, dtype=d.k.dtype, device="cuda") if with_kb else None
    ws = csa2.workspace(d.sh)
    call = dict(kb=kb, round_to_int=rounded)
    if in_place:
        csa2.kv_evict(d.sh, *args, d.k, d.v, d.x, d.mass, d.n, kept, ws, **call)
        got, untouched = host(d.k, d.v, d.x, d.mass, d.n), None
        for s in range(S):
            if int(before[4][s]) <= args[0]:
                assert all(torch.equal(a[s], b[s]) for a, b in zip(got, before))
                assert kb is None or bool((kb[s] == 99).all())
    else:
        outs = [torch.full_like(t, 3) for t in (d.k, d.v, d.x, d.mass, d.n)]
        untouched = host(*outs[:3])
        csa2.kv_evict(d.sh, *args, d.k, d.v, d.x, d.mass, d.n, kept, ws, out=outs, **call)
        got = host(*outs)
        assert all(torch.equal(a, b) for a, b in zip(host(d.k, d.v, d.x, d.mass, d.n), before))
    assert_no_device_error(csa2, ws)
    check_evict(d, before, got, kept.cpu(), None if kb is None else kb.cpu(), args, rounded, untouched)
    if with_kb:   # bit for bit what csa2_block_keys gives
        x, n = (d.x, d.n) if in_place else (outs[2], outs[4])
        ref = torch.empty_like(kb)
        csa2.block_keys(d.sh, x, n, ref, ws, round_to_int=rounded)
        for s in range(S):
            if not in_place or int(before[4][s]) > args[0]:
                assert torch.equal(kb[s], ref[s])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dk,dv,dI,block,dtype", [(5, 3, 1, 3, "bf16"), (20, 12, 8, 16, "f32"), (7, 7, 7, 1, "f32"),
                                                  (64, 72, 64, 300, "bf16"), (1024, 1, 16, 8, "bf16")])
def test_kv_evict_any_shape(csa2, dk, dv, dI, block, dtype, in_place):
    d = evict_inputs(3, 203, dk, dv, dI, block, dtype, dk, "ties", n_valid=[203, 150, 20])
    run_evict(csa2, d, (140, 120, 4, 9), in_place, rounded=False)


@pytest.mark.parametrize("N,keep", [(400001, 300000), (250000, 100), (200000, 199999)])
def test_kv_evict_long_caches(csa2, N, keep):
    """Caches whose masses fit the shared memory of 8 CTAs, of 16, or of none."""
    d = evict_inputs(1, N, 8, 4, 2, 8, "bf16", N, "ties" if keep > 1000 else "spread", n_valid=[N])
    run_evict(csa2, d, (keep, keep, 3, 7), False)


def test_kv_evict_counts_and_no_workspace(csa2):
    d = evict_inputs(3, 50, 16, 16, 8, 8, "bf16", 2, "spread", n_valid=[99, -4, 50])
    csa2.read_static_device_error()
    kept = torch.empty((3, 50), dtype=torch.int32, device="cuda")
    csa2.kv_evict(d.sh, 40, 30, 0, 0, d.k, d.v, d.x, d.mass, d.n, kept, None)
    assert csa2.read_static_device_error() == (-5, BAD_COUNT)
    assert d.n.tolist() == [30, 0, 30]


@pytest.mark.parametrize("in_place", [False, True])
def test_kv_evict_of_a_cache_beyond_32_bit_offsets(csa2, in_place):
    """K, V and indexer keys of more than 2^32 bytes each, masses of more than any cluster keeps."""
    N, keep = 2 ** 32 // 256 + 4099, 2 ** 32 // 256 - 100001
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    sh = shape(1, n_entries=N, topk=8, swa=4, k_dim=128, v_dim=128, idx_dim=128)
    e = torch.arange(N, device="cuda")
    ins = [torch.empty((1, N, 128), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    for i, x in enumerate(ins):                            # a row says which entry it is, in digits that bf16 holds
        x.zero_()
        for c in range(4):
            x[0, :, 31 * c + i] = ((e >> (7 * c)) & 127).to(torch.bfloat16)
    mass = torch.where(e % 3 == 0, 5, 1 + e % 2)[None].contiguous()
    ins += [mass, i32([N])]
    kept = torch.empty((1, N), dtype=torch.int32, device="cuda")
    kb = torch.empty((1, -(-N // 8), 128), dtype=torch.bfloat16, device="cuda")
    outs = ins if in_place else [torch.zeros_like(t) for t in ins]
    sink, recent = 1000, 5000
    mid = e[sink:N - recent]
    order = torch.sort(mass[0][mid], descending=True, stable=True).indices[:keep - sink - recent]
    want = torch.cat([e[:sink], torch.sort(mid[order]).values, e[N - recent:]])
    was = mass.clone()
    csa2.kv_evict(sh, keep, keep, sink, recent, *ins, kept, None, kb=kb, out=None if in_place else outs)
    assert int(outs[4][0]) == keep and torch.equal(kept[0, :keep].long(), want) and bool((kept[0, keep:] == -1).all())
    assert torch.equal(outs[3][0, :keep], was[0][want]) and not outs[3][0, keep:].any()
    for i in range(3):
        for c in range(4):
            assert torch.equal(outs[i][0, :keep, 31 * c + i].float(), ((want >> (7 * c)) & 127).float())
    x = outs[2][0, :keep // 8 * 8, 2].float().view(-1, 8).mean(1)
    assert torch.equal(kb[0, :keep // 8, 2].float(), x.round().to(torch.bfloat16).float())


# ------------------------------------------------------------------ together

def step_state(csa2, seed):
    S, T = 3, 6
    sh = shape(S * T, tokens=T, n_entries=256, topk=64, swa=16, **FAST)
    one = shape(S, n_entries=256, topk=64, swa=16, **FAST)
    d = tree_inputs(sh, seed, fill=16)
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    d.n_valid = i32([256, 251, 200])
    for s in range(S):
        for t in range(T):
            d.idx[s * T + t] = i32(np.sort(rng.choice(200, 64, replace=False)))
    d.qr, d.kr = torch.empty_like(d.q), torch.empty_like(d.k_draft)
    par = d.parent.cpu().numpy()
    depth = np.array([[len(R.path_of(par[s], t)) - 1 for t in range(T)] for s in range(S)])
    d.pos = i32((1000 + depth).reshape(-1))
    d.freqs, _ = csa2.rope_freqs(64)
    # k_draft [S, T, dk] as rows of one head
    d.k_draft = d.k_draft.view(S * T, -1)
    d.kr = d.kr.view(S * T, -1)
    paths = [R.path_of(par[s], T - 1)[::-1] for s in range(S)]
    d.path = i32([p + [0] * (T - len(p)) for p in paths])
    d.n_path = i32([len(p) for p in paths])
    live = np.zeros((S, T))
    for s, p in enumerate(paths):
        live[s, p] = 1
    d.live = i32(live.reshape(-1))
    d.w = torch.empty((S * T, 64), device="cuda")
    d.mass = torch.zeros((S, 256), dtype=torch.int64, device="cuda")
    d.k_idx = randn(g, (S, 256, 64), torch.bfloat16)
    d.kept = torch.empty((S, 256), dtype=torch.int32, device="cuda")
    d.kb = torch.zeros((S, 32, 64), dtype=torch.bfloat16, device="cuda")
    return sh, one, d


def run_step(csa2, sh, one, d, ws, ws1):
    """Positions, attention, the accepted queries' weights, the commit and the eviction, on the current stream."""
    csa2.rope([(d.q, d.qr, 128), (d.k_draft, d.kr, 128)], d.pos, d.freqs, interleaved=True)
    kr = d.kr.view(sh.batch // sh.tokens, sh.tokens, -1)
    csa2.tree_attn(sh, d.qr, d.k_main, d.v_main, d.idx, d.k_swa, d.v_swa, d.n_swa, kr, d.v_draft, d.out, ws,
                   swa_head=d.head, parent=d.parent, lse=d.lse)
    csa2.attn_weights(sh, d.qr, d.k_main, d.idx, d.lse, d.w, ws, live=d.live)
    csa2.tree_commit(sh, [(kr, d.v_draft, d.k_swa, d.v_swa, d.idx, d.w)], d.path, d.n_path, d.head, d.n_swa, ws, mass=d.mass)
    csa2.kv_evict(one, 250, 200, 4, 32, d.k_main, d.v_main, d.k_idx, d.mass, d.n_valid, d.kept, ws1, kb=d.kb)


STATE = ("qr", "kr", "out", "lse", "w", "k_swa", "v_swa", "head", "n_swa", "mass", "k_main", "v_main", "k_idx", "n_valid", "kept", "kb")


def test_a_step_of_all_operators(csa2):
    """Eager on the current stream, eager on another stream, and captured and replayed: the same state, and the attention,
    the mass and the eviction are what the definitions give on the step's own intermediate results."""
    sh, one, a = step_state(csa2, 17)
    before = {k: getattr(a, k).clone() for k in ("k_swa", "v_swa", "n_swa", "head", "k_main", "v_main", "k_idx", "mass", "n_valid")}
    ws, ws1 = csa2.workspace(sh), csa2.workspace(one)
    run_step(csa2, sh, one, a, ws, ws1)
    assert_no_device_error(csa2, ws)
    assert_no_device_error(csa2, ws1)
    # attention on the turned queries and keys
    ref = types.SimpleNamespace(**vars(a))
    ref.q, ref.k_draft = a.qr, a.kr.view(3, 6, -1)
    for k in ("k_swa", "v_swa", "n_swa", "head", "k_main", "v_main"):
        setattr(ref, k, before[k])
    check_tree(sh, ref)
    # the mass of the accepted queries, then the eviction by it
    mass = np.zeros((3, 256), dtype=np.int64)
    w, idx, live = a.w.cpu().numpy(), a.idx.cpu().numpy(), a.live.cpu().numpy()
    for b in range(18):
        if live[b]:
            for j in range(64):
                mass[b // 6, idx[b, j]] += int(np.rint(np.float64(w[b, j]) * 2.0 ** 32))
        else:
            assert not w[b].any()
    for s, n in enumerate([256, 251, 200]):
        ids = R.evict(n, 250, 200, 4, 32, mass[s])
        assert a.kept[s, :len(ids)].tolist() == ids
        assert a.mass[s, :len(ids)].tolist() == mass[s][ids].tolist()
        assert torch.equal(a.k_main[s, :len(ids)], before["k_main"][s][ids])
    assert a.n_valid.tolist() == [200, 200, 200]

    _, _, b = step_state(csa2, 17)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_step(csa2, sh, one, b, ws, ws1)
    torch.cuda.synchronize()
    for k in STATE:
        assert torch.equal(getattr(a, k), getattr(b, k)), k

    _, _, c = step_state(csa2, 17)
    first = {k: getattr(c, k).clone() for k in STATE}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_step(csa2, sh, one, c, ws, ws1)
    for _ in range(2):
        for k in STATE:
            getattr(c, k).copy_(first[k])
        graph.replay()
        torch.cuda.synchronize()
        for k in STATE:
            assert torch.equal(getattr(a, k), getattr(c, k)), k


def test_calls_on_two_streams_at_once(csa2):
    """The persistent and the cluster kernels of two streams, each with its own workspace and state, give what they give
    one after the other."""
    def state(seed):
        sh = shape(40 * 16, tokens=16, n_entries=600, topk=512, swa=64, **FAST)
        d = tree_inputs(sh, seed)
        d.w = torch.empty((640, 512), device="cuda")
        d.mass = torch.zeros((40, 600), dtype=torch.int64, device="cuda")
        d.path = i32(np.tile(np.arange(16), (40, 1)))
        d.n_path = i32([16] * 40)
        d.one = shape(40, n_entries=600, topk=512, swa=64, **FAST)
        d.k_idx = torch.zeros((40, 600, 64), dtype=torch.bfloat16, device="cuda")
        d.kept = torch.empty((40, 600), dtype=torch.int32, device="cuda")
        d.n_valid = i32([600] * 40)
        return sh, d, csa2.workspace(sh), csa2.workspace(d.one)

    def run(sh, d, ws, ws1):
        csa2.tree_attn(sh, d.q, d.k_main, d.v_main, d.idx, d.k_swa, d.v_swa, d.n_swa, d.k_draft, d.v_draft, d.out, ws,
                       swa_head=d.head, parent=d.parent, lse=d.lse)
        csa2.attn_weights(sh, d.q, d.k_main, d.idx, d.lse, d.w, ws)
        csa2.tree_commit(sh, [(d.k_draft, d.v_draft, d.k_swa, d.v_swa, d.idx, d.w)], d.path, d.n_path, d.head, d.n_swa, ws, mass=d.mass)
        csa2.kv_evict(d.one, 500, 400, 4, 32, d.k_main, d.v_main, d.k_idx, d.mass, d.n_valid, d.kept, ws1)

    alone = [state(31), state(32)]
    for x in alone:
        run(*x)
    torch.cuda.synchronize()
    both = [state(31), state(32)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for x, st in zip(both, streams):
        with torch.cuda.stream(st):
            run(*x)
    torch.cuda.synchronize()
    for x, y in zip(alone, both):
        for ws in x[2:] + y[2:]:
            assert_no_device_error(csa2, ws)
        for k in ("out", "lse", "w", "mass", "k_swa", "v_swa", "head", "n_swa", "k_main", "v_main", "kept", "n_valid"):
            assert torch.equal(getattr(x[1], k), getattr(y[1], k)), k


@pytest.mark.parametrize("S,T", [(3, 6), (40, 8)])
def test_steps_back_to_back_with_the_indexing_between(csa2, S, T):
    """Several steps as a server runs them, positions and evictions in place, with the calls that read some inputs before the
    launch in front of them is over (index_topk the queries behind rope, sparse_attn the windows behind a commit, index_topk the
    keys behind an eviction): the same as with a wait behind every call, and as a replayed graph."""
    N, K, W, B = 1024, 128, 16, S * T
    sh = shape(B, tokens=T, n_entries=N, topk=K, swa=W, **FAST)
    one = shape(S, n_entries=N, topk=K, swa=W, **FAST)
    g = torch.Generator().manual_seed(S)
    src = tree_inputs(sh, 40 + S, fill=W)
    src.k_draft = src.k_draft.view(B, -1)
    src.q_idx, src.w_idx = randn(g, (B, 8, 64), torch.bfloat16), torch.rand((B, 8), generator=g).cuda()
    src.k_idx, src.k1 = randn(g, (S, N, 64), torch.bfloat16), randn(g, (S, 64, 192), torch.bfloat16)
    src.n_query, src.n_valid = i32([N - 300] * B), i32([N] * S)
    src.pos, src.live = i32(np.arange(B) * 37), i32(np.arange(B) % 3 == 0)
    src.path, src.n_path = i32(np.tile(np.arange(T), (S, 1))), i32(np.arange(S) % (T + 1))
    src.weights = torch.empty((B, K), device="cuda")
    src.mass = torch.zeros((S, N), dtype=torch.int64, device="cuda")
    src.kept, src.kb = torch.empty((S, N), dtype=torch.int32, device="cuda"), torch.zeros((S, N // 8, 64), dtype=torch.bfloat16, device="cuda")
    src.idx1 = src.idx.view(S, T, K)[:, 0].contiguous()
    src.out1, src.lse1 = torch.empty((S, 64, 128), device="cuda"), torch.empty((S, 64), device="cuda")
    freqs, _ = csa2.rope_freqs(64)
    tensors = {k: v for k, v in vars(src).items() if isinstance(v, torch.Tensor)}

    def copy():
        return types.SimpleNamespace(**{k: v.clone() for k, v in tensors.items()})

    ws, ws1 = csa2.workspace(sh), csa2.workspace(one)

    def run(d, wait):
        for step in range(4):
            for call in (
                    lambda: csa2.rope([(d.q, d.q, 128), (d.k_draft, d.k_draft, 128), (d.q_idx, d.q_idx, 0)], d.pos, freqs),
                    lambda: csa2.index_topk(sh, d.q_idx, d.w_idx, d.k_idx, d.n_query, K, d.idx, ws),
                    lambda: csa2.tree_attn(sh, d.q, d.k_main, d.v_main, d.idx, d.k_swa, d.v_swa, d.n_swa, d.k_draft.view(S, T, -1),
                                           d.v_draft, d.out, ws, swa_head=d.head, parent=d.parent, lse=d.lse),
                    lambda: csa2.attn_weights(sh, d.q, d.k_main, d.idx, d.lse, d.weights, ws, live=d.live),
                    lambda: csa2.tree_commit(sh, [(d.k_draft.view(S, T, -1), d.v_draft, d.k_swa, d.v_swa, d.idx, d.weights)], d.path,
                                             d.n_path, d.head, d.n_swa, ws, mass=d.mass),
                    lambda: csa2.sparse_attn(one, d.k1, d.k_main, d.v_main, d.idx1, d.k_swa, d.v_swa, d.n_swa, d.out1, ws1, lse=d.lse1),
                    lambda: csa2.kv_evict(one, N - 1, N - 100 - step, 4, 32, d.k_main, d.v_main, d.k_idx, d.mass, d.n_valid, d.kept, ws1,
                                          kb=d.kb),
                    lambda: csa2.index_topk(one, d.q_idx.view(S, T, 8, 64)[:, 0].contiguous(), d.w_idx.view(S, T, 8)[:, 0].contiguous(),
                                            d.k_idx, d.n_valid, K, d.idx1, ws1),
                    lambda: d.n_valid.fill_(N)):
                call()
                if wait:
                    torch.cuda.synchronize()

    a = copy()
    run(a, True)
    assert torch.isfinite(a.out).all() and torch.isfinite(a.out1).all() and int(a.mass.max()) > 0
    for _ in range(5):
        b = copy()
        torch.cuda.synchronize()
        run(b, False)
        torch.cuda.synchronize()
        for k in tensors:
            assert torch.equal(getattr(a, k), getattr(b, k)), k
    c = copy()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(c, False)
    for _ in range(3):
        for k, v in tensors.items():
            getattr(c, k).copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for k in tensors:
            assert torch.equal(getattr(a, k), getattr(c, k)), k
    assert_no_device_error(csa2, ws)
    assert_no_device_error(csa2, ws1)
