"""The 4-bit main cache (csa2_kv4_append, csa2_kv4_rows, csa2_kv4_attn) and the norm with rotary positions (csa2_norm_rope)
on the GPU against plain 64-bit definitions, alone and as a serving step runs them together."""
import types

import numpy as np
import pytest

from tests import draft_reference as D
from tests import kv4_reference as R
from tests.gpu_helpers import assert_no_device_error, lib_ready, need_gpu, torch

pytestmark = pytest.mark.gpu

BAD_INDEX, BAD_COUNT = 1, 2
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a rounding step, relative
EPS32 = 2.0 ** -23
FAST = dict(q_heads=64, k_dim=192, v_dim=128, dtype="bf16")


@pytest.fixture(scope="module")
def csa2():
    need_gpu()
    return lib_ready()


def shape(batch, **kw):
    d = dict(batch=batch, n_entries=64, idx_heads=8, idx_dim=64, block=8, pool_blocks=0, topk=512, q_heads=64, k_dim=192,
             v_dim=128, swa=128, scale=0.0, relu=1, dtype="bf16", tokens=1)
    d.update(kw)
    return types.SimpleNamespace(**d)


def dtype_of(sh):
    return torch.float32 if sh.dtype == "f32" else torch.bfloat16


def randn(g, size, dtype, mul=1.0):
    return (torch.randn(size, generator=g) * mul).to(dtype).cuda()


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def f64(t):
    return t.detach().cpu().double().numpy()


# ------------------------------------------------------------------ norm with rotary positions

def norm_case(csa2, dtype, rows, heads, dim, rot, off, inter=False, center=False, each=False, fused=False, seed=0, gain=True):
    g = torch.Generator().manual_seed(seed + rows * 31 + dim)
    if fused:
        whole = randn(g, (rows, (heads + 2) * dim + 8), dtype, 1.5)
        xs = [whole[:, :heads * dim].unflatten(1, (heads, dim)), whole[:, (heads + 1) * dim:(heads + 2) * dim]]
    else:
        xs = [randn(g, (rows, heads, dim), dtype, 1.5) + 0.5, randn(g, (rows, dim), dtype, 0.01)]
    gains = [(1 + 0.3 * torch.randn((heads, dim) if each else (dim,), generator=g)).cuda(),
             (1 + 0.3 * torch.randn((dim,), generator=g)).cuda()] if gain else [None, None]
    outs = [torch.full(x.shape, 7.0, dtype=dtype, device="cuda") for x in xs]
    pos = torch.randint(0, 2 ** 20, (rows,), generator=g, dtype=torch.int32)
    pos[0] = 2 ** 31 - 1
    if rows > 2:
        pos[1], pos[2] = -12345, 0
    freqs, mag = csa2.rope_freqs(rot, scaling="yarn", factor=8.0, orig_ctx=4096) if rot else (None, 1.0)
    args = dict(pos=pos.cuda() if rot else None, freqs=freqs, mag=mag, eps=1e-5, norm="layer" if center else "rms", interleaved=inter)
    return xs, outs, gains, [off, off], args, pos


def check_norm(xs, outs, gains, offs, args, pos, dtype):
    rot = 0 if args["freqs"] is None else 2 * args["freqs"].shape[0]
    inter, mag = args["interleaved"], args["mag"]
    t = pos.numpy().astype(np.longdouble)[:, None] * args["freqs"].cpu().numpy().astype(np.longdouble)[None] if rot else None
    for x, out, gain, off in zip(xs, outs, gains, offs):
        if x.dim() == 2:
            x, out = x[:, None], out[:, None]
        dim = x.shape[-1]
        gn = np.ones(dim) if gain is None else f64(gain)
        want, plain = R.norm_rope(f64(x), gn, args["eps"], args["norm"] == "layer", t, mag, off, inter)
        # Sums of dim squares: a lane adds at most 32 of them, then 5 more, each addition half a step of a positive sum; the square
        # root halves it; division, root, the gain and the products are rounded once each.
        rel = (38 / 2 + 6) * 2.0 ** -24
        lim = rel * np.abs(plain)
        if args["norm"] == "layer":   # the mean: 37 additions of |x| (about the same lanes), its division and the subtraction, relative to |x|
            x64 = f64(x)
            inv = 1.0 / np.sqrt(x64.var(-1, keepdims=True) + args["eps"])
            lim = lim + (40 * 2.0 ** -24) * (np.abs(x64).mean(-1, keepdims=True) + np.abs(x64)) * inv * np.abs(gn)
        if rot:
            at = np.arange(rot).reshape(-1, 2).T if inter else np.arange(rot).reshape(2, -1)
            a, b = at + off
            # the angle: 2^-52 of it from the frequency's rounding, 2^-25 turns in fp32; cos and sin 2 ulp; three roundings
            angle = float(np.abs(t).max()) * 2.0 ** -51 + 2 * np.pi * 2.0 ** -25
            both = mag * ((np.abs(plain[..., a]) + np.abs(plain[..., b])) * (angle + 2.5 * EPS32) + lim[..., a] + lim[..., b])
            lim[..., a] = both
            lim[..., b] = both
        lim = lim * 1.01 + HALF[dtype] * np.abs(want) * 1.01 + 1e-30
        err = np.abs(f64(out) - want)
        assert np.all(err <= lim), (float(err.max()), float((err - lim).max()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rows,heads,dim,rot,off", [
    (1, 1, 2, 2, 0), (3, 64, 192, 64, 128), (5, 8, 64, 64, 0), (17, 3, 40, 8, 32), (2, 5, 10, 6, 3), (700, 4, 96, 16, 0),
    (4, 128, 1024, 1024, 0), (9, 2, 24, 12, 8), (33, 5, 64, 8, 56), (6, 3, 36, 24, 4), (3000, 1, 40, 40, 0), (5000, 1, 64, 8, 0),
    (2000, 2, 12, 4, 8), (7, 6, 512, 64, 448), (8, 3, 768, 256, 0), (3, 1, 1000, 10, 990), (5, 1, 1, 0, 0), (66, 7, 128, 0, 0),
    (2, 2, 48, 0, 0), (700, 65, 192, 192, 0)])
def test_norm_rope_matches_definition(csa2, dtype, inter, rows, heads, dim, rot, off):
    for center, each in ((False, False), (True, True)):
        xs, outs, gains, offs, args, pos = norm_case(csa2, dtype, rows, heads, dim, rot, off, inter, center, each)
        csa2.norm_rope(list(zip(xs, outs, gains, offs)), **args)
        check_norm(xs, outs, gains, offs, args, pos, dtype)


@pytest.mark.parametrize("dtype,dim,rot,off", [(torch.bfloat16, 192, 64, 128), (torch.float32, 128, 128, 0), (torch.bfloat16, 20, 6, 5),
                                               (torch.float32, 20, 20, 0), (torch.bfloat16, 44, 8, 36)])
@pytest.mark.parametrize("inter", [False, True])
def test_norm_rope_of_parts_of_a_projection(csa2, dtype, dim, rot, off, inter):
    """Queries and keys that lie in one projection's rows, into arrays of their own and in place; what lies between stays."""
    xs, outs, gains, offs, args, pos = norm_case(csa2, dtype, 37, 5, dim, rot, off, inter, fused=True, gain=dim != 44)
    whole = xs[0]._base if xs[0]._base is not None else xs[0]
    before = whole.clone()
    csa2.norm_rope(list(zip(xs, outs, gains, offs)), **args)
    check_norm(xs, outs, gains, offs, args, pos, dtype)
    assert torch.equal(whole, before)
    csa2.norm_rope(list(zip(xs, xs, gains, offs)), **args)
    assert torch.equal(xs[0], outs[0]) and torch.equal(xs[1], outs[1])
    mid = slice(5 * dim, 6 * dim)
    assert torch.equal(whole[:, mid], before[:, mid]) and torch.equal(whole[:, 7 * dim:], before[:, 7 * dim:])


def test_norm_rope_unaligned_and_mixed_tensors(csa2):
    """An address two bytes off, and tensors of several types and sizes in one call: each as it is alone."""
    g = torch.Generator().manual_seed(5)
    freqs, _ = csa2.rope_freqs(16)
    pos = i32(np.arange(6) * 1000)
    gain = (torch.rand(33, generator=g) + 0.5).cuda()
    cases = []
    for dtype, heads, dim, off, shift in ((torch.bfloat16, 8, 32, 16, 1), (torch.bfloat16, 8, 32, 16, 0), (torch.float32, 3, 32, 0, 0),
                                          (torch.float32, 3, 32, 0, 1), (torch.bfloat16, 1, 64, 48, 4), (torch.float32, 70, 20, 3, 0)):
        x = randn(g, (6 * heads * dim + shift,), dtype)[shift:].view(6, heads, dim)
        cases.append((x, torch.empty_like(x), gain[1:33] if dim == 32 and shift else None, off))
    csa2.norm_rope(cases, pos, freqs)
    for x, out, w, off in cases:
        alone = torch.empty((6, x.shape[1], x.shape[2]), dtype=x.dtype, device="cuda")
        csa2.norm_rope([(x, alone, w, off)], pos, freqs)
        assert torch.equal(out, alone)
        want, _ = R.norm_rope(f64(x), np.ones(x.shape[2]) if w is None else f64(w), 1e-6, False,
                              pos.cpu().numpy()[:, None].astype(np.longdouble) * freqs.cpu().numpy()[None], 1.0, off, False)
        assert np.abs(f64(out) - want).max() <= HALF[x.dtype] * np.abs(want).max() + 1e-4 * (x.dtype == torch.bfloat16) + 1e-5


def test_norm_rope_of_zeros_large_and_non_finite_heads(csa2):
    """A head of zeros gives zeros (NaN without eps), others are not touched by a neighbour's NaN or infinity."""
    x = torch.randn((4, 6, 64), generator=torch.Generator().manual_seed(1)).cuda()
    ref = torch.empty_like(x)
    csa2.norm_rope([(x, ref, None, 0)])
    y = x.clone()
    y[0, 0], y[1, 1, 5], y[2, 2, 60], y[3, 3] = 0.0, float("nan"), float("inf"), 1e18
    out = torch.empty_like(y)
    csa2.norm_rope([(y, out, None, 0)])
    odd = torch.zeros((4, 6), dtype=torch.bool)
    odd[0, 0] = odd[1, 1] = odd[2, 2] = odd[3, 3] = True
    assert torch.equal(out[~odd.cuda()], ref[~odd.cuda()])
    assert not out[0, 0].any() and out[1, 1].isnan().all() and out[2, 2, 60].isnan()
    assert torch.allclose(out[3, 3], torch.ones(64, device="cuda"), atol=1e-6)
    csa2.norm_rope([(y, out, None, 0)], eps=0.0)
    assert out[0, 0].isnan().all()


def test_norm_rope_of_far_rows(csa2):
    """Row strides that take the last rows beyond 2^32 bytes."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    rows, wide = 4500, 1 << 20
    whole = torch.zeros((rows, wide), dtype=torch.bfloat16, device="cuda")
    x = whole[:, 64:64 + 4 * 192].unflatten(1, (4, 192))
    near = randn(torch.Generator().manual_seed(3), (rows, 4, 192), torch.bfloat16)
    x.copy_(near)
    freqs, _ = csa2.rope_freqs(64)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    a, b = torch.empty_like(near), torch.empty_like(near)
    csa2.norm_rope([(x, a, None, 128)], pos, freqs)
    csa2.norm_rope([(near, b, None, 128)], pos, freqs)
    assert torch.equal(a, b)
    csa2.norm_rope([(x, x, None, 128)], pos, freqs)
    assert torch.equal(x, b) and not whole[:, :64].any() and not whole[:, 64 + 4 * 192:].any()


def test_norm_rope_refusals_of_tensors(csa2):
    x = torch.zeros((4, 3, 16), device="cuda")
    for slots, kw in (([(x, x.clone(), None, 0)], dict(pos=i32([0] * 4))), ([], {}), ([(x, x.clone()[:, :2], None, 0)], {}),
                      ([(x.transpose(1, 2), x.clone(), None, 0)], {}), ([(x, x.bfloat16(), None, 0)], {}),
                      ([(x.double(), x.double(), None, 0)], {}), ([(x, x.clone(), torch.ones(15, device="cuda"), 0)], {}),
                      ([(x, x.clone(), None, 0)], dict(norm="batch")), ([(x.cpu(), x.clone(), None, 0)], {})):
        with pytest.raises((ValueError, TypeError)):
            csa2.norm_rope(slots, **kw)
    with pytest.raises(csa2.CSA2Error):
        csa2.norm_rope([(x[:0], x[:0], None, 0)])


# ------------------------------------------------------------------ packed entries

def new_entries(sh, M, seed, spread=True):
    """k_new, v_new, kidx_new whose groups differ in size, some of zeros, some with ties at every border."""
    rng = np.random.default_rng(seed)
    dt = dtype_of(sh)
    B = sh.batch
    out = []
    for d, exp in ((sh.k_dim, sh.k_exp), (sh.v_dim, sh.v_exp)):
        x = rng.standard_normal((B, M, d))
        if spread:
            x *= np.exp2(rng.integers(-14, 13, (B, M, d // 16 + 1)))[..., np.arange(d) // 16]
        ties = rng.random((B, M)) < 0.3                    # numbers on the borders between two codes, of a group whose scale is exact
        edge = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.0, -0.25, -1.75, -5.0], (B, M, d))
        edge[..., ::16] = 6.0
        s = np.exp2(rng.integers(-7, 8, (B, M, 1))) * (1 + rng.integers(0, 8, (B, M, 1)) / 8)
        x = np.where(ties[..., None], edge * s, x)
        x[rng.random((B, M)) < 0.05] = 0.0
        out.append(torch.tensor(x * 2.0 ** exp, dtype=torch.float32).to(dt).cuda())
    return out + [torch.tensor(rng.integers(-4, 5, (B, M, sh.idx_dim)), dtype=torch.float32).to(dt).cuda()]


def packed_reference(sh, k, v):
    return R.pack(f64(k), f64(v), sh.k_exp, sh.v_exp)


def append_state(csa2, sh, M, seed, n_valid, n_new):
    g = torch.Generator().manual_seed(seed)
    dt, B, N = dtype_of(sh), sh.batch, sh.n_entries
    s = types.SimpleNamespace()
    s.k_new, s.v_new, s.x_new = new_entries(sh, M, seed)
    s.kv = torch.randint(0, 256, (B, N, csa2.kv4_bytes(sh)), generator=g, dtype=torch.uint8).cuda()
    s.k_idx = torch.randint(-4, 5, (B, N, sh.idx_dim), generator=g).to(dt).cuda()
    s.kb = torch.full((B, -(-N // sh.block), sh.idx_dim), 9.0, dtype=dt, device="cuda")
    s.n_valid, s.n_new = i32(n_valid), i32(n_new)
    return s


def run_append(csa2, sh, s, ws=None, **kw):
    csa2.kv4_append(sh, s.n_new, s.k_new, s.v_new, s.x_new, s.kv, s.k_idx, s.kb, s.n_valid, ws, k_exp=sh.k_exp, v_exp=sh.v_exp, **kw)


def check_append(sh, s, before, rounded=True, every=1):
    """The written entries byte for byte, everything else as it was."""
    for b in range(sh.batch):
        n0, m = int(before.n_valid[b]), int(before.n_new[b])
        m = min(m, sh.n_entries - n0)
        assert int(s.n_valid[b]) == n0 + m
        want, got = before.kv[b].clone(), s.kv[b]
        want[n0:n0 + m] = got[n0:n0 + m]
        assert torch.equal(want, got)
        packed = got[n0:n0 + m].cpu().numpy()
        for j in range(0, m, every):
            ref = packed_reference(sh, s.k_new[b, j], s.v_new[b, j])
            have = packed[j].copy()
            g = 8 * (R.groups(sh.k_dim) + R.groups(sh.v_dim))
            for part in (have, ref):                       # a zero's sign bit is free
                low, high = part[:g] & 15, part[:g] >> 4
                part[:g] = np.where(low == 8, 0, low) | np.where(high == 8, 0, high) << 4
            assert np.array_equal(have, ref), (b, j)
        x = before.k_idx[b].clone()
        x[n0:n0 + m] = s.x_new[b, :m]
        assert torch.equal(s.k_idx[b], x)
        kb = f64(before.kb[b])
        if m:
            mean = D.block_means(f64(x), n0 + m, sh.block, rounded)
            j0, j1 = n0 // sh.block, (n0 + m - 1) // sh.block
            kb[j0:j1 + 1] = mean[j0:j1 + 1]
        err = np.abs(f64(s.kb[b]) - kb)
        assert np.all(err <= HALF[dtype_of(sh)] * np.abs(kb) * (not rounded) * 1.01 + (1e-6 if not rounded else 0.0))


def clone(s):
    return types.SimpleNamespace(**{k: v.clone() for k, v in vars(s).items()})


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,M,dk,dv,dI,block,k_exp,v_exp", [
    (3, 64, 1, 192, 128, 64, 8, 0, 0), (2, 100, 33, 192, 128, 64, 8, -2, 3), (4, 77, 77, 64, 64, 32, 4, 5, -7), (2, 50, 20, 100, 72, 5, 3, 0, 0),
    (1, 40, 40, 1, 1, 1, 1, 0, 0), (2, 90, 70, 17, 40, 8, 100, 2, 2), (1, 20, 3, 1024, 1024, 1024, 8, 0, -64), (5, 33, 2, 16, 16, 64, 16, 64, 0),
    (1, 300, 299, 48, 80, 64, 7, -3, 1)])
def test_kv4_append(csa2, B, N, M, dk, dv, dI, block, k_exp, v_exp, dtype):
    sh = shape(B, n_entries=N, k_dim=dk, v_dim=dv, idx_dim=dI, block=block, dtype=dtype, topk=4, swa=4, k_exp=k_exp, v_exp=v_exp)
    rng = np.random.default_rng(B * N + M)
    n_new = rng.integers(0, M + 1, B)
    n_new[0] = M
    s = append_state(csa2, sh, M, N + M, rng.integers(0, N - M + 1, B), n_new)
    before, ws = clone(s), csa2.workspace(sh)
    rounded = B % 2 == 1
    run_append(csa2, sh, s, ws, round_to_int=rounded)
    assert_no_device_error(csa2, ws)
    check_append(sh, s, before, rounded)


def test_kv4_append_of_prompts(csa2):
    """Prompts of many tiles of entries, into caches that hold some already and into empty ones; and as many small steps."""
    sh = shape(3, n_entries=3001, topk=4, swa=4, k_exp=0, v_exp=0)
    s = append_state(csa2, sh, 2900, 5, [0, 101, 13], [2900, 2900, 1111])
    before, ws = clone(s), csa2.workspace(sh)
    run_append(csa2, sh, s, ws)
    assert_no_device_error(csa2, ws)
    check_append(sh, s, before, every=41)
    steps = clone(before)
    for lo in range(0, 2900, 290):
        n = (before.n_new - lo).clamp(0, 290).to(torch.int32)
        part = types.SimpleNamespace(**{**vars(steps), "n_new": n, **{k: getattr(before, k)[:, lo:lo + 290].contiguous() for k in ("k_new", "v_new", "x_new")}})
        run_append(csa2, sh, part, ws)
    for k in ("kv", "k_idx", "kb", "n_valid"):
        assert torch.equal(getattr(steps, k), getattr(s, k)), k


def test_kv4_append_counts_and_no_workspace(csa2):
    """Counts outside their ranges are clamped and recorded, entries behind the cache's end dropped; without a workspace the
    static error word has them."""
    sh = shape(4, n_entries=24, topk=4, swa=4, k_exp=0, v_exp=0)
    csa2.read_static_device_error()
    for M, ws in ((5, csa2.workspace(sh)), (60, csa2.workspace(sh)), (5, None)):
        s = append_state(csa2, sh, M, 9, [22, -3, 24, 30], [5, 2, 1, 99])
        before = clone(s)
        run_append(csa2, sh, s, ws)
        st, bits = csa2.read_device_error(ws) if ws is not None else csa2.read_static_device_error()
        assert st == -5 and bits == BAD_COUNT
        before.n_valid, before.n_new = i32([22, 0, 24, 24]), i32([5, 2, 1, 5])
        check_append(sh, s, before)
    s = append_state(csa2, sh, 3, 9, [0, 5, 24, 21], [0, 0, 0, 3])
    before = clone(s)
    s.kb, before_kb = None, before.kb
    run_append(csa2, sh, s)
    s.kb = before_kb.clone()
    s.kb[3, 2] = torch.round(s.k_idx[3, 16:24].float().mean(0)).to(s.kb.dtype)   # (what a kb would hold)
    check_append(sh, s, before)
    assert csa2.read_static_device_error() == (0, 0)


def test_kv4_append_unaligned(csa2):
    """New rows and caches of indexer keys at any element's address."""
    for off in (1, 2, 4):
        sh = shape(2, n_entries=40, topk=4, swa=4, k_exp=0, v_exp=0)
        s = append_state(csa2, sh, 37, off, [1, 3], [37, 30])
        for n in ("k_new", "v_new", "x_new", "k_idx", "kb"):
            t = getattr(s, n)
            setattr(s, n, torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")[off:].view(t.shape).copy_(t))
        before = clone(s)
        run_append(csa2, sh, s)
        check_append(sh, s, before)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_kv4_groups_that_are_not_finite_read_as_nan(csa2, dtype):
    sh = shape(1, n_entries=8, topk=4, swa=4, k_dim=48, v_dim=20, dtype=dtype, k_exp=0, v_exp=10)
    s = append_state(csa2, sh, 4, 1, [2], [4])
    s.k_new[0, 0, 17], s.k_new[0, 1, 47], s.v_new[0, 2, 19] = float("nan"), float("inf"), float("-inf")
    s.v_new[0, 3, 0] = 3e38 if dtype == "f32" else 2.0 ** 127   # finite, saturates
    run_append(csa2, sh, s)
    k, v = torch.empty((1, 4, 48), dtype=dtype_of(sh), device="cuda"), torch.empty((1, 4, 20), dtype=dtype_of(sh), device="cuda")
    csa2.kv4_rows(sh, s.kv, i32([[2, 3, 4, 5]]), k, v, None, k_exp=0, v_exp=10)
    bad = torch.zeros((4, 48), dtype=torch.bool)
    bad[0, 16:32] = bad[1, 32:48] = True
    assert torch.equal(k[0].isnan().cpu(), bad)
    bad = torch.zeros((4, 20), dtype=torch.bool)
    bad[2, 16:] = True
    assert torch.equal(v[0].isnan().cpu(), bad) and float(v[0, 3, 0]) == 2688.0 * 1024


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,N,Rn,dk,dv,k_exp,v_exp", [
    (1, 1, 1, 1, 192, 128, 0, 0), (6, 3, 70, 33, 192, 128, -2, 5), (4, 1, 50, 700, 64, 64, 0, 0), (2, 2, 20, 5, 100, 72, 64, -64), (3, 1, 9, 4, 1, 1, 0, 0),
    (2, 1, 12, 9, 1024, 1024, 0, 0), (5, 1, 30, 40, 17, 40, 0, 0), (700, 7, 40, 64, 40, 24, 1, 1)])
def test_kv4_rows(csa2, B, T, N, Rn, dk, dv, k_exp, v_exp, dtype):
    """Any bytes as entries: every code and scale, rows of any order and repeated, none, and behind the cache."""
    sh = shape(B, tokens=T, n_entries=N, k_dim=dk, v_dim=dv, dtype=dtype, topk=4, swa=4)
    rng = np.random.default_rng(B + N)
    kv = rng.integers(0, 256, (B // T, N, R.entry_bytes(dk, dv)), dtype=np.uint8)
    g = 8 * (R.groups(dk) + R.groups(dv))
    kv[..., g:] &= 0x7f                                    # scales are not negative
    idx = rng.integers(-2, N, (B, Rn))
    idx[0, 0] = N + 5
    ws = csa2.workspace(sh)
    k, v = (torch.full((B, Rn, d), 7.0, dtype=dtype_of(sh), device="cuda") for d in (dk, dv))
    csa2.kv4_rows(sh, torch.tensor(kv).cuda(), i32(idx), k, v, ws, k_exp=k_exp, v_exp=v_exp)
    st, bits = csa2.read_device_error(ws)
    assert st == -5 and bits == BAD_INDEX
    known = {}
    for b in range(0, B, max(1, B // 20)):
        for j in range(Rn):
            e = idx[b, j]
            if not 0 <= e < N:
                assert not k[b, j].any() and not v[b, j].any()
                continue
            if (b // T, e) not in known:
                known[b // T, e] = R.unpack(kv[b // T, e], dk, dv, k_exp, v_exp)
            for have, want in zip((f64(k[b, j]), f64(v[b, j])), known[b // T, e]):
                assert np.array_equal(have, want, equal_nan=True)


def test_kv4_rows_at_unaligned_outputs(csa2):
    sh = shape(2, n_entries=30, topk=4, swa=4)
    kv = torch.randint(0, 126, (2, 30, 192), dtype=torch.uint8, generator=torch.Generator().manual_seed(1)).cuda()
    idx = i32(np.arange(22).reshape(2, 11))
    want = [torch.empty((2, 11, d), dtype=torch.bfloat16, device="cuda") for d in (192, 128)]
    csa2.kv4_rows(sh, kv, idx, *want, None)
    got = [torch.empty(2 * 11 * d + 1, dtype=torch.bfloat16, device="cuda")[1:].view(2, 11, d) for d in (192, 128)]
    csa2.kv4_rows(sh, kv, idx, *got, None)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


# ------------------------------------------------------------------ attention

def attn_inputs(csa2, sh, seed, holes=1.0, fill=None, loud=1.2):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    dt = dtype_of(sh)
    B, T, N, W, K = sh.batch, sh.tokens, sh.n_entries, sh.swa, sh.topk
    S = B // T
    ke, ve = getattr(sh, "k_exp", 0), getattr(sh, "v_exp", 0)
    d = types.SimpleNamespace(dt=dt, k_exp=ke, v_exp=ve)
    codes = rng.integers(0, 256, (S, N, R.entry_bytes(sh.k_dim, sh.v_dim)), dtype=np.uint8)
    gr = 8 * (R.groups(sh.k_dim) + R.groups(sh.v_dim))
    codes[..., gr:] = rng.integers(0x24, 0x30, codes[..., gr:].shape)   # scales of 0.19 to 0.47
    d.kv = torch.tensor(codes).cuda()
    d.q = randn(g, (B, sh.q_heads, sh.k_dim), dt, loud * 2.0 ** -ke)
    d.k_swa, d.v_swa = randn(g, (B, W, sh.k_dim), dt, 2.0 ** ke), randn(g, (B, W, sh.v_dim), dt, 2.0 ** ve)
    idx = np.full((B, K), -1)
    for b in range(B):
        n = min(K, N) if holes == 0.0 else int(rng.integers(0, min(K, N) + 1))
        at = np.sort(rng.choice(K, n, replace=False)) if holes > 1.0 else np.arange(n)   # holes > 1: -1 between entries too
        idx[b, at] = np.sort(rng.choice(N, n, replace=False))
    d.idx = i32(idx)
    d.n_swa = i32(rng.integers(0, W + 1, B) if fill is None else np.full(B, fill))
    d.out = torch.full((B, sh.q_heads, sh.v_dim), 9.0, dtype=dt, device="cuda")
    d.lse = torch.full((B, sh.q_heads), 9.0, device="cuda")
    return d


def run_attn(csa2, sh, d, ws=None):
    ws = csa2.workspace(sh) if ws is None else ws
    csa2.kv4_attn(sh, d.q, d.kv, d.idx, d.k_swa, d.v_swa, d.n_swa, d.out, ws, lse=d.lse, k_exp=d.k_exp, v_exp=d.v_exp)
    return ws


def numbers(sh, d):
    """The whole cache as numbers [S, N, d], by the reference's tables."""
    kv = d.kv.cpu().numpy().astype(np.int64)
    gk, gv = R.groups(sh.k_dim), R.groups(sh.v_dim)
    g = gk + gv
    codes = np.stack([kv[..., :8 * g] & 15, kv[..., :8 * g] >> 4], -1).reshape(*kv.shape[:2], g, 16)
    b = kv[..., 8 * g:9 * g]
    x = R.LEVELS[codes % 8] * np.where(codes >= 8, -1.0, 1.0) * np.where(b == 127, np.nan, R.SCALES[np.minimum(b, 126)])[..., None]
    k = x[:, :, :gk].reshape(*kv.shape[:2], -1)[..., :sh.k_dim] * 2.0 ** d.k_exp
    return k, x[:, :, gk:].reshape(*kv.shape[:2], -1)[..., :sh.v_dim] * 2.0 ** d.v_exp


def check_attn(sh, d):
    scale = sh.scale if sh.scale > 0 else 1.0 / np.sqrt(sh.k_dim)
    k, v = numbers(sh, d)
    out, lse, absum, dot = R.attention(f64(d.q), k, v, d.idx.cpu().numpy(), f64(d.k_swa), f64(d.v_swa), d.n_swa.cpu().numpy(), scale,
                                       sh.tokens)
    got, gl = f64(d.out), f64(d.lse)
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(gl), empty)
    assert np.all(got[empty] == 0.0)
    # a logit: k_dim products summed in fp32, each addition half a step of at most the sum of |q k|
    logit = dot * (sh.k_dim + 4) * 2.0 ** -24
    # exp and log within 4 steps of a value up to |lse|, the sum of up to 1024 terms in fp32
    tol = 2 * logit + 8 * EPS32 * (1.0 + np.abs(lse[~empty])) + 64 * 2.0 ** -24
    assert np.all(np.abs(gl[~empty] - lse[~empty]) <= tol), float(np.abs(gl[~empty] - lse[~empty]).max())
    # a weight: twice the logit's error (itself and the sum), bf16: half a step of rounding; the sums of up to 1,024 terms; the
    # output's own rounding
    rel = 4 * logit + 64 * EPS32 + (HALF[torch.bfloat16] if d.dt == torch.bfloat16 else 0.0) + 1024 * 2.0 ** -24
    lim = absum * rel * 1.01 + HALF[d.dt] * np.abs(out) * 1.01 + 1e-30
    if (sh.q_heads, sh.k_dim, sh.v_dim, sh.dtype) == (64, 192, 128, "bf16"):
        # The entries' weights meet fp16 values as fp16 numbers of 2^7 times 2^(logit - e), e being at most the row's greatest
        # logit: those below fp16's least normal number, 2^-14, are off by half of its least step, 2^-25, which is 2^-32 of the
        # greatest weight or less; the sum of the weights is at least that weight.  So every entry adds at most 2^-32 |v|.
        lim = lim + sh.topk * 2.0 ** -32 * np.abs(v).max()
    err = np.abs(got - out)
    assert np.all(err <= lim), (float(err.max()), float((err - lim).max()))


@pytest.mark.parametrize("B,T,N,K,W,holes", [
    (1, 1, 40, 1, 1, 0.0), (1, 1, 600, 512, 128, 0.0), (3, 1, 700, 512, 128, 1.0), (6, 3, 300, 99, 37, 1.0), (5, 1, 64, 40, 128, 2.0),
    (2, 1, 700, 640, 0, 0.0), (40, 1, 600, 512, 128, 1.0), (64, 16, 600, 512, 128, 2.0), (2, 2, 1200, 1000, 24, 0.0), (300, 3, 200, 99, 37, 1.0),
    (1, 1, 9, 1, 0, 0.0), (33, 11, 513, 512, 4, 0.0), (200, 1, 300, 256, 64, 0.0), (170, 170, 600, 512, 128, 1.0), (3, 1, 1100, 896, 128, 1.0),
    (600, 4, 90, 64, 16, 2.0), (2, 1, 50, 16, 640, 1.0), (400, 1, 50, 24, 1000, 1.0)])
def test_kv4_attention_fast_path(csa2, B, T, N, K, W, holes):
    sh = shape(B, tokens=T, n_entries=N, topk=K, swa=W, k_exp=-2, v_exp=1, **FAST)
    d = attn_inputs(csa2, sh, B * 1000 + T, holes)
    assert_no_device_error(csa2, run_attn(csa2, sh, d))
    check_attn(sh, d)


@pytest.mark.parametrize("H,dk,dv,dtype", [(4, 16, 16, "f32"), (1, 1, 1, "f32"), (16, 64, 72, "bf16"), (40, 100, 33, "f32"), (9, 192, 128, "bf16"),
                                           (3, 1024, 1024, "bf16"), (64, 192, 128, "f32"), (5, 1024, 1024, "f32"), (6, 17, 130, "bf16"), (130, 48, 48, "bf16")])
@pytest.mark.parametrize("B,T,N,K,W,holes", [(10, 5, 50, 33, 7, 2.0), (1, 1, 9, 3, 0, 0.0), (90, 1, 30, 5, 3, 1.0), (1, 1, 1500, 900, 124, 0.0), (21, 1, 1100, 800, 37, 0.5)])
def test_kv4_attention_any_shape(csa2, H, dk, dv, dtype, B, T, N, K, W, holes):
    sh = shape(B, tokens=T, n_entries=N, topk=K, swa=W, q_heads=H, k_dim=dk, v_dim=dv, dtype=dtype, k_exp=1, v_exp=-2, scale=0.07)
    d = attn_inputs(csa2, sh, H * 7 + T, holes)
    assert_no_device_error(csa2, run_attn(csa2, sh, d))
    check_attn(sh, d)


# (shape arguments, queries) by kernel
KINDS = {"few": (FAST, 3), "many": (FAST, 330), "generic": (dict(q_heads=5, k_dim=24, v_dim=40, dtype="f32"), 7),
         "generic bf16": (dict(q_heads=20, k_dim=100, v_dim=72, dtype="bf16"), 7),
         "generic of four heads": (dict(q_heads=10, k_dim=24, v_dim=40, dtype="f32"), 30),
         "generic of many queries": (dict(q_heads=5, k_dim=24, v_dim=40, dtype="bf16"), 200),
         "fp32 of many queries": (dict(q_heads=5, k_dim=24, v_dim=48, dtype="f32"), 200),
         "odd bf16": (dict(q_heads=5, k_dim=25, v_dim=42, dtype="bf16"), 9)}


@pytest.mark.parametrize("kind", list(KINDS))
def test_kv4_attention_of_queries_that_attend_nothing(csa2, kind):
    kw, B = KINDS[kind]
    sh = shape(B, n_entries=300, topk=256, swa=16, **kw)
    d = attn_inputs(csa2, sh, 5, holes=0.0)
    d.idx[::2] = -1
    d.n_swa[::2] = 0
    d.idx[1::4] = -1
    assert_no_device_error(csa2, run_attn(csa2, sh, d))
    check_attn(sh, d)
    assert not d.out[::2].any() and torch.isneginf(d.lse[::2]).all()
    d.idx[:] = -1
    d.n_swa[:] = 0
    run_attn(csa2, sh, d)
    assert not d.out.any() and torch.isneginf(d.lse).all()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")])
def test_kv4_attention_ignores_what_it_does_not_attend(csa2, kind, what):
    """NaN and infinities in entries that are not selected and in window rows behind the count change nothing."""
    kw, B = KINDS[kind]
    sh = shape(B, n_entries=300, topk=200, swa=16, **kw)
    d = attn_inputs(csa2, sh, 6, holes=2.0, fill=9)
    d.idx[d.idx == 0] = -1
    run_attn(csa2, sh, d)
    out, lse = d.out.clone(), d.lse.clone()
    g = 8 * (R.groups(sh.k_dim) + R.groups(sh.v_dim))
    d.kv[:, 0, g:] = 0x7f
    taken = torch.zeros((B, 300), dtype=torch.bool, device="cuda").scatter_(1, d.idx.clamp(min=0).long(), True)
    d.kv[..., g:] = torch.where(taken[..., None], d.kv[..., g:], torch.full_like(d.kv[..., g:], 0x7f))
    d.k_swa[:, 9:] = what
    d.v_swa[:, 9:] = what
    d.out.fill_(9.0)
    run_attn(csa2, sh, d)
    assert torch.equal(d.out, out) and torch.equal(d.lse, lse)


@pytest.mark.parametrize("kind", list(KINDS))
def test_kv4_attention_scores_that_are_not_finite(csa2, kind):
    """A query or an attended key that is NaN makes its heads' output and lse NaN, a score of +inf too; others are not touched."""
    kw, B = KINDS[kind]
    sh = shape(B, n_entries=300, topk=256, swa=16, **kw)
    d = attn_inputs(csa2, sh, 7, holes=0.0, fill=16)
    run_attn(csa2, sh, d)
    out, lse = d.out.clone(), d.lse.clone()
    d.q[1, 2] = float("nan")                              # a head of a query
    d.k_swa[2, 3] = float("nan")                          # a window key of a query
    big = torch.zeros(sh.k_dim)
    big[0] = 1e30
    d.q[0, 1], d.k_swa[0, 5] = big.to(d.dt).cuda(), big.to(d.dt).cuda()   # +inf for one head; other heads' scores with it are large
    run_attn(csa2, sh, d)
    odd = torch.zeros((B, sh.q_heads), dtype=torch.bool, device="cuda")
    odd[1, 2] = odd[2] = odd[0, 1] = True
    assert d.out[odd].isnan().all() and d.lse[odd].isnan().all()
    odd[0] = True
    assert torch.equal(d.out[~odd], out[~odd]) and torch.equal(d.lse[~odd], lse[~odd])
    assert not d.lse[0, :1].isnan().any()
    # entries whose groups read as NaN
    d = attn_inputs(csa2, sh, 7, holes=0.0, fill=16)
    g = 8 * (R.groups(sh.k_dim) + R.groups(sh.v_dim))
    d.kv[1, int(d.idx[1, 3]), g] = 0x7f
    d.kv[2, int(d.idx[2, 9]), g + R.groups(sh.k_dim) + 1] = 0x7f   # of a value: 16 dims of the output
    run_attn(csa2, sh, d)
    assert d.out[1].isnan().all() and d.lse[1].isnan().all()
    dims = torch.zeros(sh.v_dim, dtype=torch.bool, device="cuda")
    dims[16:32] = True
    assert torch.equal(d.out[2].isnan(), dims.expand(sh.q_heads, -1)) and torch.equal(d.lse[2], lse[2])
    assert torch.equal(d.out[0], out[0]) and torch.equal(d.lse[0], lse[0])


@pytest.mark.parametrize("kind", list(KINDS))
def test_kv4_attention_large_logits_and_repeated_entries(csa2, kind):
    kw, B = KINDS[kind]
    sh = shape(B, n_entries=300, topk=256, swa=16, **kw)
    d = attn_inputs(csa2, sh, 8, holes=0.0, loud=60.0)
    d.idx[:, 100:140] = d.idx[:, 100:101]
    run_attn(csa2, sh, d)
    check_attn(sh, d)


@pytest.mark.parametrize("kind", list(KINDS))
def test_kv4_attention_bad_inputs_are_recorded(csa2, kind):
    kw, B = KINDS[kind]
    sh = shape(B, n_entries=300, topk=256, swa=16, **kw)
    d = attn_inputs(csa2, sh, 9, holes=0.0)
    ws = csa2.workspace(sh)
    d.idx[1, 7], d.idx[2, 255] = 300, 2 ** 31 - 1
    run_attn(csa2, sh, d, ws)
    assert csa2.read_device_error(ws) == (-5, BAD_INDEX)
    check_attn(sh, d)
    d.idx[1, 7] = d.idx[2, 255] = -7
    d.n_swa[0], d.n_swa[2] = -1, 17
    run_attn(csa2, sh, d, ws)
    assert csa2.read_device_error(ws) == (-5, BAD_COUNT)
    check_attn(sh, d)


@pytest.mark.parametrize("kind", list(KINDS))
def test_kv4_caches_beyond_32_bit_offsets(csa2, kind):
    """Entries that lie beyond 2^32 bytes: bit for bit what the same entries give in a cache of 90; appended and read there too."""
    kw, B = KINDS[kind]
    sh = shape(B, tokens=B, n_entries=90, topk=60, swa=8, k_exp=0, v_exp=0, **kw)
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    d = attn_inputs(csa2, sh, 3, holes=1.0)
    run_attn(csa2, sh, d)
    out, lse = d.out.clone(), d.lse.clone()
    check_attn(sh, d)
    N = min(2 ** 32 // csa2.kv4_bytes(sh) + 1000, 2 ** 28)
    far = torch.arange(90, device="cuda") * ((N - 1) // 89)
    big = torch.zeros((1, N, d.kv.shape[-1]), dtype=torch.uint8, device="cuda")
    big[:, far] = d.kv
    small, d.kv = d.kv, big
    d.idx = torch.where(d.idx < 0, d.idx, far.int()[d.idx.clamp(min=0).long()])
    sh.n_entries = N
    d.out.fill_(9.0)
    many = csa2.workspace(shape(B, tokens=B, n_entries=N, topk=60, swa=8, **kw))
    run_attn(csa2, sh, d, many)
    assert_no_device_error(csa2, many)
    assert torch.equal(d.out, out) and torch.equal(d.lse, lse)
    del many
    dt = dtype_of(sh)
    rows = [torch.empty((1, 90, x), dtype=dt, device="cuda") for x in (sh.k_dim, sh.v_dim)]
    want = [torch.empty_like(x) for x in rows]
    one = shape(1, **{**kw, "n_entries": N, "topk": 60, "swa": 8, "idx_dim": 1, "k_exp": 0, "v_exp": 0})
    csa2.kv4_rows(one, big, far.int()[None].contiguous(), *rows, None)
    csa2.kv4_rows(shape(1, **{**kw, "n_entries": 90, "topk": 60, "swa": 8}), small, i32(np.arange(90)[None]), *want, None)
    assert torch.equal(rows[0], want[0]) and torch.equal(rows[1], want[1])
    s = types.SimpleNamespace(kv=big, k_idx=torch.zeros((1, N, 1), dtype=dt, device="cuda"), n_valid=i32([N - 50]), n_new=i32([40]),
                              kb=torch.zeros((1, -(-N // 8), 1), dtype=dt, device="cuda"))
    s.k_new, s.v_new, s.x_new = new_entries(one, 40, 4)
    run_append(csa2, one, s)
    assert int(s.n_valid[0]) == N - 10
    ref = R.pack(f64(s.k_new[0, 39]), f64(s.v_new[0, 39]), 0, 0)
    have = R.unpack(s.kv[0, N - 11].cpu().numpy(), sh.k_dim, sh.v_dim, 0, 0)
    for a, b in zip(have, R.unpack(ref, sh.k_dim, sh.v_dim, 0, 0)):
        assert np.array_equal(a, b)


# ------------------------------------------------------------------ together

def step_inputs(csa2, seed):
    """Three sequences of a decode step: projections, caches of 200 entries that hold 150, 9 and 0."""
    g = torch.Generator().manual_seed(seed)
    sh = shape(3, n_entries=200, topk=64, swa=16, k_exp=0, v_exp=-1, **FAST)
    s = types.SimpleNamespace()
    s.proj = randn(g, (3, 66 * 192), torch.bfloat16, 2.0)              # 64 queries, the entry's key, the token's key
    s.gain = (1 + 0.2 * torch.randn(192, generator=g)).cuda()
    s.pos = i32([600, 37, 0])
    s.v_new, s.x_new = randn(g, (3, 1, 128), torch.bfloat16, 0.5), torch.randint(-4, 5, (3, 1, 64), generator=g).bfloat16().cuda()
    s.v_tok = randn(g, (3, 128), torch.bfloat16, 0.5)
    s.q_idx, s.w_idx = torch.randint(-4, 5, (3, 8, 64), generator=g).bfloat16().cuda(), torch.randint(1, 4, (3, 8), generator=g).float().cuda()
    s.kv = torch.zeros((3, 200, csa2.kv4_bytes(sh)), dtype=torch.uint8, device="cuda")
    s.k_idx, s.kb = torch.zeros((3, 200, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((3, 25, 64), dtype=torch.bfloat16, device="cuda")
    s.n_valid, s.prompt = i32([0, 0, 0]), i32([150, 9, 0])
    s.k_old, s.v_old = randn(g, (3, 150, 192), torch.bfloat16), randn(g, (3, 150, 128), torch.bfloat16, 0.5)
    s.x_old = torch.randint(-4, 5, (3, 150, 64), generator=g).bfloat16().cuda()
    s.one = i32([1, 1, 1])
    s.k_swa, s.v_swa = randn(g, (3, 16, 192), torch.bfloat16), randn(g, (3, 16, 128), torch.bfloat16, 0.5)
    s.head, s.n_swa = i32([3, 5, 0]), i32([16, 5, 0])
    s.idx = torch.full((3, 64), -5, dtype=torch.int32, device="cuda")
    s.out, s.lse = torch.zeros((3, 64, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((3, 64), device="cuda")
    s.rows = torch.zeros((3, 64, 192), dtype=torch.bfloat16, device="cuda")
    s.rows_v = torch.zeros((3, 64, 128), dtype=torch.bfloat16, device="cuda")
    s.weights = torch.zeros((3, 64), device="cuda")
    s.slots = torch.arange(64, dtype=torch.int32, device="cuda").repeat(3, 1)
    s.near = torch.zeros_like(s.slots)
    return sh, s


def run_step(csa2, sh, s, ws, freqs):
    """A prompt packed, then a decode step: norm and positions, the new entry and the window's token, selection, attention, and
    the attention weights over the selected rows as numbers."""
    q, k = s.proj[:, :64 * 192].unflatten(1, (64, 192)), s.proj[:, 64 * 192:].unflatten(1, (2, 192))
    ex = dict(k_exp=sh.k_exp, v_exp=sh.v_exp)
    csa2.kv4_append(sh, s.prompt, s.k_old, s.v_old, s.x_old, s.kv, s.k_idx, s.kb, s.n_valid, ws, **ex)
    csa2.norm_rope([(q, q, s.gain, 128), (k, k, s.gain, 128)], s.pos, freqs)
    csa2.kv4_append(sh, s.one, k[:, :1].contiguous(), s.v_new, s.x_new, s.kv, s.k_idx, s.kb, s.n_valid, ws, **ex)
    csa2.swa_append(sh, [(k[:, 1].contiguous(), s.v_tok, s.k_swa, s.v_swa)], s.head, s.n_swa, ws)
    csa2.index_topk(sh, s.q_idx, s.w_idx, s.k_idx, s.n_valid, 64, s.idx, ws)
    q = q.contiguous()
    csa2.kv4_attn(sh, q, s.kv, s.idx, s.k_swa, s.v_swa, s.n_swa, s.out, ws, lse=s.lse, **ex)
    csa2.kv4_rows(sh, s.kv, s.idx, s.rows, s.rows_v, ws, **ex)
    s.near.copy_(torch.where(s.idx < 0, s.idx, s.slots))
    csa2.attn_weights(shape(3, n_entries=64, topk=64, swa=16, **FAST), q, s.rows, s.near, s.lse, s.weights, ws)


STEP = ("proj", "kv", "k_idx", "kb", "n_valid", "k_swa", "v_swa", "head", "n_swa", "idx", "out", "lse", "rows", "rows_v", "weights")


def test_a_step_of_all_operators(csa2):
    """Eager, on another stream, and captured and replayed: the same; the attention is the definition's on the step's own
    intermediate results, as csa2_sparse_attn over the rows as numbers has it, and the weights sum to what the window leaves."""
    freqs, _ = csa2.rope_freqs(64)
    sh, a = step_inputs(csa2, 4)
    ws = csa2.workspace(sh)
    first = clone(a)
    run_step(csa2, sh, a, ws, freqs)
    assert_no_device_error(csa2, ws)
    assert a.n_valid.tolist() == [151, 10, 1] and (a.idx >= 0).sum(1).tolist() == [64, 10, 1]
    d = types.SimpleNamespace(dt=torch.bfloat16, k_exp=sh.k_exp, v_exp=sh.v_exp, **{k: getattr(a, k) for k in ("kv", "idx", "k_swa", "v_swa", "n_swa", "out", "lse")})
    d.q = a.proj[:, :64 * 192].unflatten(1, (64, 192))
    check_attn(sh, d)
    wide = shape(3, n_entries=64, topk=64, swa=16, **FAST)
    out, lse = torch.empty((3, 64, 128), device="cuda"), torch.empty((3, 64), device="cuda")
    csa2.sparse_attn(wide, d.q.contiguous(), a.rows, a.rows_v, a.near, a.k_swa, a.v_swa, a.n_swa, out, csa2.workspace(wide), lse=lse)
    assert float((lse - a.lse).abs().max()) <= 1e-5
    assert float((out - a.out.float()).abs().max()) <= 2 * HALF[torch.bfloat16] * float(a.v_swa.abs().max() + a.rows_v.abs().max())
    k, _ = numbers(sh, d)
    w = D.attention_weights(f64(d.q), k, a.idx.cpu().numpy(), f64(a.lse), 192 ** -0.5, 1)
    assert np.abs(f64(a.weights) - w).max() <= 2e-4 * w.max()
    b = clone(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_step(csa2, sh, b, ws, freqs)
    side.synchronize()
    c = clone(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_step(csa2, sh, c, ws, freqs)
    for _ in range(2):
        for k in vars(first):
            getattr(c, k).copy_(getattr(first, k))
        graph.replay()
        torch.cuda.synchronize()
        for k in STEP:
            assert torch.equal(getattr(a, k), getattr(b, k)) and torch.equal(getattr(a, k), getattr(c, k)), k


def test_calls_on_two_streams_at_once(csa2):
    """The attention's kernels on two streams, each with its own workspace, give what they give one after the other, whatever
    stream is current (the one that is passed counts)."""
    sh = shape(330, n_entries=600, topk=512, swa=64, k_exp=-2, v_exp=0, **FAST)
    sets = [attn_inputs(csa2, sh, 41), attn_inputs(csa2, sh, 42)]
    works = [csa2.workspace(sh), csa2.workspace(sh)]
    want = []
    for d, ws in zip(sets, works):
        run_attn(csa2, sh, d, ws)
        want.append((d.out.clone(), d.lse.clone()))
        d.out.fill_(9.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for d, ws, st in zip(sets, works, streams):
            csa2.kv4_attn(sh, d.q, d.kv, d.idx, d.k_swa, d.v_swa, d.n_swa, d.out, ws, lse=d.lse, k_exp=-2, v_exp=0, stream=st)
    torch.cuda.synchronize()
    for d, (out, lse), ws in zip(sets, want, works):
        assert torch.equal(d.out, out) and torch.equal(d.lse, lse)
        assert_no_device_error(csa2, ws)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("ke,ve,near", [(64, -64, False), (-64, 64, False), (-64, -64, True), (64, 64, True)])
def test_kv4_attention_at_the_exponents_ends(csa2, kind, ke, ve, near):
    """Keys and values of 2^-64 to 2^64; `near`: window values about 1, far from what the entries' are."""
    kw, n = KINDS[kind]
    sh = shape(n, n_entries=70, topk=48, swa=20, k_exp=ke, v_exp=ve, scale=0.1, **kw)
    d = attn_inputs(csa2, sh, 77, 1.0)
    if near:
        d.v_swa.copy_(d.v_swa * 2.0 ** -ve)
    assert_no_device_error(csa2, run_attn(csa2, sh, d))
    check_attn(sh, d)


@pytest.mark.parametrize("kind", list(KINDS))
def test_kv4_attention_captured(csa2, kind):
    """A captured call reads what its arrays hold when it is replayed; two graphs share a workspace."""
    kw, n = KINDS[kind]
    sh = shape(n, n_entries=90, topk=70, swa=30, k_exp=-2, v_exp=0, **kw)
    sets = [attn_inputs(csa2, sh, seed, 1.0) for seed in (5, 6)]
    ws, want = csa2.workspace(sh), []
    for d in sets:
        run_attn(csa2, sh, d, ws)
        want.append((d.out.clone(), d.lse.clone()))
    graphs = []
    for d in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run_attn(csa2, sh, d, ws)
        graphs.append(graph)
    for turn in range(3):
        for d, graph, (out, lse) in zip(sets, graphs, want):
            d.out.fill_(9.0)
            d.lse.fill_(9.0)
            graph.replay()
            assert torch.equal(d.out, out) and torch.equal(d.lse, lse), turn
        for name in ("q", "kv", "idx", "k_swa", "v_swa", "n_swa"):   # each graph with the other's inputs
            a, b = (getattr(d, name) for d in sets)
            keep = a.clone()
            a.copy_(b)
            b.copy_(keep)
        want.reverse()
    assert_no_device_error(csa2, ws)


@pytest.mark.parametrize("kind", list(KINDS))
def test_kv4_attention_without_windows_takes_no_counts(csa2, kind):
    kw, n = KINDS[kind]
    sh = shape(n, n_entries=50, topk=30, swa=0, k_exp=0, v_exp=0, **kw)
    d = attn_inputs(csa2, sh, 9, 0.0, fill=0)
    run_attn(csa2, sh, d)
    out, lse = d.out.clone(), d.lse.clone()
    d.n_swa.fill_(77)
    assert_no_device_error(csa2, run_attn(csa2, sh, d))
    assert torch.equal(d.out, out) and torch.equal(d.lse, lse)
    check_attn(sh, types.SimpleNamespace(**{**vars(d), "n_swa": torch.zeros_like(d.n_swa)}))


def test_norm_rope_before_an_attention_that_reads_early(csa2):
    """Queries and windows that csa2_norm_rope writes, straight into csa2_sparse_attn, which looks at them before its turn; and
    rows that csa2_kv4_rows writes as its main cache."""
    B, N, K, W = 40, 300, 256, 64
    sh = shape(B, n_entries=N, topk=K, swa=W, k_exp=0, v_exp=0, **FAST)
    d = attn_inputs(csa2, sh, 3, 0.0)
    wide = shape(B, n_entries=K, topk=K, swa=W, **FAST)
    ws = csa2.workspace(wide)
    rows_k = torch.empty(B, K, 192, dtype=d.dt, device="cuda")
    rows_v = torch.empty(B, K, 128, dtype=d.dt, device="cuda")
    own = torch.arange(K, dtype=torch.int32, device="cuda").repeat(B, 1)
    q = torch.empty_like(d.q)
    out, lse = torch.empty(B, 64, 128, device="cuda"), torch.empty(B, 64, device="cuda")
    got = []
    for wait in (True, False, False, False):
        for t in (q, rows_k, rows_v):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        csa2.kv4_rows(sh, d.kv, d.idx, rows_k, rows_v, None)
        csa2.norm_rope([(d.q, q, None, 0)])
        if wait:
            torch.cuda.synchronize()
        csa2.sparse_attn(wide, q, rows_k, rows_v, own, d.k_swa, d.v_swa, d.n_swa, out, ws, lse=lse)
        got.append((out.clone(), lse.clone()))
    for o, l in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(l, got[0][1])
    assert torch.isfinite(got[0][0]).all()


@pytest.mark.parametrize("shift", [1, 2, 4])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_kv4_attention_of_windows_at_odd_addresses(csa2, dtype, shift):
    """Windows (and queries) that begin `shift` elements behind a 16-byte address."""
    sh = shape(20, n_entries=60, topk=40, swa=33, k_exp=-1, v_exp=1, q_heads=18, k_dim=80, v_dim=48, dtype=dtype)
    d = attn_inputs(csa2, sh, shift, 1.0)
    for name in ("q", "k_swa", "v_swa"):
        x = getattr(d, name)
        moved = torch.empty(x.numel() + shift, dtype=x.dtype, device="cuda")[shift:].view(x.shape)
        moved.copy_(x)
        setattr(d, name, moved)
    assert_no_device_error(csa2, run_attn(csa2, sh, d))
    check_attn(sh, d)


def test_norm_rope_of_strided_views(csa2):
    """Heads that do not lie side by side are refused, rows that lie apart are not; sizes of one may have any stride."""
    x = torch.randn((4, 6, 16), device="cuda")
    for view in (x[:, ::2], x[..., ::2], x[:, :, :1], x.transpose(0, 1)[:, :3], x[:, :1].expand(4, 6, 16), x[..., :1].expand(4, 6, 16)):
        with pytest.raises(ValueError):
            csa2.norm_rope([(view, torch.empty(view.shape, device="cuda"), None, 0)])
    with pytest.raises(csa2.CSA2Error):                       # one row for all
        csa2.norm_rope([(x[:1].expand(4, 6, 16), torch.empty_like(x), None, 0)])
    for view in (x[::2], x[:, 2:4], x[1:2], x[:, 3], x[:, :1], x[..., 3:4][:, 2:3], x[:1].expand(1, 6, 16)):
        out = torch.empty(view.shape, device="cuda")
        csa2.norm_rope([(view, out, None, 0)], eps=0.0)
        want = view.double() / view.double().square().mean(-1, keepdim=True).sqrt()
        # 16 squares, their sum, the mean, a root and two products in fp32: 24 half steps of a value
        assert ((out.double() - want).abs() <= 24 * 2.0 ** -24 * want.abs() + 1e-30).all()


@pytest.mark.parametrize("B,H,dk,dv,K,W", [(1, 5, 64, 64, 512, 128), (3, 20, 100, 72, 500, 100), (9, 40, 192, 128, 250, 6), (6, 16, 40, 1024, 900, 124),
                                           (2, 64, 1024, 24, 128, 0)])
def test_kv4_attention_of_few_queries_split_over_clusters(csa2, B, H, dk, dv, K, W):
    """bf16 shapes whose slots several CTAs share: parts that hold nothing, scores that are not finite in one part alone."""
    sh = shape(B, n_entries=1300, topk=K, swa=W, k_exp=-1, v_exp=1, q_heads=H, k_dim=dk, v_dim=dv, dtype="bf16", scale=0.07)
    d = attn_inputs(csa2, sh, B + H, 2.0)
    d.idx[0, :K // 2], d.idx[0, K - 1] = -1, 7                # the first parts of a query have nothing
    if B > 1:
        d.idx[1, 10:] = -1                                    # nor the last ones of another
        d.n_swa[1] = 0
    if B > 2:
        d.idx[2] = -1
        d.n_swa[2] = 0
    assert_no_device_error(csa2, run_attn(csa2, sh, d))
    check_attn(sh, d)
    out, lse = d.out.clone(), d.lse.clone()
    d.q[0, 1] = float("nan")                                  # one head of one query
    run_attn(csa2, sh, d)
    assert torch.isnan(d.out[0, 1]).all() and torch.isnan(d.lse[0, 1])
    keep = torch.ones_like(d.lse, dtype=torch.bool)
    keep[0, 1] = False
    assert torch.equal(d.out[keep], out[keep]) and torch.equal(d.lse[keep], lse[keep])
    d.idx[0, 3] = 1300                                        # beyond the cache: skipped and recorded
    assert csa2.read_device_error(run_attn(csa2, sh, d)) == (-5, BAD_INDEX)
    assert torch.equal(d.out[keep], out[keep])


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("k_exp,scale", [(-46, 0.0), (-47, 0.0), (-64, 0.0), (64, 0.0), (-2, 1e-30), (-64, 1e-18)])
def test_kv4_attention_of_queries_of_zeros_and_tiny_ones(csa2, kind, k_exp, scale):
    """Heads of zeros (rows of a padded batch) and of about 2^-100 weigh all that they attend alike, whatever the exponent, the
    softmax scale and the holes in their lists."""
    kw, B = KINDS[kind]
    sh = shape(B, n_entries=300, topk=200, swa=40, k_exp=k_exp, v_exp=0, scale=scale, **kw)
    d = attn_inputs(csa2, sh, 31, holes=2.0)
    d.idx[0, ::2], d.n_swa[0] = -1, 0                       # every second slot of a list is a hole, and nothing else is attended
    d.q[:, ::2] = 0.0
    d.q[:, 1] = randn(torch.Generator().manual_seed(3), (B, sh.k_dim), d.dt, 2.0 ** -100)
    d.q[B - 1] = 0.0
    assert_no_device_error(csa2, run_attn(csa2, sh, d))
    check_attn(sh, d)
    count = (d.idx >= 0).sum(1) + d.n_swa
    flat = d.lse[:, ::2].double()
    # log of a count of up to 240: exp and log within 4 steps, the sum exact or half a step an addition
    assert ((flat - count.double().log()[:, None]).abs() <= 8 * EPS32 * 7 + 240 * 2.0 ** -24)[count > 0].all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(192, 128), (20, 24)])
def test_kv4_append_of_numbers_beyond_the_range_of_their_quotients(csa2, dtype, dk, dv):
    """Exponents of -64: numbers from 2^64 on, whose quotients by 2^exp are beyond fp32, saturate as any large number does; only
    NaN and infinities read as NaN."""
    sh = shape(2, n_entries=40, k_dim=dk, v_dim=dv, dtype=dtype, topk=4, swa=4, k_exp=-64, v_exp=-64)
    s = append_state(csa2, sh, 24, 13, [3, 0], [24, 24])
    rng = np.random.default_rng(17)
    for t in (s.k_new, s.v_new):
        top = np.exp2(rng.integers(60, 127, t.shape[:2] + (1,)) + rng.random(t.shape[:2] + (1,)))
        x = rng.choice([1.0, -1.0, 0.6, 2.0 ** -61, -2.0 ** -64, 0.0], t.shape) * top
        x[0, 0], x[0, 1], x[0, 2] = 2.0 ** 64, -2.0 ** 127, 3e38
        x[0, 3, 5], x[1, 4, 19] = np.inf, np.nan
        t.copy_(torch.tensor(x, dtype=torch.float32).to(t.dtype))
    before, ws = clone(s), csa2.workspace(sh)
    run_append(csa2, sh, s, ws)
    assert_no_device_error(csa2, ws)
    check_append(sh, s, before)
    k, v = torch.empty_like(s.k_new), torch.empty_like(s.v_new)
    csa2.kv4_rows(sh, s.kv, i32(np.arange(24) + np.array([[3], [0]])), k, v, ws, k_exp=-64, v_exp=-64)
    for x in (k, v):
        assert (x[0, 0] == 2688.0 * 2.0 ** -64).all() and (x[0, 1] == -2688.0 * 2.0 ** -64).all() and int(x.isnan().sum()) == min(16, x.shape[2]) + min(16, x.shape[2] - 16)


@pytest.mark.parametrize("B,K,W,fill", [(3, 512, 128, 128), (330, 512, 128, 128), (40, 64, 512, 300), (330, 1, 128, 50)])
def test_kv4_attention_waits_that_give_up(csa2, B, K, W, fill):
    """A stage that never fills, of a query split over a cluster, of many queries a CTA, and in a window: every role gives up, the
    call returns with the timeout recorded and writes nothing but its outputs; the same workspace then serves a normal call."""
    sh = shape(B, n_entries=600, topk=K, swa=W, **FAST)
    d = attn_inputs(csa2, sh, 12, holes=0.0, fill=fill)
    if fill == 50:
        d.idx[:] = -1
    ws = run_attn(csa2, sh, d)
    out, lse = d.out.clone(), d.lse.clone()
    whole, sums = torch.full((B + 2, *out.shape[1:]), 5.0, dtype=out.dtype, device="cuda"), torch.full((B + 2, 64), 5.0, device="cuda")
    csa2.debug_kv4_wait_timeout(sh, d.q, d.kv, d.idx, d.k_swa, d.v_swa, d.n_swa, whole[1:-1], 2000000, ws, lse=sums[1:-1])
    st, bits = csa2.read_device_error(ws)
    assert st == -6 and bits == 4
    for x in (whole, sums):
        assert (x[0] == 5.0).all() and (x[-1] == 5.0).all()
    for t in (d.out, d.lse):
        t.fill_(9.0)
    assert_no_device_error(csa2, run_attn(csa2, sh, d, ws))
    assert torch.equal(d.out, out) and torch.equal(d.lse, lse)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("ve,power", [(64, -60), (-64, 33), (64, 64), (-64, -64)])
def test_kv4_attention_of_windows_far_from_the_entries(csa2, kind, ve, power):
    """Windows alone, whose values are of 2^power: down to 2^(v_exp - 126), up to 2^(v_exp + 100)."""
    kw, B = KINDS[kind]
    sh = shape(B, n_entries=70, topk=48, swa=40, k_exp=0, v_exp=ve, **kw)
    d = attn_inputs(csa2, sh, 77, fill=40)
    d.idx[:] = -1
    d.v_swa.copy_(d.v_swa.float() * 2.0 ** (power - ve))
    assert_no_device_error(csa2, run_attn(csa2, sh, d))
    check_attn(sh, d)


@pytest.mark.parametrize("kind", list(KINDS))
def test_kv4_attention_without_lse(csa2, kind):
    kw, B = KINDS[kind]
    sh = shape(B, n_entries=90, topk=70, swa=30, k_exp=-2, v_exp=0, **kw)
    d = attn_inputs(csa2, sh, 5, 1.0)
    ws = run_attn(csa2, sh, d)
    out = d.out.clone()
    d.out.fill_(9.0)
    csa2.kv4_attn(sh, d.q, d.kv, d.idx, d.k_swa, d.v_swa, d.n_swa, d.out, ws, k_exp=-2, v_exp=0)
    assert torch.equal(d.out, out)
    assert_no_device_error(csa2, ws)
