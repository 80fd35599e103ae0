"""Host-side checks of the drafted-tree operators (no GPU): the calls that the header refuses are refused before
anything is enqueued (the fake pointers are never dereferenced), and the rotary frequencies against their formulas."""
import ctypes
import math

import pytest

from sparse_attention_decode_index_gb300 import build as B
from sparse_attention_decode_index_gb300 import workloads as W

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
FAKE = 0x7f0000000000
STEP = 1 << 36                      # fake arrays far apart
MIS = FAKE + 8


@pytest.fixture(scope="module")
def csa2():
    B.build()
    from sparse_attention_decode_index_gb300 import csa2 as m
    m.lib()
    return m


def _shape(csa2, **kw):
    base = dict(batch=8, n_entries=4096, pool_blocks=0, tokens=4)
    base.update(kw)
    return csa2.c_shape(W.Shape(**base))


def _ws(csa2, s):
    return csa2.lib().csa2_workspace_bytes(ctypes.byref(s))


def test_rope_freqs(csa2):
    lib = csa2.lib()
    buf = (ctypes.c_double * 512)()
    mag = ctypes.c_float(0)

    def call(rot=8, base=10000.0, kind=0, factor=1.0, ctx=0, fast=32.0, slow=1.0, out=buf):
        return lib.csa2_rope_freqs(rot, base, kind, factor, ctx, fast, slow, ctypes.cast(out, ctypes.c_void_p) if out else None,
                                   ctypes.byref(mag))

    for bad in (dict(rot=0), dict(rot=7), dict(rot=-2), dict(rot=1026), dict(base=1.0), dict(base=math.nan), dict(base=math.inf),
                dict(kind=4), dict(kind=-1), dict(kind=1, factor=0.5), dict(kind=1, factor=math.nan), dict(kind=2, rot=2, factor=2.0),
                dict(kind=3, factor=2.0), dict(kind=3, factor=2.0, ctx=100, fast=1.0), dict(kind=3, factor=2.0, ctx=100, slow=0.0),
                dict(out=None)):
        assert call(**bad) == INVALID, bad
    assert call() == OK and mag.value == 1.0
    assert list(buf[:4]) == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-15)
    assert call(kind=1, factor=4.0) == OK
    assert list(buf[:4]) == pytest.approx([0.25, 0.025, 0.0025, 0.00025], rel=1e-15)
    assert call(kind=2, factor=16.0) == OK                 # base 10000 * 16^(8/6)
    b = 10000.0 * 16.0 ** (8.0 / 6.0)
    assert list(buf[:4]) == pytest.approx([b ** (-i / 4.0) for i in range(4)], rel=1e-14)
    # the slowest pair of the scaled base turns as the slowest of the plain one does at 1 / factor
    assert buf[3] == pytest.approx(0.001 / 16.0, rel=1e-12)
    assert call(rot=64, kind=3, factor=8.0, ctx=4096) == OK
    assert mag.value == pytest.approx(0.1 * math.log(8.0) + 1.0, rel=1e-7)
    for i in range(32):
        f = 10000.0 ** (-i / 32.0)
        turns = 4096 * f / (2 * math.pi)
        if turns > 36:                                     # well above beta_fast: kept
            assert buf[i] == pytest.approx(f, rel=1e-14)
        elif turns < 0.75:                                 # well below beta_slow: scaled
            assert buf[i] == pytest.approx(f / 8.0, rel=1e-14)
        else:
            assert f / 8.0 * (1 - 1e-12) <= buf[i] <= f * (1 + 1e-12)
    assert all(buf[i] > buf[i + 1] for i in range(31))


def test_rope_freqs_of_a_base_that_overflows(csa2):
    """An NTK base beyond doubles (10000 * 1e160^2) would leave every pair but the first unturned."""
    lib = csa2.lib()
    buf, mag = (ctypes.c_double * 2)(), ctypes.c_float(0)
    args = (4, 10000.0, 2), (0, 32.0, 1.0, ctypes.cast(buf, ctypes.c_void_p), ctypes.byref(mag))
    assert lib.csa2_rope_freqs(*args[0], 1e160, *args[1]) == INVALID
    assert lib.csa2_rope_freqs(*args[0], 1e150, *args[1]) == OK
    assert list(buf) == pytest.approx([1.0, 1e-152], rel=1e-12)


def test_rope_refusals(csa2):
    lib = csa2.lib()
    good = dict(x=FAKE, out=FAKE + STEP, heads=64, dim=192, rot_off=128, dtype=0)

    def call(slots=(good,), n=None, rows=4, rot=64, inter=0, pos=FAKE + 4 * STEP, freqs=FAKE + 5 * STEP, mag=1.0, inv=0):
        arr = (csa2.CRopeSlot * max(1, len(slots)))(*[csa2.CRopeSlot(*[y[k] for k in ("x", "out", "heads", "dim", "rot_off", "dtype")])
                                                      for y in slots])
        return lib.csa2_rope(ctypes.cast(arr, ctypes.c_void_p), len(slots) if n is None else n, rows, rot, inter, pos, freqs, mag,
                             inv, None)

    for bad in (dict(n=0), dict(n=17), dict(rows=0), dict(rows=-1), dict(rot=0), dict(rot=63), dict(inter=2), dict(inv=-1), dict(pos=None),
                dict(freqs=None), dict(freqs=FAKE + 5 * STEP + 4), dict(mag=0.0), dict(mag=-1.0), dict(mag=math.nan), dict(mag=math.inf),
                dict(rot=66)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(x=None), dict(out=None), dict(heads=0), dict(dim=0), dict(rot_off=-1), dict(rot_off=129), dict(dtype=2),
                dict(out=FAKE + 2),                        # overlaps its input without being it
                dict(out=FAKE + 4 * STEP), dict(out=FAKE + 5 * STEP)):   # the positions, the frequencies
        assert call(slots=({**good, **bad},)) == INVALID, bad
    assert call(slots=({**good, "heads": 1025},)) == UNSUPPORTED
    assert call(slots=({**good, "dim": 1025},)) == UNSUPPORTED
    assert call(rot=1026, slots=({**good, "dim": 1026, "rot_off": 0},)) == UNSUPPORTED
    other = dict(good, x=FAKE + 2 * STEP)
    assert call(slots=(good, other)) == INVALID            # one output twice
    assert call(slots=(good, dict(other, out=FAKE))) == INVALID   # over another slot's input


def _tree_args(**kw):
    names = ("q", "k_main", "v_main", "idx", "k_swa", "v_swa", "swa_head", "n_swa", "k_draft", "v_draft", "parent", "n_draft", "out",
             "lse")
    d = {n: FAKE + i * STEP for i, n in enumerate(names)}
    d.update(kw)
    return [d[n] for n in names]


def test_tree_attn_refusals(csa2):
    lib = csa2.lib()
    s = _shape(csa2)

    def call(s=s, ws=FAKE, nbytes=None, **kw):
        n = _ws(csa2, s) if nbytes is None else nbytes
        return lib.csa2_tree_attn(ctypes.byref(s), *_tree_args(**kw), ws, n, None)

    for n in ("q", "k_main", "v_main", "idx", "k_swa", "v_swa", "n_swa", "k_draft", "v_draft", "out"):
        assert call(**{n: None}) == INVALID, n
    for n in ("q", "k_main", "v_main", "k_swa", "v_swa", "k_draft", "v_draft", "out"):
        assert call(**{n: MIS}) == INVALID, n
    assert call(nbytes=_ws(csa2, s) - 1) == WORKSPACE
    assert call(ws=None) == WORKSPACE and call(ws=FAKE + 16) == WORKSPACE
    assert call(s=_shape(csa2, swa=0)) == INVALID
    assert call(s=_shape(csa2, batch=129, tokens=129)) == UNSUPPORTED
    assert call(s=_shape(csa2, batch=65536, n_entries=1, topk=1, swa=1)) == UNSUPPORTED
    bad = _shape(csa2)
    bad.batch = 6                                          # not whole sequences of 4 tokens
    assert lib.csa2_tree_attn(ctypes.byref(bad), *_tree_args(), FAKE, 1 << 30, None) == INVALID
    assert lib.csa2_tree_attn(None, *_tree_args(), FAKE, 1 << 30, None) == INVALID


def test_outputs_over_other_arrays_are_refused(csa2):
    """A written array that shares a byte with any other is refused, whichever of the two starts first; arrays that only
    touch are not looked at here (nothing may be launched without a GPU)."""
    lib = csa2.lib()
    s = _shape(csa2)                                       # 8 queries, 2 sequences, 64 heads of 192 / 128
    names = ("q", "k_main", "v_main", "idx", "k_swa", "v_swa", "swa_head", "n_swa", "k_draft", "v_draft", "parent", "n_draft", "out",
             "lse")
    size = dict(q=8 * 64 * 384, k_main=2 * 4096 * 384, v_main=2 * 4096 * 256, idx=8 * 2048, k_swa=2 * 128 * 384, v_swa=2 * 128 * 256,
                swa_head=8, n_swa=8, k_draft=8 * 384, v_draft=8 * 256, parent=32, n_draft=8, out=8 * 64 * 256, lse=8 * 64 * 4)
    at = {n: FAKE + i * STEP for i, n in enumerate(names)}
    for n in names:
        for w in ("out", "lse"):
            if n == w:
                continue
            last = at[n] + (size[n] - 1) // 16 * 16        # in n's last bytes; and n in the written array's last ones
            for p in (at[n], last, at[n] - (size[w] - 1) // 16 * 16):
                assert lib.csa2_tree_attn(ctypes.byref(s), *_tree_args(**{w: p}), FAKE - STEP, _ws(csa2, s), None) == INVALID, (n, w)
    keys = ("q", "k_main", "idx", "lse", "live", "weights")
    for n in keys[:-1]:
        d = {x: FAKE + i * STEP for i, x in enumerate(keys)}
        d["weights"] = d[n] + (16 if n != "live" else 28)
        assert lib.csa2_attn_weights(ctypes.byref(s), *d.values(), FAKE - STEP, _ws(csa2, s), None) == INVALID, n
    far = [FAKE + i * STEP for i in range(20)]

    def commit(slots, *rest):
        arr = (csa2.CTreeSlot * len(slots))(*[csa2.CTreeSlot(*y) for y in slots])
        return lib.csa2_tree_commit(ctypes.byref(s), ctypes.cast(arr, ctypes.c_void_p), len(slots), *rest, FAKE - STEP, _ws(csa2, s), None)

    one, two, rest = far[:6], far[6:10] + far[4:6], far[10:15]   # the layers share their idx and weights
    for i in (2, 3):                                       # a window: over each other array
        for p in one[:2] + two[:4] + far[4:6] + rest:
            assert commit([one, two[:i] + [p if p != two[i] else one[i]] + two[i + 1:]], *rest) == INVALID, (i, p)
    for i in (2, 3, 4):                                    # head, fill count, mass
        for p in one + two[:4] + [x for x in rest if x != rest[i]]:
            assert commit([one, two], *rest[:i], p, *rest[i + 1:]) == INVALID, (i, p)


def test_arrays_in_the_workspace_are_refused(csa2):
    """The workspace is written (its error word, the key lists of trees), so that no array of a call may share a byte with it:
    not its first, not its last."""
    lib = csa2.lib()
    s, one = _shape(csa2), _shape(csa2, tokens=1)
    n, n1, ws = _ws(csa2, s), _ws(csa2, one), FAKE - STEP
    names = ("q", "k_main", "v_main", "idx", "k_swa", "v_swa", "swa_head", "n_swa", "k_draft", "v_draft", "parent", "n_draft", "out",
             "lse")
    for x in names:
        for p in (ws, ws + n - 16, ws - 16):               # (every array is longer than 16 bytes or starts inside)
            if p < ws and x in ("swa_head", "n_swa", "n_draft"):
                p = ws - 4
            assert lib.csa2_tree_attn(ctypes.byref(s), *_tree_args(**{x: p}), ws, n, None) == INVALID, (x, p)
    keys = ("q", "k_main", "idx", "lse", "live", "weights")
    for x in keys:
        for p in (ws, ws + n - 16, ws - 16):
            d = {y: FAKE + i * STEP for i, y in enumerate(keys)}
            d[x] = p
            assert lib.csa2_attn_weights(ctypes.byref(s), *d.values(), ws, n, None) == INVALID, (x, p)
    far = [FAKE + i * STEP for i in range(20)]
    for i in range(11):
        for p in (ws, ws + n - 16, ws - 4):
            at = far[:i] + [p] + far[i + 1:]
            arr = (csa2.CTreeSlot * 1)(csa2.CTreeSlot(*at[:6]))
            rest = at[6:11]
            if i == 10 and p == ws - 4:
                continue                                   # (masses are 8 bytes apart)
            assert lib.csa2_tree_commit(ctypes.byref(s), ctypes.cast(arr, ctypes.c_void_p), 1, *rest, ws, n, None) == INVALID, (i, p)
    for i in range(12):
        for p in (ws, ws + n1 - 16, ws - 16):
            at = far[:i] + [p] + far[i + 1:12]
            assert lib.csa2_kv_evict(ctypes.byref(one), 4000, 3000, 4, 64, *at, 1, ws, n1, None) == INVALID, (i, p)
    for i in range(5):                                     # in place
        at = far[:i] + [ws] + far[i + 1:5]
        assert lib.csa2_kv_evict(ctypes.byref(one), 4000, 3000, 4, 64, *at, *at, *far[10:12], 1, ws, n1, None) == INVALID, i


@pytest.mark.parametrize("dtype,heads,dk", [("bf16", 64, 192), ("bf16", 5, 7), ("f32", 5, 7)])
def test_arrays_between_elements_are_refused(csa2, dtype, heads, dk):
    """An array that does not begin at a multiple of its elements' size would fault the kernel."""
    lib = csa2.lib()
    e = 4 if dtype == "f32" else 2
    kw = dict(dtype=dtype, q_heads=heads, k_dim=dk, v_dim=128 if heads == 64 else 9, swa=128)
    s, one = _shape(csa2, **kw), _shape(csa2, tokens=1, **kw)
    n, n1, ws = _ws(csa2, s), _ws(csa2, one), FAKE - STEP
    elems = ("q", "k_main", "v_main", "k_swa", "v_swa", "k_draft", "v_draft", "out")
    for i, x in enumerate(("q", "k_main", "v_main", "idx", "k_swa", "v_swa", "swa_head", "n_swa", "k_draft", "v_draft", "parent",
                           "n_draft", "out", "lse")):
        for off in ((e // 2,) if x in elems else (1, 2)):
            assert lib.csa2_tree_attn(ctypes.byref(s), *_tree_args(**{x: FAKE + i * STEP + off}), ws, n, None) == INVALID, x
    far = [FAKE + i * STEP for i in range(20)]
    for i in range(6):
        at = far[:i] + [far[i] + (e // 2 if i < 2 else 2)] + far[i + 1:6]
        assert lib.csa2_attn_weights(ctypes.byref(s), *at, ws, n, None) == INVALID, i
    for i in range(11):                                    # k_draft, v_draft, k_swa, v_swa, idx, weights, path, n_path, head, n_swa, mass
        at = far[:i] + [far[i] + (e // 2 if i < 4 else 4 if i == 10 else 2)] + far[i + 1:11]
        arr = (csa2.CTreeSlot * 1)(csa2.CTreeSlot(*at[:6]))
        assert lib.csa2_tree_commit(ctypes.byref(s), ctypes.cast(arr, ctypes.c_void_p), 1, *at[6:], ws, n, None) == INVALID, i
    for i in range(12):                                    # k, v, x, mass, n, the same behind, kept, kb
        off = 4 if i in (3, 8) else 2 if i in (4, 9, 10) else e // 2
        at = far[:i] + [far[i] + off] + far[i + 1:12]
        assert lib.csa2_kv_evict(ctypes.byref(one), 4000, 3000, 4, 64, *at, 1, ws, n1, None) == INVALID, i
    for i in range(4):                                     # x, out, pos, freqs
        at = far[:i] + [far[i] + (e // 2 if i < 2 else 2)] + far[i + 1:4]
        arr = (csa2.CRopeSlot * 1)(csa2.CRopeSlot(at[0], at[1], 3, 16, 0, 1 if dtype == "f32" else 0))
        assert lib.csa2_rope(ctypes.cast(arr, ctypes.c_void_p), 1, 4, 8, 0, at[2], at[3], 1.0, 0, None) == INVALID, i


def test_workspace_holds_the_key_lists_of_trees(csa2):
    """Short caches with long lists: the workspace grows by the lists of csa2_tree_attn; fp32 and long caches keep theirs."""
    small = _shape(csa2, batch=208, tokens=16, n_entries=57, topk=512, swa=128)
    lists = 208 // 2 * (2 * 512 + 128 + 16) * 4            # two tokens a list: both selections, the window, the drafted rows
    assert _ws(csa2, small) > lists
    plain = _shape(csa2, batch=208, tokens=16, n_entries=57, topk=512, swa=128, dtype="f32")
    assert _ws(csa2, plain) < lists + 65536
    big = dict(batch=208, tokens=16, n_entries=4096, topk=512, swa=128)
    assert _ws(csa2, _shape(csa2, **big)) == _ws(csa2, _shape(csa2, dtype="f32", **big))


def test_attn_weights_refusals(csa2):
    lib = csa2.lib()
    s = _shape(csa2)

    def call(s=s, ws=FAKE, nbytes=None, **kw):
        d = dict(q=FAKE, k_main=FAKE, idx=FAKE, lse=FAKE, live=None, weights=FAKE)
        d.update(kw)
        return lib.csa2_attn_weights(ctypes.byref(s), *d.values(), ws, _ws(csa2, s) if nbytes is None else nbytes, None)

    for n in ("q", "k_main", "idx", "lse", "weights"):
        assert call(**{n: None}) == INVALID, n
    assert call(q=MIS) == INVALID and call(k_main=MIS) == INVALID
    assert call(nbytes=0) == WORKSPACE and call(ws=None) == WORKSPACE
    assert call(s=_shape(csa2, batch=65536, n_entries=1, topk=1, swa=1)) == UNSUPPORTED


def test_tree_commit_refusals(csa2):
    lib = csa2.lib()
    s = _shape(csa2)
    slot = (FAKE, FAKE, FAKE, FAKE, FAKE, FAKE)

    def call(s=s, slots=(slot,), n=None, ws=FAKE, nbytes=None, **kw):
        d = dict(path=FAKE, n_path=FAKE, head=FAKE, n_swa=FAKE, mass=FAKE)
        d.update(kw)
        arr = (csa2.CTreeSlot * max(1, len(slots)))(*[csa2.CTreeSlot(*y) for y in slots])
        return lib.csa2_tree_commit(ctypes.byref(s), ctypes.cast(arr, ctypes.c_void_p), len(slots) if n is None else n, *d.values(),
                                    ws, _ws(csa2, s) if nbytes is None else nbytes, None)

    for n in ("path", "n_path", "head", "n_swa"):
        assert call(**{n: None}) == INVALID, n
    assert call(n=0) == INVALID and call(n=65) == INVALID and call(mass=FAKE + 4) == INVALID
    for i in range(4):
        assert call(slots=(slot, slot[:i] + (None,) + slot[i + 1:])) == INVALID
    assert call(slots=(slot[:4] + (None, FAKE),)) == INVALID and call(slots=(slot[:4] + (FAKE, None),)) == INVALID
    assert call(s=_shape(csa2, swa=0)) == INVALID
    assert call(s=_shape(csa2, batch=129, tokens=129)) == UNSUPPORTED
    assert call(nbytes=8) == WORKSPACE


def test_kv_evict_refusals(csa2):
    lib = csa2.lib()
    s = _shape(csa2, tokens=1)
    names = ("k", "v", "x", "mass", "n", "ko", "vo", "xo", "masso", "no", "kept", "kb")

    def call(s=s, trigger=4000, keep=3000, sink=4, recent=64, rnd=1, ws=FAKE, nbytes=None, **kw):
        d = {n: FAKE + i * STEP for i, n in enumerate(names)}
        d.update(kw)
        return lib.csa2_kv_evict(ctypes.byref(s), trigger, keep, sink, recent, *d.values(), rnd, ws,
                                 _ws(csa2, s) if nbytes is None else nbytes, None)

    for n in names[:-1]:
        assert call(**{n: None}) == INVALID, n
    for bad in (dict(keep=0), dict(trigger=2999), dict(trigger=4097), dict(sink=-1), dict(recent=-1), dict(sink=2000, recent=1001),
                dict(sink=3001, recent=0), dict(rnd=2), dict(mass=FAKE + 3 * STEP + 4), dict(masso=FAKE + 8 * STEP + 4)):
        assert call(**bad) == INVALID, bad
    at = {n: FAKE + i * STEP for i, n in enumerate(names)}
    assert call(ko=at["k"]) == INVALID                     # in place for one array only
    assert call(ko=at["k"] + 16) == INVALID                # overlaps its input
    assert call(ko=at["v"]) == INVALID and call(kept=at["k"]) == INVALID and call(kb=at["xo"]) == INVALID
    assert call(kb=at["kept"] + 4) == INVALID and call(vo=at["ko"]) == INVALID
    assert call(s=_shape(csa2, tokens=4)) == UNSUPPORTED
    assert call(nbytes=16) == WORKSPACE
    assert call(ws=FAKE + 16) == WORKSPACE


def test_binding_refuses_tensors_that_do_not_fit(csa2):
    torch = pytest.importorskip("torch")
    cpu = torch.zeros(4, 192)
    with pytest.raises(ValueError, match="CUDA"):
        csa2.rope([(cpu, cpu, 0)], torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.float64))
    with pytest.raises(ValueError, match="x must be"):
        csa2.rope([(cpu.half(), cpu.half(), 0)], torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.float64))
    with pytest.raises(ValueError, match="scaling"):
        csa2.rope_freqs(64, scaling="other", device="cpu")
    f, mag = csa2.rope_freqs(64, scaling="linear", factor=2.0, device="cpu")
    assert f.dtype == torch.float64 and tuple(f.shape) == (32,) and mag == 1.0

    class Fake(torch.Tensor):                              # a CUDA tensor as far as the checks look
        is_cuda = True

        def data_ptr(self):
            return FAKE

    t = torch.zeros(4, 3, dtype=torch.int32).as_subclass(Fake)
    assert csa2._arr(t, torch.int32, (4, 3), "t") == FAKE
    with pytest.raises(ValueError, match="shape"):
        csa2._arr(t, torch.int32, (4, 4), "t")
    with pytest.raises(TypeError, match="int32|float32"):
        csa2._arr(t, torch.float32, (4, 3), "t")
    with pytest.raises(ValueError, match="contiguous"):
        csa2._arr(t[:, ::2], torch.int32, (4, 2), "t")
    with pytest.raises(ValueError, match="is on"):
        csa2._arr(t, torch.int32, (4, 3), "t", torch.device("cuda", 1))
    with pytest.raises(TypeError, match="missing"):
        csa2._arr(None, torch.int32, (4, 3), "t")
    assert csa2._arr(None, torch.int32, (4, 3), "t", optional=True) is None
