"""Host-side checks of the 4-bit main cache and the norm with rotary positions (no GPU): the calls that the header refuses are
refused before anything is enqueued (the fake pointers are never dereferenced), and the references against hand cases."""
import ctypes
import math

import numpy as np
import pytest

from sparse_attention_decode_index_gb300 import build as B
from sparse_attention_decode_index_gb300 import workloads as W
from tests import kv4_reference as R

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
FAKE = 0x7f0000000000
STEP = 1 << 36                      # fake arrays far apart


@pytest.fixture(scope="module")
def csa2():
    B.build()
    from sparse_attention_decode_index_gb300 import csa2 as m
    m.lib()
    return m


def _shape(csa2, **kw):
    base = dict(batch=8, n_entries=4096, pool_blocks=0, tokens=1)
    base.update(kw)
    return csa2.c_shape(W.Shape(**base))


def _ws(csa2, s):
    return csa2.lib().csa2_workspace_bytes(ctypes.byref(s))


def test_entry_bytes(csa2):
    lib = csa2.lib()
    for dk, dv in ((192, 128), (1, 1), (16, 16), (17, 15), (100, 72), (1024, 1024), (64, 63)):
        assert lib.csa2_kv4_bytes(dk, dv) == R.entry_bytes(dk, dv)
    assert lib.csa2_kv4_bytes(192, 128) == 192
    for dk, dv in ((0, 1), (1, 0), (1025, 1), (1, 1025), (-1, 16)):
        assert lib.csa2_kv4_bytes(dk, dv) == 0


def test_reference_by_hand():
    """16 numbers whose scale is exact, ties of both kinds, a scale that is rounded up and one that saturates."""
    x = np.array([6.0, -6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, 0.0, 0.26, 0.24, 4.9, 5.1])
    codes, scales = R.quantise(x, 0)
    assert scales.tolist() == [0x38]                       # 1.0: exponent field 7, mantissa 0
    want = [6, -6, 0, 1, 1, 2, 2, 4, 4, 0, -1, 0, 0.5, 0, 4, 6]
    assert R.values(codes, scales, 16, 0).tolist() == want
    assert R.values(*R.quantise(x * 2.0 ** 5, 5), 16, 5).tolist() == [32.0 * w for w in want]
    assert R.SCALES[126] == 448.0 and R.SCALES[1] == 2.0 ** -9 and len(R.SCALES) == 127
    codes, scales = R.quantise(np.full(16, 10000.0), 0)    # beyond 2,688: the largest code of the largest scale
    assert R.values(codes, scales, 16, 0).tolist() == [2688.0] * 16
    codes, scales = R.quantise(np.full(16, 1e-6), 0)       # below the smallest scale's first code
    assert scales.tolist() == [1] and not codes.any()
    codes, scales = R.quantise(np.full(16, 6 * 1.0625), 0)   # a sixth between 1 and 1.125: to the even one
    assert R.SCALES[scales[0]] == 1.0
    codes, scales = R.quantise(np.full(16, 6 * 1.1875), 0)
    assert R.SCALES[scales[0]] == 1.25
    k = np.arange(1, 18, dtype=float)                      # a group and a part of one
    e = R.pack(k, -k[:3], 0, 0)
    assert len(e) == 32 and e[24:27].tolist() == R.quantise(k, 0)[1].tolist() + R.quantise(k[:3], 0)[1].tolist()
    back = R.unpack(e, 17, 3, 0, 0)
    assert back[0][16] == 17.0 or abs(back[0][16] - 17.0) <= 17.0 / 16 and len(back[1]) == 3


def test_norm_rope_refusals(csa2):
    lib = csa2.lib()
    good = dict(x=FAKE, out=FAKE + STEP, gain=FAKE + 2 * STEP, x_stride=64 * 192, out_stride=64 * 192, heads=64, dim=192, rot_off=128,
                dtype=0, gain_each=0)

    def call(slots=(good,), n=None, rows=4, rot=64, inter=0, center=0, pos=FAKE + 4 * STEP, freqs=FAKE + 5 * STEP, mag=1.0, eps=1e-6):
        arr = (csa2.CNormRopeSlot * max(1, len(slots)))(*[csa2.CNormRopeSlot(*y.values()) for y in slots])
        return lib.csa2_norm_rope(ctypes.cast(arr, ctypes.c_void_p), len(slots) if n is None else n, rows, rot, inter, center, pos, freqs,
                                  mag, eps, None)

    for bad in (dict(n=0), dict(n=17), dict(rows=0), dict(rot=-2), dict(rot=63), dict(inter=2), dict(center=2), dict(center=-1),
                dict(pos=None), dict(freqs=None), dict(freqs=FAKE + 5 * STEP + 4), dict(pos=FAKE + 2), dict(mag=0.0), dict(mag=math.nan),
                dict(mag=math.inf), dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf), dict(rot=66)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(x=None), dict(out=None), dict(heads=0), dict(dim=0), dict(rot_off=-1), dict(rot_off=129), dict(dtype=2),
                dict(gain_each=2), dict(x_stride=64 * 192 - 1), dict(out_stride=64 * 192 - 1), dict(x=FAKE + 1), dict(gain=FAKE + 2),
                dict(out=FAKE + 2),                        # over its input without being it
                dict(out=FAKE, out_stride=64 * 192 + 8),   # its input with other strides
                dict(out=FAKE + 4 * STEP), dict(out=FAKE + 5 * STEP), dict(out=FAKE + 2 * STEP)):   # positions, frequencies, gains
        assert call(slots=({**good, **bad},)) == INVALID, bad
    assert call(slots=({**good, "heads": 1025, "x_stride": 1 << 20, "out_stride": 1 << 20},)) == UNSUPPORTED
    assert call(slots=({**good, "dim": 1025, "x_stride": 1 << 20, "out_stride": 1 << 20},)) == UNSUPPORTED
    assert call(slots=({**good, "x_stride": (1 << 28) + 8},)) == UNSUPPORTED
    assert call(rot=1026, slots=({**good, "dim": 1026, "rot_off": 0, "x_stride": 1 << 20, "out_stride": 1 << 20},)) == UNSUPPORTED
    other = dict(good, x=FAKE + 3 * STEP)
    assert call(slots=(good, other)) == INVALID            # one output twice
    assert call(slots=(good, dict(other, out=FAKE))) == INVALID   # over another slot's input
    # two parts of one projection, in place: the second overlaps the first by one number, from either side
    wide = dict(good, out=FAKE, x_stride=66 * 192, out_stride=66 * 192)
    for at in (2 * 64 * 192 - 2, 2 * 65 * 192 + 2, 2 * (66 * 192 * 2 + 64 * 192) - 2):
        part = dict(wide, x=FAKE + at, out=FAKE + at, heads=1)
        assert call(slots=(wide, part)) == INVALID, at


NAMES = {"append": ("n_new", "k_new", "v_new", "kidx_new", "kv4", "k_idx", "kb", "n_valid"),
         "rows": ("kv4", "idx", "k_out", "v_out"),
         "attn": ("q", "kv4", "idx", "k_swa", "v_swa", "n_swa", "out", "lse")}
WRITTEN = {"append": ("kv4", "k_idx", "kb", "n_valid"), "rows": ("k_out", "v_out"), "attn": ("out", "lse")}


def _call(csa2, op, s, ws=FAKE - STEP, nbytes=None, exps=(0, 0), max_new=3, n_rows=5, rounded=1, **kw):
    lib = csa2.lib()
    d = {n: FAKE + i * STEP for i, n in enumerate(NAMES[op])}
    d.update(kw)
    n = _ws(csa2, s) if nbytes is None else nbytes
    p = list(d.values())
    if op == "append":
        return lib.csa2_kv4_append(ctypes.byref(s), max_new, *p, *exps, rounded, ws, n, None)
    if op == "rows":
        return lib.csa2_kv4_rows(ctypes.byref(s), *p[:2], n_rows, *p[2:], *exps, ws, n, None)
    return lib.csa2_kv4_attn(ctypes.byref(s), *p, *exps, ws, n, None)


@pytest.mark.parametrize("op", list(NAMES))
def test_kv4_refusals(csa2, op):
    s = _shape(csa2)
    for n in NAMES[op]:
        if n not in ("kb", "lse"):
            assert _call(csa2, op, s, **{n: None}) == INVALID, n
        assert _call(csa2, op, s, **{n: FAKE + 9 * STEP + 1}) == INVALID, n
    assert _call(csa2, op, s, kv4=FAKE + 8) == INVALID
    for exps in ((65, 0), (-65, 0), (0, 65), (0, -65)):
        assert _call(csa2, op, s, exps=exps) == INVALID
    assert _call(csa2, op, s, nbytes=_ws(csa2, s) - 1) == WORKSPACE
    assert _call(csa2, op, s, ws=FAKE - STEP + 16) == WORKSPACE
    bad = _shape(csa2)
    bad.topk = 0
    assert _call(csa2, op, bad, nbytes=1 << 30) == INVALID
    if op == "append":
        assert _call(csa2, op, s, max_new=0) == INVALID and _call(csa2, op, s, max_new=-1) == INVALID
        assert _call(csa2, op, s, rounded=2) == INVALID
        assert _call(csa2, op, _shape(csa2, tokens=2)) == UNSUPPORTED
        assert _call(csa2, op, _shape(csa2, batch=65536, n_entries=1)) == UNSUPPORTED
    if op == "rows":
        assert _call(csa2, op, s, n_rows=0) == INVALID
        assert _call(csa2, op, s, n_rows=1 << 28) == UNSUPPORTED
    if op == "attn":
        assert _call(csa2, op, s, ws=None, nbytes=0) == WORKSPACE
        assert _call(csa2, op, _shape(csa2, batch=65536, n_entries=1)) == UNSUPPORTED
        for n in ("q", "k_swa", "v_swa", "out"):
            assert _call(csa2, op, s, **{n: FAKE + 9 * STEP + 8}) == INVALID, n


@pytest.mark.parametrize("op", list(NAMES))
def test_kv4_outputs_over_other_arrays_are_refused(csa2, op):
    """A written array that shares a byte with any other, whichever starts first, or with the workspace."""
    s = _shape(csa2, batch=2, n_entries=64, topk=8, swa=4)
    size = dict(n_new=8, k_new=6 * 384, v_new=6 * 256, kidx_new=6 * 128, kv4=2 * 64 * 192, k_idx=2 * 64 * 128, kb=2 * 8 * 128, n_valid=8,
                idx=2 * (5 if op == "rows" else 8) * 4, k_out=10 * 384, v_out=10 * 256, q=2 * 64 * 384, k_swa=8 * 384, v_swa=8 * 256,
                n_swa=8, out=2 * 64 * 256, lse=2 * 64 * 4)
    at = {n: FAKE + i * STEP for i, n in enumerate(NAMES[op])}
    for w in WRITTEN[op]:
        for n in NAMES[op]:
            if n == w:
                continue
            for p in (at[n], at[n] + (size[n] - 1) // 16 * 16, at[n] - (size[w] - 1) // 16 * 16):
                assert _call(csa2, op, s, **{w: p}) == INVALID, (w, n)
    ws, n = FAKE - STEP, _ws(csa2, s)
    for x in NAMES[op]:
        for p in (ws, ws + n - 16, ws - (size[x] - 1) // 16 * 16):
            if p + size[x] > ws:
                assert _call(csa2, op, s, **{x: p}) == INVALID, x


def test_wait_hook_refusals(csa2):
    """The test hook of the attention's waits checks what the attention checks, its limit, and that the fast kernel serves the shape."""
    def call(s, limit=2000000, **kw):
        d = {n: FAKE + i * STEP for i, n in enumerate(NAMES["attn"])}
        d.update(kw)
        return csa2.lib().csa2_debug_kv4_wait_timeout(ctypes.byref(s), *d.values(), 0, 0, limit, FAKE - STEP, _ws(csa2, s), None)

    s = _shape(csa2)
    for limit in (0, 9999, 200000001):
        assert call(s, limit) == INVALID
    assert call(s, q=None) == INVALID and call(s, out=FAKE) == INVALID
    assert call(_shape(csa2, q_heads=16)) == UNSUPPORTED
