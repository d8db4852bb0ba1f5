"""Host-side checks of the attention side: every refusal of the C entry points
and of the binding, phase tables, tree masks.  None of these touch a GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

from long_context_misa_b200 import attention as A
from long_context_misa_b200 import misa as M

FAKE = 0x10000  # 16-byte aligned, never dereferenced on the host
L = M._lib
by = ctypes.byref
INV, UNS, WS = M.MISA_ERR_INVALID, M.MISA_ERR_UNSUPPORTED, M.MISA_ERR_WORKSPACE


def kv(**f):
    d = dict(k=FAKE, v=FAKE, k_scale=None, v_scale=None, seq_len=FAKE, status=None, n_seq=2, L_cap=4096, H_kv=4, d=128,
             dtype=M.MISA_KEY_BF16)
    return A.misa_kv(**{**d, **f})


def rope(**f):
    return A.misa_rope(**{**dict(phase=FAKE, rot=64, first=0, layout=0, amplitude=1.0), **f})


def rows(**f):
    d = dict(x=FAKE, y=FAKE, pos=FAKE, x_row=512, x_head=128, y_row=512, y_head=128, n=3, H=4, d=128)
    return A.misa_rope_rows(**{**d, **f})


def new(**f):
    d = dict(k=FAKE, v=FAKE, k_seq=512, k_tok=512, k_head=128, v_seq=512, v_tok=512, v_head=128)
    return A.misa_new_kv(**{**d, **f})


def queries(**f):
    return A.misa_attend_queries(**{**dict(q=FAKE << 8, q_seq=FAKE, q_pos=FAKE, n_q=3, H=8, scale=0.1), **f})


def draft(**f):
    return A.misa_draft(**{**dict(start=FAKE, mask=FAKE, n=5), **f})


def test_exports_every_declared_symbol():
    names = M.header_symbols(A.HEADER)
    assert sorted(names) == sorted(["misa_rope_phases", "misa_apply_rope", "misa_append_kv", "misa_read_kv",
                                    "misa_attend", "misa_attend_workspace_bytes"])
    for n in names:
        assert hasattr(L, n), n


BAD_KV = [(dict(k=None), INV), (dict(v=None), INV), (dict(seq_len=None), INV), (dict(dtype=5), INV),
          (dict(k_scale=FAKE), INV), (dict(v_scale=FAKE), INV), (dict(dtype=M.MISA_KEY_FP8_E4M3), INV),
          (dict(dtype=M.MISA_KEY_FP8_E4M3, k_scale=FAKE), INV), (dict(d=96), UNS), (dict(d=0), UNS),
          (dict(n_seq=0), INV), (dict(L_cap=0), INV), (dict(H_kv=0), INV), (dict(H_kv=129), UNS),
          (dict(L_cap=(1 << 18) + 1), UNS), (dict(k=FAKE + 8), INV), (dict(v=FAKE + 2), INV)]


@pytest.mark.parametrize("bad,status", BAD_KV)
def test_cache_refusals(bad, status):
    c = kv(**bad)
    assert L.misa_append_kv(by(c), by(new()), FAKE, 1, None, None, 1, None) == status
    assert L.misa_read_kv(by(c), FAKE, FAKE, 1, 1, FAKE, FAKE, None) == status
    assert L.misa_attend(by(c), by(queries(H=c.H_kv if c.H_kv > 0 else 1)), FAKE, 4, None, FAKE, None, FAKE, 1 << 30,
                         None) == status
    assert M.last_error() != ""


@pytest.mark.parametrize("bad", [dict(phase=None), dict(rot=3), dict(rot=0), dict(first=-2), dict(first=66),
                                 dict(rot=130), dict(layout=2), dict(amplitude=math.inf), dict(amplitude=math.nan)])
def test_rope_refusals(bad):
    assert L.misa_apply_rope(by(rope(**bad)), by(rows()), 1, None) == INV
    assert L.misa_append_kv(by(kv()), by(new()), FAKE, 1, by(rope(**bad)), None, 1, None) == INV


@pytest.mark.parametrize("bad,status", [(dict(x=None), INV), (dict(y=None), INV), (dict(pos=None), INV),
                                        (dict(n=-1), INV), (dict(H=-1), INV), (dict(d=0), INV), (dict(d=1032), UNS),
                                        (dict(x_row=1024), INV), (dict(y_head=256), INV)])
def test_rope_rows_refusals(bad, status):
    assert L.misa_apply_rope(by(rope()), by(rows(**bad)), 1, None) == status


def test_rope_group_counts():
    g = (A.misa_rope_rows * 5)(*[rows() for _ in range(5)])
    assert L.misa_apply_rope(by(rope()), g, 0, None) == INV
    assert L.misa_apply_rope(by(rope()), g, 5, None) == INV
    assert L.misa_apply_rope(None, g, 1, None) == INV
    assert L.misa_apply_rope(by(rope()), None, 1, None) == INV
    with pytest.raises(ValueError):
        A.apply_rope(A.Rope(64, device="cpu"), [])


def test_append_refusals():
    def call(c=kv(), n=new(), pos=FAKE, count=1, r=None, rp=None):
        return L.misa_append_kv(by(c), by(n) if n else None, pos, count, r, rp, 1, None)
    assert call(count=0) == INV
    assert call(count=4097) == INV
    assert call(n=None) == INV
    assert call(n=new(k=None)) == INV
    assert call(n=new(v=None)) == INV
    assert call(pos=None) == INV
    assert call(rp=FAKE) == INV                     # rope_pos without rope
    assert call(n=new(k=FAKE + 8)) == INV
    for s in ("k_seq", "k_tok", "k_head", "v_seq", "v_tok", "v_head"):
        assert call(n=new(**{s: 132})) == INV


def test_append_positions_that_overlap_the_lengths():
    """seq_len itself may say where the tokens go; an array that shares a part of it may not."""
    c = kv(n_seq=4)
    for off in (-12, -4, 4, 12):
        assert L.misa_append_kv(by(c), by(new()), c.seq_len + off, 1, None, None, 1, None) == INV
    M.debug_fail_next(4)
    try:
        for off, commit in ((-4, 0), (0, 1), (16, 1), (-16, 1)):
            assert L.misa_append_kv(by(c), by(new()), c.seq_len + off, 1, None, None, commit, None) == M.MISA_ERR_CUDA
    finally:
        M.debug_fail_next(0)


def test_outputs_that_meet_are_refused():
    c, q = kv(), queries()
    size = q.n_q * q.H * c.d * 2
    for off in (0, 16, size - 16, 16 - size):
        assert L.misa_attend(by(c), by(q), FAKE, 4, None, q.q + off, None, FAKE, 1 << 30, None) == INV
    rows_bytes = 3 * 4 * c.H_kv * c.d * 2
    for off in (0, 16, rows_bytes - 16):
        assert L.misa_read_kv(by(c), FAKE, FAKE, 3, 4, FAKE, FAKE + off, None) == INV
    for bad in (dict(y_row=0, n=2), dict(y_head=0, H=2), dict(y_row=128, y_head=128, n=2, H=2),
                dict(y_row=128, y_head=64, n=1, H=2, d=128), dict(y_row=256, y_head=256, n=2, H=2, d=128)):
        bad = {"n": 2, "H": 2, "d": 128, **bad, "y": FAKE + (1 << 20)}
        assert L.misa_apply_rope(by(rope()), by(rows(**bad)), 1, None) == INV, bad
    two = (A.misa_rope_rows * 2)(rows(), rows())
    assert L.misa_apply_rope(by(rope()), two, 2, None) == INV       # the same rows twice
    two = (A.misa_rope_rows * 2)(rows(y=FAKE + (1 << 20)), rows(x=FAKE + (1 << 20), y=FAKE + (1 << 21)))
    assert L.misa_apply_rope(by(rope()), two, 2, None) == INV       # what the other writes
    M.debug_fail_next(3)
    try:
        good = dict(n=3, H=4, d=128, y=FAKE + (1 << 20))
        for st in (dict(y_row=512, y_head=128), dict(y_row=128, y_head=384), dict(y_row=9000, y_head=2000)):
            assert L.misa_apply_rope(by(rope()), by(rows(**good, **st)), 1, None) == M.MISA_ERR_CUDA
    finally:
        M.debug_fail_next(0)


def _addresses(p, row, head, n, H, d):
    return {p // 2 + i * row + h * head + e for i in range(n) for h in range(H) for e in range(d)}


def test_rotated_rows_that_meet_are_refused_and_no_others():
    """Random strides and offsets against the sets of elements themselves: in and out of one group, and of two."""
    rng = np.random.default_rng(3)
    good = bad = 0
    base = 1 << 24

    def strides(n, H, d):
        if rng.integers(2):                            # heads inside rows, or the other way round
            head = d + int(rng.integers(0, 7))
            return head * (H - 1) + d + int(rng.integers(0, 3 * d)), head
        row = d + int(rng.integers(0, 7))
        return row, row * (n - 1) + d + int(rng.integers(0, 2 * d))

    for _ in range(4000):
        n, H, d = int(rng.integers(1, 6)), int(rng.integers(1, 4)), int(rng.choice([8, 16]))
        m, J = int(rng.integers(1, 6)), int(rng.integers(1, 4))
        (xr, xh), (yr, yh) = strides(n, H, d), strides(n, H, d)
        if rng.integers(2):
            yr, yh = xr, xh                            # slices of one projection
        if rng.integers(6) == 0:
            xr = 0                                     # one row for all
        pr, ph = (xr, xh) if rng.integers(2) and xr else strides(m, J, d)
        if rng.integers(8) == 0:
            yr, yh = -yr, -yh
        x = base
        y = base + 2 * int(rng.integers(-120, 120))
        z = base + 2 * int(rng.integers(-400, 400))
        one = rows(x=x, y=y, x_row=xr, x_head=xh, y_row=yr, y_head=yh, n=n, H=H, d=d)
        two = rows(x=z, y=z, x_row=pr, x_head=ph, y_row=pr, y_head=ph, n=m, H=J, d=d)
        X, Y, Z = _addresses(x, xr, xh, n, H, d), _addresses(y, yr, yh, n, H, d), _addresses(z, pr, ph, m, J, d)
        if len(Z) < m * J * d or len(Y) < n * H * d:
            continue
        in_place = x == y and (xr, xh) == (yr, yh)
        first = x != y and bool(X & Y) or x == y and not in_place
        both = first or bool(Z & (X | Y))
        r = rope(rot=8)
        for groups, meets in (((one,), first), ((one, two), both), ((two, one), both)):
            M.debug_fail_next(1)
            try:
                st = L.misa_apply_rope(by(r), (A.misa_rope_rows * len(groups))(*groups), len(groups), None)
            finally:
                M.debug_fail_next(0)
            assert st == (INV if meets else M.MISA_ERR_CUDA), (st, M.last_error(), n, H, d, xr, xh, yr, yh, y - x, pr, ph, z - x)
            good, bad = good + (not meets), bad + meets
    assert good > 1000 and bad > 1000


def test_attention_outputs_that_meet_are_refused():
    c, q = kv(L_cap=65536), queries(n_q=1)
    need = L.misa_attend_workspace_bytes(by(c), by(q), 0, 0)
    row, out, lse, ws = q.H * c.d * 2, 1 << 32, 1 << 33, 1 << 34

    def call(out=out, lse=lse, ws=ws):
        return L.misa_attend(by(c), by(q), None, 0, None, out, lse, ws, need, None)

    M.debug_fail_next(7)
    try:
        for ok in (dict(), dict(lse=out + row), dict(lse=out - 4 * q.H), dict(ws=out + row), dict(ws=out - need),
                   dict(lse=ws + need), dict(lse=None)):
            assert call(**ok) == M.MISA_ERR_CUDA, ok
    finally:
        M.debug_fail_next(0)
    for bad in (dict(lse=out), dict(lse=out + row - 4), dict(lse=q.q), dict(lse=q.q - 4 * q.H + 4), dict(ws=out + row - 16),
                dict(ws=out - need + 16), dict(ws=q.q), dict(lse=ws), dict(lse=ws + need - 4)):
        assert call(**bad) == INV, bad


def test_host_tensors_are_refused():
    """Pointers to host memory never reach a kernel."""
    k = torch.zeros(1, 8, 1, 64, dtype=torch.bfloat16)
    n = torch.zeros(1, dtype=torch.int32)
    c = A.KVCache(k, k.clone(), None, None, n)
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    for call in (lambda: A.append_kv(c, k[:, :1], k[:, :1], n), lambda: A.read_kv(c, n, n.view(1, 1)),
                 lambda: A.attend(c, A.AttentionQueries(x, n, n)),
                 lambda: A.apply_rope(A.Rope(64, device="cpu"), [(x, n, x)])):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_read_refusals():
    c = kv()
    assert L.misa_read_kv(by(c), FAKE, FAKE, -1, 1, FAKE, FAKE << 8, None) == INV
    assert L.misa_read_kv(by(c), FAKE, FAKE, 1, 0, FAKE, FAKE << 8, None) == INV
    assert L.misa_read_kv(by(c), None, FAKE, 1, 1, FAKE, FAKE << 8, None) == INV
    assert L.misa_read_kv(by(c), FAKE, None, 1, 1, FAKE, FAKE << 8, None) == INV
    assert L.misa_read_kv(by(c), FAKE, FAKE, 1, 1, None, None, None) == INV
    assert L.misa_read_kv(by(c), FAKE, FAKE, 1, 1, FAKE + 4, FAKE << 8, None) == INV


@pytest.mark.parametrize("bad,status", [(dict(q=None), INV), (dict(q_seq=None), INV), (dict(q_pos=None), INV),
                                        (dict(n_q=-1), INV), (dict(n_q=65536), INV), (dict(H=0), INV), (dict(H=6), INV),
                                        (dict(H=132), UNS), (dict(scale=math.nan), INV), (dict(scale=math.inf), INV),
                                        (dict(q=(FAKE << 8) + 8), INV)])
def test_attend_query_refusals(bad, status):
    assert L.misa_attend(by(kv()), by(queries(**bad)), FAKE, 4, None, FAKE, None, FAKE, 1 << 30, None) == status


def test_attend_refusals():
    def call(topk=FAKE, k=4, d=None, out=FAKE, ws=FAKE, nb=1 << 30, c=kv(), q=queries()):
        return L.misa_attend(by(c), by(q), topk, k, by(d) if d else None, out, None, ws, nb, None)
    assert call(k=0) == INV
    assert call(k=-1) == INV
    assert call(topk=None) == INV
    assert call(k=(1 << 18) + 1) == UNS
    assert call(out=None) == INV
    assert call(out=FAKE + 8) == INV
    assert call(d=draft(n=0)) == INV
    assert call(d=draft(n=-1)) == INV
    assert call(d=draft(n=1025)) == UNS
    assert call(d=draft(start=None)) == INV
    assert call(d=draft(mask=None)) == INV
    big = dict(topk=None, k=0, c=kv(L_cap=65536), q=queries(n_q=1))  # a long prefix: split over CTAs
    need = L.misa_attend_workspace_bytes(by(big["c"]), by(big["q"]), 0, 0)
    assert need > 0 and need % 256 == 0
    assert call(nb=need - 1, **big) == WS
    assert call(ws=None, nb=need, **big) == INV
    assert call(ws=FAKE + 8, nb=need, **big) == INV
    assert L.misa_attend_workspace_bytes(by(kv(d=96)), by(queries()), 0, 0) == 0
    assert L.misa_attend_workspace_bytes(None, by(queries()), 0, 0) == 0
    assert L.misa_attend(None, by(queries()), FAKE, 4, None, FAKE, None, FAKE, 1 << 30, None) == INV
    assert L.misa_attend(by(kv()), None, FAKE, 4, None, FAKE, None, FAKE, 1 << 30, None) == INV


def test_empty_batches_have_no_memory():
    """Nothing to do is done whatever the pointers: torch gives an empty tensor's as 0."""
    none = queries(n_q=0, q=None, q_seq=None, q_pos=None)
    for d in (None, draft(start=None, mask=None), draft(mask=None)):
        for k in (0, 4):
            assert L.misa_attend(by(kv()), by(none), None, k, by(d) if d else None, None, None, None, 0, None) == M.MISA_OK
    assert L.misa_attend(by(kv()), by(none), FAKE, 0, None, None, None, None, 0, None) == INV
    assert L.misa_attend(by(kv()), by(none), None, 4, by(draft(n=0)), None, None, None, 0, None) == INV
    assert L.misa_read_kv(by(kv()), None, None, 0, 3, None, None, None) == M.MISA_OK
    assert L.misa_read_kv(by(kv()), None, None, 0, 0, None, None, None) == INV
    for g in (rows(n=0, x=None, y=None, pos=None, y_row=1024), rows(H=0, x=None, y=None, x_head=64, y_head=64, n=2)):
        assert L.misa_apply_rope(by(rope()), by(g), 1, None) == M.MISA_OK
        assert L.misa_apply_rope(by(rope(rot=3)), by(g), 1, None) == INV


def test_a_growing_workspace_keeps_nothing():
    ws = M.Workspace("cpu")
    for n in range(1000, 100000, 1000):
        assert ws.get(n).numel() == n
    assert ws.get(5).numel() == 99000 and ws.outgrown == []


def test_injected_failures():
    M.debug_fail_next(4)
    try:
        assert L.misa_append_kv(by(kv()), by(new()), FAKE, 0, None, None, 1, None) == INV  # consumes none
        assert L.misa_apply_rope(by(rope()), by(rows()), 1, None) == M.MISA_ERR_CUDA
        assert L.misa_append_kv(by(kv()), by(new()), FAKE, 1, None, None, 1, None) == M.MISA_ERR_CUDA
        assert L.misa_read_kv(by(kv()), FAKE, FAKE, 1, 1, FAKE, FAKE << 8, None) == M.MISA_ERR_CUDA
        assert L.misa_attend(by(kv()), by(queries()), FAKE, 4, None, FAKE, None, FAKE, 1 << 30, None) == M.MISA_ERR_CUDA
        assert "injected" in M.last_error()
    finally:
        M.debug_fail_next(0)


@pytest.mark.parametrize("args", [dict(rot=1), dict(rot=0), dict(base=0.0), dict(base=-1.0), dict(base=math.inf),
                                  dict(base=math.nan), dict(scaling=9), dict(scaling=1, factor=0.0),
                                  dict(scaling=3, factor=2.0, orig=0.0), dict(scaling=3, factor=2.0, fast=1.0, slow=2.0),
                                  dict(scaling=3, factor=2.0, slow=0.0), dict(scaling=3, factor=math.inf)])
def test_phase_refusals(args):
    a = {**dict(rot=64, base=1e4, scaling=0, factor=1.0, orig=4096.0, fast=32.0, slow=1.0), **args}
    buf = (ctypes.c_uint64 * 64)()
    assert L.misa_rope_phases(buf, a["rot"], a["base"], a["scaling"], a["factor"], a["orig"], a["fast"], a["slow"]) == INV
    assert L.misa_rope_phases(None, 64, 1e4, 0, 1.0, 1.0, 1.0, 1.0) == INV


def _turns(r):
    return np.array([int(x) & (2**64 - 1) for x in r.phases.tolist()], dtype=object)


@pytest.mark.parametrize("rot", [2, 6, 64, 128])
def test_phases_are_the_frequencies(rot):
    i = np.arange(rot // 2)
    f = 10000.0 ** (-2.0 * i / rot) / (2 * math.pi)
    # the doubles that lead to a phase are right to 2^-51; phases to 2^-64
    tol = 2.0 ** 64 * f * 2.0 ** -51 + 1
    assert np.all(np.abs(_turns(A.Rope(rot, device="cpu")) - f * 2.0 ** 64) <= tol)
    lin = A.Rope(rot, scaling="linear", factor=8.0, device="cpu")
    assert np.all(np.abs(_turns(lin) - f / 8 * 2.0 ** 64) <= tol)
    ntk = A.Rope(rot, scaling="ntk", factor=8.0, device="cpu")
    b = 10000.0 * 8.0 ** (rot / (rot - 2)) if rot > 2 else 10000.0
    g = b ** (-2.0 * i / rot) / (2 * math.pi)
    assert np.all(np.abs(_turns(ntk) - g * 2.0 ** 64) <= 2.0 ** 64 * g * 2.0 ** -48 + 1)
    assert A.Rope(rot, device="cpu").amplitude == 1.0


def test_yarn_keeps_fast_pairs_and_interpolates_slow_ones():
    f = _turns(A.Rope(64, device="cpu"))
    y = _turns(A.Rope(64, scaling="yarn", factor=16.0, orig_len=4096, device="cpu"))
    r = np.array([float(a) / float(b) for a, b in zip(y, f)])
    turns = 4096 * f.astype(float) / 2.0 ** 64  # in the original length
    assert np.all(np.abs(r[turns > 40] - 1) < 1e-12) and np.all(np.abs(r[turns < 0.7] - 1 / 16) < 1e-12)
    assert np.all(np.diff(r) <= 1e-12)
    assert A.Rope(64, scaling="yarn", factor=16.0, device="cpu").amplitude == pytest.approx(0.1 * math.log(16) + 1)


def test_tree_mask():
    m = A.tree_mask([-1, 0, 0, 1, -1, 4])
    assert m.tolist() == [[0b1], [0b11], [0b101], [0b1011], [0b10000], [0b110000]]
    chain = A.tree_mask(list(range(-1, 69)), n=100)
    assert tuple(chain.shape) == (70, 4)
    full = [int(x) & 0xFFFFFFFF for x in chain[69]]
    assert full == [0xFFFFFFFF, 0xFFFFFFFF, 0b111111, 0]
    for bad in ([0], [-1, 1], [-2]):
        with pytest.raises(ValueError):
            A.tree_mask(bad)
    with pytest.raises(ValueError):
        A.tree_mask([-1, 0], n=1)


def test_tree_mask_of_no_nodes():
    """A sequence without drafted tokens has no rows of words."""
    assert tuple(A.tree_mask([], n=40).shape) == (0, 2) and A.tree_mask([], n=40).dtype == torch.int32
    assert tuple(A.tree_mask([]).shape) == (0, 0)


def test_binding_refusals():
    k = torch.zeros(2, 16, 4, 128, dtype=torch.bfloat16)
    n = torch.zeros(2, dtype=torch.int32)
    s = torch.zeros(2, 16, 4)
    c = A.KVCache(k, k.clone(), None, None, n)
    with pytest.raises(ValueError):
        A.KVCache(k, k[:, :8], None, None, n)
    with pytest.raises(ValueError):
        A.KVCache(k.transpose(0, 1), k.transpose(0, 1), None, None, n)
    with pytest.raises(ValueError):
        A.KVCache(k, k, s, s, n)                                    # scales of a bf16 cache
    with pytest.raises(ValueError):
        A.KVCache(k.to(torch.uint8), k.to(torch.uint8), s, None, n)
    with pytest.raises(ValueError):
        A.KVCache(k.to(torch.uint8), k.to(torch.uint8), s, s[:, :8], n)
    with pytest.raises(TypeError):
        A.KVCache(k.float(), k.float(), None, None, n)
    with pytest.raises(TypeError):
        A.KVCache(k, k.view(torch.int16), None, None, n)
    with pytest.raises(TypeError):
        A.KVCache(k, k, None, None, n.long())
    with pytest.raises(ValueError):
        A.KVCache(k, k, None, None, n[:1])
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    idx = torch.zeros(3, dtype=torch.int32)
    qs = A.AttentionQueries(q, idx, idx)
    assert (qs.n_q, qs.H, qs.d) == (3, 8, 128) and qs.scale == pytest.approx(128 ** -0.5)
    with pytest.raises(TypeError):
        A.AttentionQueries(q.float(), idx, idx)
    with pytest.raises(TypeError):
        A.AttentionQueries(q, idx.long(), idx)
    with pytest.raises(ValueError):
        A.AttentionQueries(q, idx[:2], idx)
    with pytest.raises(ValueError):
        A.attend(c, A.AttentionQueries(q[:, :, :64].contiguous(), idx, idx))
    with pytest.raises(ValueError):
        A.attend(c, qs, topk=torch.zeros(2, 4, dtype=torch.int32))
    with pytest.raises(TypeError):
        A.attend(c, qs, topk=torch.zeros(3, 4, dtype=torch.int64))
    with pytest.raises(ValueError):
        A.attend(c, qs, draft=A.Draft(n, torch.zeros(2, 1, dtype=torch.int32), 5))
    with pytest.raises(ValueError):
        A.attend(c, qs, draft=A.Draft(n[:1], torch.zeros(3, 1, dtype=torch.int32), 5))
    with pytest.raises(ValueError):
        A.Draft(n, torch.zeros(3, 1, dtype=torch.int32), 33)
    with pytest.raises(TypeError):
        A.Draft(n, torch.zeros(3, 1), 3)
    kn = torch.zeros(2, 1, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        A.append_kv(c, kn[:1], kn, n)
    with pytest.raises(ValueError):
        A.append_kv(c, kn, torch.zeros(2, 2, 4, 128, dtype=torch.bfloat16), n)
    with pytest.raises(TypeError):
        A.append_kv(c, kn.float(), kn, n)
    with pytest.raises(ValueError):
        A.read_kv(c, n, torch.zeros(3, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        A.Rope(63, device="cpu")
    with pytest.raises(ValueError):
        A.Rope(64, layout="spiral", device="cpu")
    with pytest.raises(ValueError):
        A.Rope(64, scaling="other", device="cpu")
    r = A.Rope(64, device="cpu")
    x = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        A.apply_rope(r, [(x.float(), idx, x.float())])
    with pytest.raises(ValueError):
        A.apply_rope(r, [(x, idx, x[:2])])
    with pytest.raises(ValueError):
        A.apply_rope(r, [(x.transpose(1, 2), idx, x.transpose(1, 2))])


def test_a_list_of_nothing_stays_a_list(monkeypatch):
    """topk [n_q][0] has no memory (a NULL pointer): the call must not take it for the absence of a list."""
    k = torch.zeros(2, 16, 4, 128, dtype=torch.bfloat16)
    n = torch.zeros(2, dtype=torch.int32)
    c = A.KVCache(k, k.clone(), None, None, n)
    seen = []

    def call(fn, device, stream, kv_p, qs_p, topk, entries, *rest):
        seen.append((entries, (ctypes.c_int32 * (3 * entries)).from_address(topk)[:]))

    monkeypatch.setattr(A, "_call", call)
    idx = torch.zeros(3, dtype=torch.int32)
    qs = A.AttentionQueries(torch.zeros(3, 8, 128, dtype=torch.bfloat16), idx, idx)
    for topk in (torch.empty(3, 0, dtype=torch.int32), torch.zeros(3, 5, dtype=torch.int32)[:, :0]):
        A.attend(c, qs, topk=topk)
        A.attend(c, qs, topk=topk, draft=A.Draft(n, torch.zeros(3, 1, dtype=torch.int32), 3))
    assert seen == [(1, [-1, -1, -1])] * 4
