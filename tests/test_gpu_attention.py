"""GPU tests of the attention side against plain implementations in 64 bits.

Tolerances.  A rounding to a type is off by at most half a step: 2^-8 of the
value for bf16, 2^-11 for f16, 2^-24 for fp32, 2^-4 for e4m3 (half a step of
its subnormals, 2^-10, below 2^-6).

Rotary rows: one bf16 rounding, and fp32 arithmetic on cos and sin that are
right to 2 units (2^-23 each) with a rounded product and sum, at most
4 * 2^-23 of |a| + |b|.

Attention: with E = scale * max_t sum_e |q_e k_te| every logit is off by at
most (d + 8) 2^-23 E (a sum of d products in fp32, however it is ordered and
whether it is rounded or truncated, and the factors after it) plus 2^-22 of
the largest |logit| + 1 for the base-2 argument and exponential; call that
delta.  The weights are then off by 2 delta + 2^-20 relatively (numerator and
sum), and by their rounding to bf16 (2^-8) or f16 (2^-11, and 2^-25 of the
largest weight below its normal range) before they meet the values, so with
A = sum_t p_t |v_t| / sum_t p_t
    |out - exact| <= 2^-8 |exact| + (rounding + 2 delta + 2^-20) A
                     [+ 2^-25 max_t(p_t vs_t) sum_t |code_t| / sum_t p_t],
    |lse - exact| <= delta + 2^-20 + 2^-23 |exact|.
"""
import math

import pytest
import torch

from long_context_misa_b200 import attention as A
from long_context_misa_b200 import misa as M

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = 2.0 ** -8


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------- rotary

def rope64(x, pos, r):
    """Exact rotation of x [..., H, d] at pos [...], and |a| + |b| per element."""
    x = x.double()
    i = torch.arange(r.rot // 2, device=DEV)
    ia, ib = ((r.first + i, r.first + r.rot // 2 + i) if r.layout == "half" else (r.first + 2 * i, r.first + 2 * i + 1))
    # whole turns of the table's own 64-bit increments, in exact integers
    turn = torch.tensor([[(int(p) * (int(f) % 2 ** 64)) % 2 ** 64 / 2 ** 64 for f in r.phases.tolist()]
                         for p in pos.reshape(-1).tolist()], dtype=torch.float64, device=DEV)
    t = (2 * math.pi * turn).view(*pos.shape, 1, -1)
    a, b = x[..., ia], x[..., ib]
    y, m = x.clone(), torch.zeros_like(x)
    y[..., ia] = r.amplitude * (a * t.cos() - b * t.sin())
    y[..., ib] = r.amplitude * (b * t.cos() + a * t.sin())
    m[..., ia] = m[..., ib] = abs(r.amplitude) * (a.abs() + b.abs())
    return y, m


def check_rope(out, x, pos, r):
    y, m = rope64(x, pos, r)
    tol = BF16 * y.abs() + 4 * 2.0 ** -23 * m
    assert bool(((out.double() - y).abs() <= tol).all())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot,first", [(128, 64, 0), (128, 64, 64), (128, 128, 0), (64, 32, 8), (128, 48, 16),
                                         (96, 10, 3), (128, 2, 126), (40, 32, 8), (7, 6, 1), (192, 176, 8)])
@pytest.mark.parametrize("n,H", [(1, 1), (37, 5)])
def test_rope_rows(layout, d, rot, first, n, H):
    g = gen(1)
    r = A.Rope(rot, layout=layout, first=first, scaling="yarn", factor=4.0)
    x = randn(g, n, H, d).bfloat16()
    pos = torch.randint(0, 1 << 18, (n,), generator=g, device=DEV).int()
    pos[0] = (1 << 18) - 1
    out = torch.full_like(x, 7.0)
    A.apply_rope(r, [(x, pos, out)])
    check_rope(out, x, pos, r)
    here = x.clone()
    A.apply_rope(r, [(here, pos, here)])
    assert torch.equal(here, out)


def test_rope_groups_strides_and_negative_positions():
    g = gen(2)
    r = A.Rope(64, layout="half", first=32)
    wide = randn(g, 50, 6, 3, 128).bfloat16()         # heads inside a fused projection
    x = wide[:, :, 1]
    odd = randn(g, 9, 3, 130).bfloat16()[:, :, 1:129]  # rows off 16 bytes
    seqs = [(x, torch.arange(-25, 25, device=DEV).int()), (odd, ints([0, 1, -1, 5, 2 ** 31 - 1, -2 ** 31, 3, 4, 262143])),
            (randn(g, 0, 4, 128).bfloat16(), ints([])), (randn(g, 2000, 40, 128).bfloat16(), torch.arange(2000, device=DEV).int())]
    outs = [torch.empty_like(v) for v, _ in seqs]
    A.apply_rope(r, [(v, p, o) for (v, p), o in zip(seqs, outs)])
    for (v, p), o in zip(seqs[:2], outs):
        check_rope(o, v, p, r)
    check_rope(outs[3][::97], seqs[3][0][::97], seqs[3][1][::97], r)
    before = wide.clone()
    A.apply_rope(r, [(x, seqs[0][1], x)])             # in place inside the projection
    check_rope(x, before[:, :, 1], seqs[0][1], r)
    assert torch.equal(wide[:, :, 0], before[:, :, 0]) and torch.equal(wide[:, :, 2], before[:, :, 2])


def test_rope_turns_back():
    """Positions that differ by the same amount give the same products of rows (the point of a rotation)."""
    g = gen(3)
    r = A.Rope(128)
    a, b = randn(g, 1, 1, 128).bfloat16(), randn(g, 1, 1, 128).bfloat16()
    dots = []
    for p in (0, 1000, 262000):
        x = torch.cat([a, b])
        A.apply_rope(r, [(x, ints([p + 13, p]), x)])
        dots.append(float((x[0].double() * x[1].double()).sum()))
    # each rotated element is off by 2^-8 of itself (and fp32 terms far below)
    lim = 2 * 2.1 * BF16 * float(a.double().norm() * b.double().norm())
    assert max(dots) - min(dots) <= lim


# -------------------------------------------------------------------- cache

def plain_codes(x):
    """The cache's quantisation rule on fp32 rows, on the CPU."""
    x = x.float().cpu()
    amax = x.abs().amax(-1)
    sc = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return (x / sc[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV), sc.to(DEV)


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("d,H_kv", [(128, 8), (128, 1), (64, 3)])
@pytest.mark.parametrize("count", [1, 7, 300])
def test_append_plain(e4m3, d, H_kv, count):
    g = gen(4)
    kv = A.KVCache.empty(3, 512, H_kv, d, e4m3)
    for t in (kv.k, kv.v):
        t.fill_(33 if e4m3 else 33.0)
    k, v = (randn(g, 3, count, H_kv, d).bfloat16() for _ in range(2))
    k[0, 0, 0] = 0                                     # a zero row
    pos = ints([5, -1, 512 - count])
    A.append_kv(kv, k, v, pos)
    assert kv.device_status() == 0
    assert kv.seq_len.tolist() == [5 + count, 0, 512]
    for new, rows, sc in ((k, kv.k, kv.k_scale), (v, kv.v, kv.v_scale)):
        want, scale = plain_codes(new) if e4m3 else (new, None)
        for s, p in ((0, 5), (2, 512 - count)):
            assert torch.equal(rows[s, p:p + count], want[s])
            if e4m3:
                assert torch.equal(sc[s, p:p + count], scale[s])
        keep = torch.ones(3, 512, dtype=torch.bool)
        keep[0, 5:5 + count] = keep[2, 512 - count:] = False
        assert bool((rows[keep.to(DEV)] == 33).all())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot,first", [(128, 128, 0), (128, 64, 64), (128, 32, 8), (128, 10, 3), (64, 64, 0), (64, 6, 58)])
@pytest.mark.parametrize("e4m3", [True, False])
def test_append_rotated(layout, d, rot, first, e4m3):
    g = gen(5)
    r = A.Rope(rot, layout=layout, first=first)
    n, count, H_kv = 2, 19, 4
    kv = A.KVCache.empty(n, 262144 if d == 64 else 64, H_kv, d, e4m3)
    fused = randn(g, n, count, 2, H_kv, d).bfloat16()  # keys and values of one projection
    k, v = fused[:, :, 0], fused[:, :, 1]
    pos = ints([3, kv.L_cap - count])
    at = pos[:, None] + torch.arange(count, device=DEV).int()
    for given in (None, (at * 3 - 50).contiguous()):
        A.append_kv(kv, k, v, pos, rope=r, rope_pos=given, commit=given is None)
        y, m = rope64(k, at if given is None else given, r)
        for s in range(n):
            p = int(pos[s])
            rows = kv.k[s, p:p + count]
            exact, mix = y[s], m[s]
            fp32 = 4 * 2.0 ** -23 * mix
            if e4m3:
                sc = kv.k_scale[s, p:p + count].double()
                top = exact.abs().amax(-1)
                # amax carries its element's fp32 error, the quotient one rounding
                assert bool(((sc - top / 448).abs() <= (fp32.amax(-1) + 2.0 ** -23 * top) / 448).all())
                got = rows.view(torch.float8_e4m3fn).double() * sc[..., None]
                step = torch.maximum(2.0 ** -4 * exact.abs(), 2.0 ** -10 * sc[..., None])
                assert bool(((got - exact).abs() <= step * (1 + 2.0 ** -18) + 2 * fp32 + 2.0 ** -22 * top[..., None]).all())
            else:
                assert bool(((rows.double() - exact).abs() <= BF16 * exact.abs() + fp32).all())
            want = plain_codes(v[s])[0] if e4m3 else v[s]
            assert torch.equal(kv.v[s, p:p + count], want)
    assert kv.seq_len.tolist() == [3 + count, kv.L_cap]


@pytest.mark.parametrize("e4m3", [True, False])
def test_append_behind_what_is_there(e4m3):
    """seq_len itself says where the tokens go, captured and replayed too."""
    g, n_seq, count = gen(8), 300, 3
    rope = A.Rope(32, device=DEV)
    start = torch.randint(0, 20, (n_seq,), generator=g, device=DEV).int()
    start[7], start[100] = -1, 38                      # stays; would pass the end
    a, b = (A.KVCache.empty(n_seq, 40, 8, 128, e4m3) for _ in range(2))
    a.seq_len.copy_(start), b.seq_len.copy_(start)
    k, v = (randn(g, n_seq, count, 8, 128).bfloat16() for _ in range(2))
    one = k[:, :1], v[:, :1]
    pos = start.clone()

    def plain(x, y, n):
        A.append_kv(b, x, y, pos.clone(), rope=rope)
        pos.copy_(torch.where((pos < 0) | (pos + n > 40), pos, pos + n))

    A.append_kv(a, k, v, a.seq_len, rope=rope)
    plain(k, v, count)
    assert a.seq_len.tolist() == b.seq_len.tolist() == pos.tolist()
    assert a.device_status() == b.device_status() == M.DEV_APPEND_RANGE
    A.append_kv(a, *one, a.seq_len, rope=rope, rope_pos=a.seq_len)
    plain(*one, 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        A.append_kv(a, k, v, a.seq_len, rope=rope)
    for _ in range(2):
        graph.replay()
        plain(k, v, count)
    assert torch.equal(a.seq_len, b.seq_len)
    for x, y in ((a.k, b.k), (a.v, b.v), (a.k_scale, b.k_scale), (a.v_scale, b.v_scale)):
        assert x is None or torch.equal(x, y)


@pytest.mark.parametrize("d", [64, 128])
def test_append_codes_are_the_rounded_quotients(d):
    """Codes and scales bit for bit: every bf16 significand as a row's largest and as its elements, ties, zeros of
    both signs, tiny and huge rows, and scales next to numbers of few bits."""
    n = 4096
    k, v = (torch.empty(1, n, 2, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    g = gen(9)
    top = (1.0 + torch.arange(128, device=DEV) / 128).repeat(n * 2 // 128).view(1, n, 2)
    for t, e in ((k, torch.randint(-120, 120, (1, n, 2), generator=g, device=DEV)),
                 (v, torch.randint(-6, 7, (1, n, 2), generator=g, device=DEV))):
        x = torch.randint(-128, 129, (1, n, 2, d), generator=g, device=DEV) / 128.0
        x = x * 2.0 ** -torch.randint(0, 22, (1, n, 2, 1), generator=g, device=DEV).float()
        x[..., 0] = 1.0
        x[..., 1], x[..., 2] = 0.0, -0.0
        t.copy_((x.double() * top[..., None].double() * 2.0 ** e[..., None].double()).bfloat16())
    k[:, 5], v[:, 6] = 0.0, -0.0
    kv = A.KVCache.empty(1, n, 2, d, True)
    A.append_kv(kv, k, v, ints([0]))
    # rotated: fp32 rows, by an amplitude that puts their scales within a few ulp of numbers of four bits
    for x, codes, scale in ((k, kv.k, kv.k_scale), (v, kv.v, kv.v_scale)):
        want, ws = plain_codes(x[0])
        assert torch.equal(scale[0], ws.view(n, 2)) and torch.equal(codes[0], want)
    k.copy_(torch.randint(-256, 257, (1, n, 2, d), generator=g, device=DEV) / 256.0 * 448)
    k[..., 0] = 448.0
    for ulps in range(-9, 10):
        amp = float(torch.tensor(1.5) * (1 + ulps * 2.0 ** -23))
        rope = A.Rope(d, amplitude=amp, phases=torch.zeros(d // 2, dtype=torch.int64), device=DEV)
        A.append_kv(kv, k, v, ints([0]), rope=rope)
        x = k[0].float() * torch.tensor(amp, device=DEV)
        want, ws = plain_codes(x)
        assert torch.equal(kv.k_scale[0], ws.view(n, 2)) and torch.equal(kv.k[0], want)


def test_append_past_the_end_and_special_values():
    g = gen(6)
    kv = A.KVCache.empty(3, 16, 2, 64, True)
    k, v = (randn(g, 3, 4, 2, 64).bfloat16() for _ in range(2))
    k[0, 1, 0, 5] = math.nan
    v[0, 2, 1, 7] = math.inf
    A.append_kv(kv, k, v, ints([0, 13, 2 ** 31 - 1]))
    assert kv.device_status() == M.DEV_APPEND_RANGE
    assert kv.seq_len.tolist() == [4, 0, 0]
    assert not bool(kv.k[1:].any()) and not bool(kv.v[1:].any())
    read_k = kv.k.view(torch.float8_e4m3fn).float()[0, :4]
    assert bool(torch.isnan(read_k[1, 0, 5])) and int(torch.isnan(read_k).sum()) == 1
    read_v = kv.v.view(torch.float8_e4m3fn).float()[0, :4] * kv.v_scale[0, :4, :, None]
    assert not bool(torch.isfinite(read_v[2, 1, 7]))
    assert bool(torch.isfinite(read_v[3]).all())


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("d,H_kv", [(128, 8), (64, 1), (64, 5)])
def test_read_back(e4m3, d, H_kv):
    g = gen(7)
    kv = A.KVCache.empty(3, 100, H_kv, d, e4m3)
    k, v = (randn(g, 3, 100, H_kv, d).bfloat16() for _ in range(2))
    A.append_kv(kv, k, v, ints([0, 0, 0]))
    tok = torch.randint(-1, 100, (4, 33), generator=g, device=DEV).int()
    tok[1, 3:6] = 7                                    # the same token three times
    seq = ints([2, 0, 0, 1])
    ko, vo = A.read_kv(kv, seq, tok)
    assert kv.device_status() == 0
    for out, rows, sc in ((ko, kv.k, kv.k_scale), (vo, kv.v, kv.v_scale)):
        x = (rows.view(torch.float8_e4m3fn).float() * sc[..., None]) if e4m3 else rows.float()
        want = x[seq.long()[:, None], tok.long().clamp_min(0)].bfloat16()
        want[tok < 0] = 0
        assert torch.equal(out, want)
    bad = ints([[0, 100, 2 ** 31 - 1], [-2, 5, -1]])
    ko, vo = A.read_kv(kv, ints([0, 3]), bad)
    assert kv.device_status() == M.DEV_BAD_POSITION
    assert torch.equal(ko[0, 0], A.read_kv(kv, ints([0]), ints([[0]]))[0][0, 0])
    assert not bool(ko[0, 1:].any()) and not bool(ko[1].any()) and not bool(vo[0, 1:].any()) and not bool(vo[1].any())
    only = torch.empty(1, 1, H_kv, d, dtype=torch.bfloat16, device=DEV)
    st = torch.cuda.current_stream().cuda_stream
    import ctypes
    assert M._lib.misa_read_kv(ctypes.byref(kv.struct), seq.data_ptr(), ints([[7]]).data_ptr(), 1, 1, None,
                               only.data_ptr(), st) == 0
    assert torch.equal(only, A.read_kv(kv, seq[:1], ints([[7]]))[1])


# ---------------------------------------------------------------- attention

class Case:
    """Random cache, queries, lists and drafted trees; everything nobody sees can be poisoned."""

    def __init__(self, e4m3=True, d=128, H_kv=2, G=4, lens=(300, 77), per=(1, 1), k=0, drafts=0, seed=0, causal=False,
                 spread=1.0, slack=40):
        g = self.g = gen(seed)
        self.e4m3, self.d, self.H_kv, self.G, self.lens, self.drafts = e4m3, d, H_kv, G, lens, drafts
        n_seq, cap = len(lens), max(lens) + drafts + slack
        self.cap = cap
        if e4m3:
            codes = [torch.randint(0, 127, (n_seq, cap, H_kv, d), generator=g, device=DEV) +
                     128 * torch.randint(0, 2, (n_seq, cap, H_kv, d), generator=g, device=DEV) for _ in range(2)]
            self.k, self.v = (c.to(torch.uint8) for c in codes)
            self.ks, self.vs = (torch.exp(spread * randn(g, n_seq, cap, H_kv)) / 200 for _ in range(2))
        else:
            self.k, self.v = (randn(g, n_seq, cap, H_kv, d).bfloat16() for _ in range(2))
            self.ks = self.vs = None
        self.kv = A.KVCache(self.k, self.v, self.ks, self.vs, ints(lens))
        seq = [s for s, n in enumerate(per) for _ in range(n)]
        pos = [lens[s] - 1 - (per[s] - 1 - i if causal else 0) for s in range(n_seq) for i in range(per[s])]
        self.seq, self.pos = seq, [max(p, -1) for p in pos]
        self.n = len(seq)
        self.q = randn(g, self.n, H_kv * G, d).bfloat16()
        self.topk = None
        if k:
            rows = []
            for s, p in zip(seq, self.pos):
                t = torch.randperm(p + 1, generator=g, device=DEV)[:k] if p >= 0 else ints([])
                t = t.int().sort().values
                rows.append(torch.cat([t, torch.full((k - t.numel(),), -1, dtype=torch.int32, device=DEV)]))
            self.topk = torch.stack(rows) if rows else torch.empty(0, k, dtype=torch.int32, device=DEV)
        self.draft = None
        if drafts:
            cg = torch.Generator().manual_seed(seed)
            masks = []
            for s in range(n_seq):
                par = [int(torch.randint(-1, j, (1,), generator=cg)) if j else -1 for j in range(drafts)]
                m = A.tree_mask(par, drafts)
                masks += [m[i % drafts] for i in range(per[s])]
            self.mask = torch.stack(masks).to(DEV) if masks else torch.empty(0, -(-drafts // 32), dtype=torch.int32, device=DEV)
            self.start = ints([x + 3 for x in lens])
            self.draft = A.Draft(self.start, self.mask, drafts)

    def queries(self, scale=None):
        return A.AttentionQueries(self.q, ints(self.seq), ints(self.pos), scale)

    def sees(self, i):
        """Tokens that query i sees (with repetitions)."""
        s, p = self.seq[i], min(self.pos[i], self.lens[self.seq[i]] - 1)
        if self.topk is None:
            t = list(range(p + 1))
        else:
            t = [x for x in self.topk[i].tolist() if 0 <= x <= p]
        if self.draft is not None:
            w = self.mask[i].tolist()
            t += [int(self.start[s]) + j for j in range(self.drafts) if (w[j // 32] >> (j % 32)) & 1]
        return t

    def poison(self):
        """NaN and infinities in every row that no query sees."""
        seen = torch.zeros(len(self.lens), self.cap, dtype=torch.bool, device=DEV)
        for i in range(self.n):
            t = self.sees(i)
            if t:
                seen[self.seq[i], torch.tensor(t, device=DEV)] = True
        self._spoil(~seen)

    def _spoil(self, where):
        for x, s in ((self.k, self.ks), (self.v, self.vs)):
            if self.e4m3:
                x[where] = 0x7F
                s[where] = math.nan
                s.view(-1)[::2] = torch.where(where.reshape(-1)[:, None].expand(-1, self.H_kv).reshape(-1)[::2],
                                              math.inf, s.view(-1)[::2])
            else:
                x[where] = math.inf
                x[..., ::3] = torch.where(where[..., None, None], math.nan, x[..., ::3])

    def rows64(self, i):
        s, t = self.seq[i], torch.tensor(self.sees(i), dtype=torch.long, device=DEV)
        out = []
        for x, sc in ((self.k, self.ks), (self.v, self.vs)):
            if self.e4m3:
                c = x[s][t].view(torch.float8_e4m3fn).double()
                out.append((c, sc[s][t].double()))
            else:
                out.append((x[s][t].double(), torch.ones(t.numel(), self.H_kv, dtype=torch.float64, device=DEV)))
        return out

    def check(self, out, lse, scale=None, only=None):
        scale = self.d ** -0.5 if scale is None else scale
        for i in range(self.n) if only is None else only:
            (kc, ks), (vc, vs) = self.rows64(i)
            q = self.q[i].double().view(self.H_kv, self.G, self.d)
            o, l_ = out[i].double().view(q.shape), lse[i].double().view(q.shape[:2])
            if kc.shape[0] == 0:
                assert bool((o == 0).all()) and bool((l_ == -math.inf).all())
                continue
            k = kc * ks[..., None]
            s = torch.einsum("hgd,thd->hgt", q, k) * scale
            E = (torch.einsum("hgd,thd->hgt", q.abs(), k.abs()) * abs(scale)).amax(-1)
            delta = (self.d + 8) * 2.0 ** -23 * E + 2.0 ** -22 * (s.abs().amax(-1) + 1)
            m = s.amax(-1, keepdim=True)
            p = torch.exp(s - m)
            tot = p.sum(-1)
            exact = torch.einsum("hgt,thd->hgd", p, vc * vs[..., None]) / tot[..., None]
            mass = torch.einsum("hgt,thd->hgd", p, vc.abs() * vs[..., None]) / tot[..., None]
            e_lse = m[..., 0] + torch.log(tot)
            rounding = 2.0 ** -11 if self.e4m3 else BF16
            tol = BF16 * exact.abs() + (rounding + 2 * delta[..., None] + 2.0 ** -20) * mass
            if self.e4m3:
                w = (p * vs.t()[:, None, :]).amax(-1)
                tol = tol + 2.0 ** -25 * (w / tot)[..., None] * vc.abs().sum(0)[:, None, :]
            bad = ~((o - exact).abs() <= tol)
            assert not bool(bad.any()), (i, int(bad.sum()), float((o - exact).abs().max()), float(tol.min()))
            off = (l_ - e_lse).abs()
            assert bool((off <= delta + 2.0 ** -20 + 2.0 ** -23 * e_lse.abs()).all()), (i, float(off.max()))

    def run(self, scale=None, check=True, **kw):
        out, lse = A.attend(self.kv, self.queries(scale), topk=self.topk, draft=self.draft, with_lse=True, **kw)
        if check:
            self.check(out, lse, scale)
        return out, lse


TYPES = [(True, 128), (False, 128), (True, 64), (False, 64)]


@pytest.mark.parametrize("e4m3,d", TYPES)
@pytest.mark.parametrize("H_kv,G", [(1, 1), (2, 4), (3, 7), (1, 16), (1, 24), (2, 40), (1, 128)])
def test_selected(e4m3, d, H_kv, G):
    c = Case(e4m3, d, H_kv, G, lens=(300, 1, 77), per=(2, 1, 3), k=100, causal=True, seed=11)
    c.poison()
    c.run()
    assert c.kv.device_status() == 0


@pytest.mark.parametrize("e4m3,d", TYPES)
@pytest.mark.parametrize("H_kv,G", [(1, 1), (2, 4), (3, 7), (1, 16), (2, 40), (1, 128)])
def test_whole_prefixes(e4m3, d, H_kv, G):
    c = Case(e4m3, d, H_kv, G, lens=(300, 1, 77), per=(9, 1, 3), causal=True, seed=12)
    c.poison()
    c.run()
    assert c.kv.device_status() == 0


@pytest.mark.parametrize("e4m3,d", TYPES)
@pytest.mark.parametrize("drafts", [1, 5, 31, 32, 33, 70])
@pytest.mark.parametrize("k", [0, 50])
def test_drafted_trees(e4m3, d, drafts, k):
    c = Case(e4m3, d, 2, 3, lens=(130, 40, 5), per=(drafts, min(3, drafts), drafts), k=k, drafts=drafts, seed=13)
    c.poison()
    c.run()
    assert c.kv.device_status() == 0


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("k", [1, 2, 15, 16, 17, 31, 33, 255, 256, 257, 2048, 5000])
def test_list_lengths(e4m3, k):
    c = Case(e4m3, 128, 2, 4, lens=(6000, 40), per=(2, 1), k=k, seed=k)
    c.poison()
    c.run()


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 32, 33, 127, 129, 4097, 20001])
def test_prefix_lengths(e4m3, L):
    c = Case(e4m3, 128, 1, 5, lens=(L,), per=(3,), seed=L)
    c.poison()
    c.run()


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("drafts", [0, 24])
def test_many_rows_share_a_prefix(e4m3, drafts):
    """Rows of many queries of one sequence, more than a tile."""
    c = Case(e4m3, 128, 2, 8, lens=(500, 1300), per=(24, 19), drafts=drafts, causal=drafts == 0, seed=21)
    c.poison()
    c.run()


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("k", [0, 20])
def test_rows_that_see_nothing(e4m3, k):
    c = Case(e4m3, 128, 2, 4, lens=(50, 20, 30), per=(2, 2, 2), k=k, drafts=3, seed=31)
    c.pos = [-1, 49, 19, -1, 29, 29]
    c.mask[0] = 0                                      # neither prefix nor drafts
    c.mask[4] = 0
    if k:
        c.topk[4] = -1                                 # a list of nothing
    c.poison()
    out, lse = c.run()
    assert not bool(out[0].any()) and bool((lse[0] == -math.inf).all())
    assert c.kv.device_status() == 0


@pytest.mark.parametrize("e4m3", [True, False])
def test_empty_sequence_and_empty_batch(e4m3):
    c = Case(e4m3, 64, 2, 2, lens=(10, 10), per=(1, 1), seed=32)
    c.kv.seq_len[1] = 0
    c.lens, c.pos = (10, 0), [9, -1]
    c.poison()
    c.run()
    assert c.kv.device_status() == 0
    e = Case(e4m3, 64, 2, 2, lens=(10,), per=(0,), seed=33)
    out, lse = e.run()
    assert out.shape[0] == 0 and lse.shape[0] == 0


@pytest.mark.parametrize("e4m3", [True, False])
def test_calls_on_nothing(e4m3):
    """An empty batch with a list, a draft or both; nothing to read back, nothing to rotate."""
    for k, drafts in ((8, 0), (0, 5), (8, 40)):
        c = Case(e4m3, 64, 2, 2, lens=(10,), per=(0,), k=k, drafts=drafts, seed=33)
        out, lse = c.run()
        assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    ko, vo = A.read_kv(c.kv, ints([]), ints([]).view(0, 7))
    assert ko.shape == vo.shape == (0, 7, 2, 64)
    wide = torch.zeros(5, 3, 128, dtype=torch.bfloat16, device=DEV)
    A.apply_rope(A.Rope(64), [(wide[:0, ::2], ints([]), torch.zeros(0, 2, 128, dtype=torch.bfloat16, device=DEV)),
                              (wide[:, :0], torch.zeros(5, dtype=torch.int32, device=DEV), wide[:, :0])])
    assert c.kv.device_status() == 0


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("G", [3, 40])
def test_lists_without_entries(e4m3, G):
    """A list of nothing shows the drafted tokens alone; without them nothing."""
    c = Case(e4m3, 128, 2, G, lens=(50, 20), per=(2, 2), drafts=3, seed=46)
    c.topk = torch.empty(4, 0, dtype=torch.int32, device=DEV)
    c.poison()
    c.run()
    c.draft = None
    out, lse = c.run()
    assert not bool(out.any()) and bool((lse == -math.inf).all())
    assert c.kv.device_status() == 0


@pytest.mark.parametrize("e4m3", [True, False])
def test_lists_in_any_order_with_repeats_and_strangers(e4m3):
    c = Case(e4m3, 128, 2, 4, lens=(300, 200), per=(1, 2), k=64, seed=34)
    g = c.g
    c.topk = torch.randint(-1, 300, (3, 64), generator=g, device=DEV).int()
    c.topk[0, 5] = c.topk[0, 60] = 17                  # counts twice
    c.topk[1, ::3] = -1
    c.topk[2, 1] = 2 ** 31 - 1
    c.topk[2, 2] = -2 ** 31
    c.pos[2] = 50                                      # tokens 51.. of its list are outside its prefix
    c.poison()
    c.run()
    assert c.kv.device_status() == 0


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("k", [0, 30])
def test_queries_outside_the_cache(e4m3, k):
    c = Case(e4m3, 128, 1, 3, lens=(60, 40), per=(2, 2), k=k, drafts=2, seed=35)
    want, wl = c.run()
    seq, pos = ints([0, 2, -1, 1]), ints([59, 5, 5, -7])
    out, lse = A.attend(c.kv, A.AttentionQueries(c.q, seq, pos), topk=c.topk, draft=c.draft, with_lse=True)
    assert c.kv.device_status() == M.DEV_BAD_POSITION
    # the same query may run in another split or tile: same tokens, other order of sums
    c.check(out, lse, only=[0])
    assert not bool(out[1:].any()) and bool((lse[1:] == -math.inf).all())
    c.kv.status.zero_()
    out, lse = A.attend(c.kv, A.AttentionQueries(c.q, ints(c.seq), ints([59, 60, 39, 39])), topk=c.topk, draft=c.draft,
                        with_lse=True)
    assert c.kv.device_status() == M.DEV_BAD_POSITION  # clamped to the sequence
    if k == 0:
        c.check(out, lse)


def test_drafts_outside_the_cache():
    c = Case(True, 128, 1, 3, lens=(60, 40), per=(3, 3), drafts=3, seed=36, slack=0)
    c.start.copy_(ints([c.cap - 2, -1]))               # slot 2 of sequence 0 and slot 0 of sequence 1 are outside
    for topk in (None, ints([[1, 2, 3, -1]] * 6)):
        c.topk = topk
        c.kv.status.zero_()
        c.mask.copy_(ints([[0b011]] * 3 + [[0b110]] * 3))
        c.run()
        assert c.kv.device_status() == 0
        c.mask[2] = 0b111
        keep = c.mask.clone()
        out, lse = c.run(check=False)
        assert c.kv.device_status() == M.DEV_BAD_POSITION
        c.mask[2] = 0b011                              # what is outside is not seen
        c.check(out, lse)
        c.mask.copy_(keep)


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("G", [2, 12])
def test_interleaved_sequences(e4m3, G):
    """Queries of one sequence not side by side: still right."""
    c = Case(e4m3, 128, 2, G, lens=(100, 64, 33), per=(4, 4, 4), seed=37)
    order = [0, 4, 8, 1, 5, 9, 2, 6, 10, 3, 7, 11]
    c.seq, c.pos = [c.seq[i] for i in order], [c.pos[i] - (i % 3) for i in order]
    c.poison()
    c.run()


@pytest.mark.parametrize("k", [0, 40])
@pytest.mark.parametrize("G", [1, 3, 12, 40])
@pytest.mark.parametrize("e4m3", [True, False])
def test_values_seen_by_some(e4m3, G, k):
    """NaN and infinities in a drafted value or at a causal border reach the queries that see them, no others."""
    c = Case(e4m3, 128, 2, G, lens=(70, 90), per=(6, 6), k=k, drafts=6, seed=38)
    bad = {0: int(c.start[0]) + 2, 1: 85}
    c.pos[6:] = [80, 81, 84, 85, 86, 89]
    if k:
        c.topk[6:, 0] = 85                             # listed by all, in the prefix of three
    for s, t in bad.items():
        if e4m3:
            c.v[s, t, 1, 5] = 0xFF
            c.v[s, t, 0, 64] = 0x7F
        else:
            c.v[s, t, 1, 5] = math.nan
            c.v[s, t, 0, 64] = -math.inf
    out, lse = c.run(check=False)
    hit = [i for i in range(c.n) if bad[c.seq[i]] in c.sees(i)]
    assert 0 < len(hit) < c.n
    o = out.double().view(c.n, 2, G, 128)
    for i in range(c.n):
        where = ~torch.isfinite(o[i])
        if i in hit:
            assert bool(where[1, :, 5].all()) and bool(where[0, :, 64].all()) and int(where.sum()) == 2 * G
        else:
            assert not bool(where.any())
    c.check(out, lse, only=[i for i in range(c.n) if i not in hit])


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("G", [3, 12])
def test_many_values_seen_by_some(e4m3, G):
    """More non-finite values in one chunk than are handled at a time: whole rows of a drafted branch."""
    c = Case(e4m3, 128, 1, G, lens=(70,), per=(5,), drafts=5, seed=45)
    c.mask.copy_(ints([[1], [3], [7], [9], [17]]))
    at = int(c.start[0])
    for j in (1, 2):
        c.v[0, at + j] = 0x7F if e4m3 else math.nan
    out, lse = c.run(check=False)
    assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(out[2]).all())
    c.check(out, lse, only=[0, 3, 4])


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("drafts,bad", [(6, 2), (6, 5), (200, 150), (300, 290)])
def test_bad_values_behind_a_clean_border(e4m3, drafts, bad):
    """Several chunks in a row are searched for non-finite values (a causal border, then drafted tokens): only a later
    one holds any, and many CTAs meet them at different speeds."""
    n = 8
    c = Case(e4m3, 128, 4, 12, lens=(70, 140, 260, 33), per=(n,) * 4, drafts=drafts, seed=47)
    c.pos = [x - 1 - 3 * i for x in c.lens for i in range(n)]
    words = torch.zeros(4 * n, -(-drafts // 32), dtype=torch.int32)
    words[:, 0] = 1                                    # all see slot 0, two of a sequence the spoiled one
    for i in range(4 * n):
        if i % n in (2, 5):
            words[i, bad // 32] |= (1 << (bad % 32)) - (1 << 32 if bad % 32 == 31 else 0)
    c.mask.copy_(words)
    for s in range(4):
        c.v[s, int(c.start[s]) + bad, :, 7] = 0x7F if e4m3 else math.nan
    first = None
    for _ in range(20):
        out, lse = c.run(check=False)
        o = out.view(c.n, 48, 128)
        hit = torch.isnan(o)
        want = torch.zeros_like(hit)
        want[[i for i in range(c.n) if i % n in (2, 5)], :, 7] = True
        assert torch.equal(hit, want)
        first = first if first is not None else (out.clone(), lse.clone())
        assert torch.equal(out.view(torch.int16), first[0].view(torch.int16)) and torch.equal(lse, first[1])
    c.check(out, lse, only=[i for i in range(c.n) if i % n not in (2, 5)])
    assert c.kv.device_status() == 0


@pytest.mark.parametrize("G", [2, 12])
def test_a_nan_key_reaches_its_reader_only(G):
    c = Case(False, 128, 1, G, lens=(70,), per=(3,), drafts=3, seed=39)
    c.mask.copy_(ints([[1], [3], [5]]))
    c.k[0, int(c.start[0]) + 1, 0, 7] = math.nan
    out, lse = c.run(check=False)
    assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(lse[1]).all())
    c.check(out, lse, only=[0, 2])


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("G", [3, 20])
def test_large_and_negative_logits(e4m3, G):
    for scale in (8.0, -0.3, 1e-6, 0.0):
        c = Case(e4m3, 64, 2, G, lens=(400, 90), per=(2, 2), seed=40, spread=0.2)
        c.run(scale=scale)


def test_logits_of_minus_infinity():
    """A visible token whose logit is -inf weighs nothing; alone, it leaves nothing."""
    c = Case(False, 128, 1, 1, lens=(200, 1), per=(1, 1), seed=43)
    for i, t in ((0, 77), (0, 3), (1, 0)):
        e = int(c.q[i, 0].float().abs().argmax())
        c.k[i, t, 0, e] = -math.inf if float(c.q[i, 0, e]) > 0 else math.inf
    out, lse = c.run(check=False)
    assert not bool(out[1].any()) and float(lse[1]) == -math.inf
    keep = [t for t in range(200) if t not in (3, 77)]
    s = (c.k[0, keep, 0].double() @ c.q[0, 0].double()) * 128 ** -0.5
    assert abs(float(lse[0, 0]) - float(torch.logsumexp(s, 0))) < 1e-4
    want = torch.softmax(s, 0) @ c.v[0, keep, 0].double()
    # as in the module's bound, |v| < 6 and the weights' sum 1
    assert float((out[0, 0].double() - want).abs().max()) < 6 * 2 * BF16


@pytest.mark.parametrize("G", [3, 8, 20, 40])
@pytest.mark.parametrize("k", [0, 64])
@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("up", [16, 18, 20, 22, 24, 26, 40, 60, 100])
def test_logits_beyond_their_own_precision(e4m3, G, k, up):
    """Logits so large that half a step of theirs is a power of ten of weight: the largest takes all."""
    c = Case(e4m3, 128, 1, G, lens=(300,), per=(2,), k=k, seed=50)
    for f in (min(up, 60), up - min(up, 60)):
        c.q *= 2.0 ** f
    out, lse = c.run(check=False)
    for i in range(c.n):
        (kc, ks), (vc, vs) = c.rows64(i)
        q = c.q[i].double()
        s = torch.einsum("gd,td->gt", q, kc[:, 0] * ks) * 128 ** -0.5
        E = (torch.einsum("gd,td->gt", q.abs(), kc[:, 0].abs() * ks) * 128 ** -0.5).amax(-1)
        delta = (128 + 8) * 2.0 ** -23 * E + 2.0 ** -22 * (s.abs().amax(-1) + 1)
        two = s.topk(2, dim=-1)
        clear = two.values[:, 0] - two.values[:, 1] > 2 * delta + 200
        assert up < 60 or bool(clear.any())
        assert bool(((lse[i].double() - two.values[:, 0]).abs() <= delta + 6 + 2.0 ** -23 * s.abs().amax(-1)).all())
        assert bool(torch.isfinite(out[i].float()).all())
        v = vc[two.indices[:, 0], 0] * vs[two.indices[:, 0]]
        # one value, its weight and its sum alike but for roundings of the weight, the quotient and the output
        tol = (BF16 + (2.0 ** -11 if e4m3 else BF16) + 2.0 ** -20) * v.abs() + (2.0 ** -25 * 448 if e4m3 else 0.0)
        assert bool(((out[i].double() - v).abs() <= tol)[clear].all())


@pytest.mark.parametrize("G", [3, 20, 40])
@pytest.mark.parametrize("k", [0, 64])
def test_queries_of_any_magnitude(G, k):
    """e4m3 caches meet f16 queries scaled by a power of two: the size of a query does not matter, and a row with an
    infinity leaves the others alone."""
    c = Case(True, 128, 1, G, lens=(150,), per=(2,), k=k, seed=44)
    want, wl = c.run()
    c.q.mul_(2.0 ** 100)
    out, lse = c.run(scale=128 ** -0.5 * 2.0 ** -100, check=False)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    c.q.mul_(2.0 ** -100).mul_(2.0 ** -100)            # (2^-200 is not an fp32 number)
    out, lse = c.run(scale=128 ** -0.5 * 2.0 ** 100, check=False)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    c.q.mul_(2.0 ** 100)
    c.q[1, 1, 3] = math.inf
    out, lse = c.run(check=False)
    c.check(out, lse, only=[0])
    assert torch.equal(out[1, 2], want[1, 2]) and not bool(torch.isfinite(out[1, 1].float()).all())


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("G", [3, 8, 12, 20, 40])
@pytest.mark.parametrize("k", [0, 64])
def test_rows_of_very_different_magnitude(e4m3, G, k):
    """Heads and queries side by side whose q differ by more than f16's range, and rows that see nothing whatever they
    hold: no row costs another any bits."""
    c = Case(e4m3, 128, 2, G, lens=(150, 90), per=(4, 3), k=k, seed=48)
    c.q[0] *= 2.0 ** -60
    c.q[0] *= 2.0 ** -40                               # a query at 2^-100
    c.q[1, 1::3] *= 2.0 ** 12                          # heads of one query, 2^32 apart
    c.q[1, 2::3] *= 2.0 ** -20
    c.q[2] = 0
    c.q[4] *= 2.0 ** 60
    c.q[4] *= 2.0 ** 40                                # one at 2^100
    c.pos[5] = -1                                      # padding: sees nothing
    c.q[5] = 3e38
    if k:
        c.topk[5] = -1
    out, lse = c.run()
    assert not bool(out[5].any()) and bool((lse[5] == -math.inf).all())
    assert c.kv.device_status() == 0


@pytest.mark.parametrize("G", [4, 24])
def test_scales_of_very_different_size(G):
    """e4m3 rows whose scales span many orders, zero among them."""
    c = Case(True, 128, 2, G, lens=(500, 90), per=(2, 2), k=80, seed=41, spread=6.0)
    c.ks.clamp_(max=0.02)
    c.vs[:, ::7] = 0.0
    c.run()
    c.topk = None
    c.run()


@pytest.mark.parametrize("G", [2, 12, 24, 40])
def test_values_of_scale_zero_come_first(G):
    """Rows of scale 0 weigh in the sum although they add nothing: alone, before any other token, and with logits far
    above every other's."""
    c = Case(True, 128, 1, G, lens=(700,), per=(2,), k=256, seed=45)
    c.vs[:, :400] = 0.0
    full = c.topk.clone()
    for n in (1, 100, 256):                            # listed tokens, nothing listed before them
        c.topk = torch.full_like(full, -1)
        c.topk[:, 256 - n:] = full[:, :n]              # (sorted: those of scale 0 first)
        c.run()
    c.topk = None
    c.run()
    for p in (0, 300, 450):
        c.pos = [-1, p]
        c.run()
    # logits of up to +-450 (base 2); the others' weights are below 2^-200 of the sum, and come out below 2^-90
    c.pos = [699, 699]
    big = 300.0 / float((c.q[0].float().abs().amax() * 30))
    c.k[0, 350] = torch.where(c.q[0, 0] >= 0, 0x7E, 0xFE).to(torch.uint8)
    c.k[0, 450] = 0
    c.ks[0, 350] = big
    c.q[:] = c.q[:1, :1].abs() * torch.sign(c.q[:1, :1])
    for t in (None, ints([[450, 350], [350, 450]])):
        c.topk = t
        out, lse = c.run(check=False)
        (kc, ks), _ = c.rows64(0)
        s = torch.einsum("d,td->t", c.q[0, 0].double(), kc[:, 0] * ks) * 128 ** -0.5
        assert float(s.amax()) > 200 + float(s[s < s.amax()].amax())
        assert bool((out.float().abs() <= 2.0 ** -90).all())
        assert bool(((lse.double() - s.amax()).abs() <= 2.0 ** -14 * s.amax()).all())


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("H_kv,G,per,listed", [(8, 4, 80, True), (1, 40, 148, True), (1, 16, 1184, False)])
@pytest.mark.parametrize("at", [0, 100])
def test_many_small_weights_beside_a_large_one(e4m3, H_kv, G, per, listed, at):
    """One token of value 0 holds nearly all of the weight and 128K tokens 17.4 nats below it the rest, all of value 1:
    the result is their share of the sum."""
    L = 1 << 17
    c = Case(e4m3, 64, H_kv, G, lens=(L,), per=(per,), seed=49, slack=0)
    one = 0x38 if e4m3 else 1.0                        # 1 in e4m3
    c.k.zero_()
    c.v.fill_(one)
    c.k[0, at, :, 0] = one
    c.v[0, at] = 0
    if e4m3:
        c.ks.fill_(1.0)
        c.vs.fill_(1.0)
    c.q.zero_()
    c.q[:, :, 0] = 17.375
    if listed:
        c.topk = torch.arange(L, device=DEV).int().expand(per, L).contiguous()
    out, lse = c.run(scale=1.0, check=False)
    # the output's half step; weights that lose at most 2^-11 (f16) or 2^-8 (bf16) of themselves, in f16 up to 2^-32 of
    # the largest (2^-25 of 2^7); sums in L / 16 products of 16 tokens, each off by 2^-23 of what is there
    share = (L - 1) * math.exp(-17.375)
    exact = share / (1 + share)
    tol = exact * (BF16 + (2.0 ** -11 if e4m3 else BF16) + L / 16 * 2.0 ** -23) + (L * 2.0 ** -32 if e4m3 else 0.0)
    assert tol < exact / 32
    assert bool(((out.double() - exact).abs() <= tol).all()), (exact, float(out.min()), float(out.max()))
    assert bool(((lse.double() - 17.375 - math.log1p(share)).abs() <= 2.0 ** -10).all())


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("G,per", [(1, (37, 1, 1, 1)), (8, (60, 1, 0, 2))])
def test_uneven_batches(e4m3, G, per):
    """More tiles than an even spread of the queries has."""
    c = Case(e4m3, 128, 2, G, lens=(300, 64, 33, 100), per=per, seed=46, causal=True)
    c.poison()
    c.run()


@pytest.mark.parametrize("e4m3", [True, False])
def test_more_queries_than_one_scan(e4m3):
    """Runs of queries beyond the first 1024 of a batch, one cut there."""
    c = Case(e4m3, 64, 1, 2, lens=(20,) * 600, per=(2,) * 600, seed=47, slack=0)
    out, lse = c.run(check=False)
    c.check(out, lse, only=list(range(0, 40)) + list(range(1000, 1060)) + list(range(1180, 1200)))
    c = Case(e4m3, 64, 1, 4, lens=(700, 900), per=(500, 800), seed=48, causal=True, slack=0)
    out, lse = c.run(check=False)
    c.check(out, lse, only=list(range(0, 1300, 37)) + list(range(1015, 1035)) + [1299])
    assert c.kv.device_status() == 0


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("G", [1, 8])
@pytest.mark.parametrize("k", [0, 30])
def test_large_drafts(e4m3, G, k):
    c = Case(e4m3, 64, 1, G, lens=(90, 40), per=(7, 2), k=k, drafts=1024, seed=49)
    g = torch.Generator().manual_seed(1)
    c.mask.copy_(torch.randint(-2 ** 31, 2 ** 31, c.mask.shape, generator=g).to(torch.int32))
    c.poison()
    c.run()
    assert c.kv.device_status() == 0


@pytest.mark.parametrize("e4m3,d", TYPES)
def test_long_prefixes_of_many_rows(e4m3, d):
    """Shares of a long prefix, joined through the workspace."""
    c = Case(e4m3, d, 1, 6, lens=(9000, 5000), per=(5, 4), drafts=5, seed=55)
    c.poison()
    c.run()


def test_far_offsets():
    """A cache beyond 2^32 bytes and 2^31 elements: rows of its far end."""
    L, H_kv, d = 1 << 18, 80, 128
    kv = A.KVCache.empty(2, L, H_kv, d, True)
    assert kv.k.numel() > 1 << 32
    g = gen(42)
    k, v = (randn(g, 2, 50, H_kv, d).bfloat16() for _ in range(2))
    pos = ints([L - 50, L - 50])
    A.append_kv(kv, k, v, pos)
    assert kv.device_status() == 0 and kv.seq_len.tolist() == [L, L]
    ko, vo = A.read_kv(kv, ints([1]), ints([[L - 1, L - 50]]))
    want, sc = plain_codes(k[1])
    deq = (want.view(torch.float8_e4m3fn).float() * sc[..., None]).bfloat16()
    assert torch.equal(ko[0], deq[[49, 0]])
    c = Case.__new__(Case)
    c.e4m3, c.d, c.H_kv, c.G, c.lens, c.draft, c.cap = True, d, H_kv, 1, (L, L), None, L
    c.k, c.v, c.ks, c.vs, c.kv = kv.k, kv.v, kv.k_scale, kv.v_scale, kv
    c.seq, c.pos, c.n = [1, 0], [L - 1, L - 3], 2
    c.q = randn(g, 2, H_kv, d).bfloat16()
    c.topk = torch.arange(L - 60, L, device=DEV).int().repeat(2, 1)
    c.run()


def test_streams_and_graphs():
    c = Case(True, 128, 2, 4, lens=(5000, 777), per=(2, 1), k=300, drafts=2, seed=50)
    ws = M.Workspace(DEV)
    qs = c.queries()
    want, wl = c.run(ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = A.attend(c.kv, qs, topk=c.topk, draft=c.draft, with_lse=True, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)
    # two graphs that share a workspace, replayed in turn on new inputs
    p = Case(True, 128, 2, 4, lens=(5000, 777), per=(2, 1), seed=51)
    pq, pw = p.queries(), p.run(ws=ws)
    graphs = []
    for case, q in ((c, qs), (p, pq)):
        o, l_ = torch.empty_like(q.q), torch.empty(q.n_q, q.H, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            A.attend(case.kv, q, topk=case.topk, draft=case.draft, out=o, lse=l_, ws=ws)
        graphs.append((g, o, l_))
    ws.get(ws.buf.numel() * 4)                         # outgrown: the graphs' addresses stay good
    for _ in range(3):
        for g, o, l_ in graphs:
            o.zero_(), l_.zero_()
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], want) and torch.equal(graphs[0][2], wl)
    assert torch.equal(graphs[1][1], pw[0]) and torch.equal(graphs[1][2], pw[1])
    c.q.copy_(c.q.flip(0))
    graphs[0][0].replay()
    torch.cuda.synchronize()
    c.check(graphs[0][1], graphs[0][2])


def test_workspaces_keep_what_others_may_still_use():
    """Outgrown buffers stay for graphs and other streams, together below twice the one in use; else they are dropped."""
    ws = M.Workspace(DEV)
    for n in range(1 << 20, 1 << 24, 1 << 18):
        assert ws.get(n).numel() == n
    assert ws.outgrown == []
    side = torch.cuda.Stream()
    held = []
    for n in range(1 << 24, 1 << 27, 1 << 20):
        way = (n >> 20) % 3
        if way == 0:
            held.append(ws.get(n, stream=side).data_ptr())
        elif way == 1:
            with torch.cuda.stream(side):
                ws.get(n)                              # (its own where it grows here: torch's allocator sees to that)
        else:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                buf = ws.get(n)
                buf[:1].zero_()
            held.append(buf.data_ptr())
    have = {b.data_ptr() for b in ws.outgrown} | {ws.buf.data_ptr()}
    assert set(held) <= have and len(ws.outgrown) < 12
    assert sum(b.numel() for b in ws.outgrown) <= 2 * ws.buf.numel()


def test_a_call_on_another_stream_keeps_its_own_workspace(monkeypatch):
    """Scratch that a call allocates for itself is not handed out again while the call waits on its stream."""
    from long_context_misa_b200 import inputs as G
    inp = G.make_inputs(G.WORKLOADS["tiny_decode"], 0)
    cache, qs = M.device_inputs(inp)
    M.pool_keys(cache)
    heads = M.route_heads(cache, qs, 8)
    want = M.score_topk(cache, qs, heads, 256)
    had = []
    get = M.Workspace.get

    def noted(self, nbytes, stream=None):
        buf = get(self, nbytes, stream)
        had.append((buf.data_ptr(), buf.numel()))
        return buf
    monkeypatch.setattr(M.Workspace, "get", noted)
    side = torch.cuda.Stream()
    top = torch.empty_like(want)
    torch.cuda.synchronize()
    for given in (side, side.cuda_stream):
        had.clear()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)              # about 10 ms in which the call cannot start
        M.score_topk(cache, qs, heads, 256, topk=top, stream=given)
        for at, size in had:
            x = torch.empty(size, dtype=torch.uint8, device=DEV)
            assert x.data_ptr() != at
            x.fill_(255)
        side.synchronize()
        assert had and torch.equal(top, want)


def test_same_call_same_bits():
    c = Case(False, 128, 4, 4, lens=(30000, 777), per=(3, 2), seed=52)
    a = c.run()
    for _ in range(3):
        b = c.run(check=False)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_outputs_of_other_rows_stay():
    c = Case(True, 128, 2, 4, lens=(300,), per=(2,), k=50, seed=53)
    big = torch.full((6, 8, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((6, 8), 3.0, device=DEV)
    out, l_ = c.run(out=big[2:4], lse=lse[2:4])
    assert bool((big[:2] == 3).all()) and bool((big[4:] == 3).all()) and bool((lse[:2] == 3).all()) and bool((lse[4:] == 3).all())


def test_bits_and_bf16_tensors_are_the_same():
    c = Case(False, 128, 2, 2, lens=(100,), per=(2,), seed=54)
    want, wl = c.run()
    kv = A.KVCache(c.k.view(torch.int16), c.v.view(torch.int16), None, None, ints(c.lens))
    out, lse = A.attend(kv, A.AttentionQueries(c.q.view(torch.int16), ints(c.seq), ints(c.pos)), with_lse=True)
    assert out.dtype == torch.int16 and torch.equal(out.view(torch.bfloat16), want) and torch.equal(lse, wl)


def test_a_run_of_them_together():
    """A prompt written, a decode step with selection, a drafted tree verified, its accepted path committed."""
    g = gen(60)
    n_seq, L0, H_kv, G, d, k = 2, 400, 2, 4, 128, 64
    r = A.Rope(64, base=500000.0, layout="interleaved", scaling="yarn", factor=8.0)
    kv = A.KVCache.empty(n_seq, 512, H_kv, d, True)
    c = Case.__new__(Case)
    c.e4m3, c.d, c.H_kv, c.G, c.cap, c.kv = True, d, H_kv, G, 512, kv
    c.k, c.v, c.ks, c.vs, c.draft, c.topk = kv.k, kv.v, kv.k_scale, kv.v_scale, None, None
    # prompt
    new = [randn(g, n_seq, L0, H_kv, d).bfloat16() for _ in range(2)]
    A.append_kv(kv, *new, ints([0, 0]), rope=r)
    # one decode step: index keys and queries rotated, appended, selected by the dense indexer, attended
    keys = torch.zeros(n_seq, 512, 128, dtype=torch.int16, device=DEV)
    cache = M.KeyCache(keys, None, ints([L0, L0]), 64)
    ik = randn(g, n_seq * L0, 1, 128).bfloat16()
    pos_all = torch.arange(L0, device=DEV).int().repeat(n_seq)
    A.apply_rope(r, [(ik, pos_all, ik)])
    keys[:, :L0] = ik.view(torch.int16).view(n_seq, L0, 128)
    M.pool_keys(cache)
    iq, q = randn(g, n_seq, 16, 128).bfloat16(), randn(g, n_seq, H_kv * G, d).bfloat16()
    pos = ints([L0, L0])
    nk = randn(g, n_seq, 1, 128).bfloat16()
    A.apply_rope(r, [(iq, pos, iq), (nk, pos, nk), (q, pos, q)])
    M.pool_keys(cache, nk.view(torch.int16), None, pos)
    A.append_kv(kv, randn(g, n_seq, 1, H_kv, d).bfloat16(), randn(g, n_seq, 1, H_kv, d).bfloat16(), pos, rope=r)
    seq = ints([0, 1])
    qs = M.Queries(iq.view(torch.int16), randn(g, n_seq, 16), seq, pos)
    c.topk = M.dense_score_topk(cache, qs, k)
    c.seq, c.pos, c.n, c.lens, c.q = [0, 1], [L0, L0], 2, (L0 + 1, L0 + 1), q
    c.run()
    assert kv.device_status() == 0 and cache.device_status() == 0
    # five drafted tokens in a tree, at the positions of their depths
    parents, T = [-1, 0, 0, 1, 2], 5
    depth = ints([[0, 1, 1, 2, 2]] * n_seq) + L0 + 1
    dk, dv = (randn(g, n_seq, T, H_kv, d).bfloat16() for _ in range(2))
    start = ints([L0 + 1, L0 + 1])
    A.append_kv(kv, dk, dv, start, rope=r, rope_pos=depth, commit=False)
    assert kv.seq_len.tolist() == [L0 + 1] * 2
    c.q = randn(g, n_seq * T, H_kv * G, d).bfloat16()
    A.apply_rope(r, [(c.q, depth.view(-1), c.q)])
    c.seq, c.pos, c.n = [0] * T + [1] * T, [L0] * (2 * T), 2 * T
    c.mask, c.start, c.drafts = A.tree_mask(parents).repeat(n_seq, 1).to(DEV), start, T
    c.draft = A.Draft(start, c.mask, T)
    c.topk = c.topk.repeat_interleave(T, 0).contiguous()
    tree_out, _ = c.run()
    # accept nodes 0, 2, 4 of sequence 0, node 0 of sequence 1: written again at their places
    for s, path in ((0, [0, 2, 4]), (1, [0])):
        at = ints([L0 + 1 if x == s else -1 for x in range(n_seq)])
        A.append_kv(kv, dk[:, path], dv[:, path], at, rope=r)
    assert kv.seq_len.tolist() == [L0 + 4, L0 + 2]
    # the accepted node's query, over the committed prefix: what the tree gave it
    c.draft, c.topk = None, torch.cat([c.topk[[4, 5]], ints([[L0 + 1, L0 + 2, L0 + 3], [L0 + 1, -1, -1]])], dim=1)
    c.lens, c.n, c.seq, c.pos, c.q = (L0 + 4, L0 + 2), 2, [0, 1], [L0 + 3, L0 + 1], c.q[[4, 5]].contiguous()
    out, _ = c.run()
    # the same tokens and bits in another order of sums: within both calls' bounds of one exact value
    assert float((out.double() - tree_out[[4, 5]].double()).abs().max()) <= 4 * BF16 * float(out.abs().max())
    assert kv.device_status() == 0


def test_decode_step_with_its_attention():
    """MisaDaggerDecode with the attention in it: the separate calls' results, run, captured and replayed; the
    selection is what the step without it selects."""
    from long_context_misa_b200 import inputs as G
    wl = G.WORKLOADS["tiny_decode"].scaled(k_prime=1024)
    inp = G.make_inputs(wl, 0)
    cache, qs = M.device_inputs(inp)
    n, L, H_kv, H, d = wl.n_seq, cache.L_cap, 4, 16, 128
    g = gen(70)
    pos = ints((inp.seq_len - 1).tolist())
    cache.seq_len.copy_(pos)
    M.pool_keys(cache)
    last = torch.stack([cache.keys[s, int(pos[s]):int(pos[s]) + 1] for s in range(n)]).clone()
    plain = M.MisaDaggerDecode(cache, qs, wl.h, wl.k_prime, wl.k, last, None, pos)
    plain.run()
    # the step's raw rows, unrotated, as projections give them
    r = A.Rope(64, layout="interleaved", base=500000.0)
    raw_iq = qs.q.clone().view(torch.bfloat16)
    raw_q = randn(g, qs.n_q, H, d).bfloat16()
    q = torch.empty_like(raw_q)
    kv = A.KVCache.empty(n, L, H_kv, d, True)
    hist = [randn(g, n, L - 1, H_kv, d).bfloat16() for _ in range(2)]
    A.append_kv(kv, *hist, ints([0] * n), rope=r)
    kv.seq_len.copy_(pos)
    new = [randn(g, n, 1, H_kv, d).bfloat16() for _ in range(2)]
    aq = A.AttentionQueries(q, qs.q_seq, qs.q_pos)

    def sparse(rotate):
        return A.SparseAttention(kv, aq, *new, pos, wl.k, rope=r, rotate=rotate, kv_rope=r)
    # attention queries rotated only: the selection does not change
    step = M.MisaDaggerDecode(cache, qs, wl.h, wl.k_prime, wl.k, last, None, pos, attention=sparse([(raw_q, qs.q_pos, q)]))
    step.run()
    assert torch.equal(step.topk, plain.topk)
    want = A.attend(kv, aq, topk=plain.topk, with_lse=True)
    assert torch.equal(step.attention.out, want[0]) and torch.equal(step.attention.lse, want[1])
    # index queries rotated as well, the step captured and replayed on new rows
    step = M.MisaDaggerDecode(cache, qs, wl.h, wl.k_prime, wl.k, last, None, pos,
                              attention=sparse([(raw_iq, qs.q_pos, qs.q.view(torch.bfloat16)), (raw_q, qs.q_pos, q)]))
    step.run()
    step.capture()
    for i in range(2):
        raw_iq.copy_(randn(g, *raw_iq.shape)), raw_q.copy_(randn(g, *raw_q.shape)), new[0].copy_(randn(g, *new[0].shape))
        step.replay()
        torch.cuda.synchronize()
        c = Case.__new__(Case)
        c.e4m3, c.d, c.H_kv, c.G, c.lens, c.draft, c.cap = True, d, H_kv, H // H_kv, tuple(inp.seq_len.tolist()), None, L
        c.k, c.v, c.ks, c.vs, c.kv = kv.k, kv.v, kv.k_scale, kv.v_scale, kv
        c.seq, c.pos, c.n, c.q, c.topk = qs.q_seq.tolist(), qs.q_pos.tolist(), qs.n_q, q, step.topk
        check_rope(q, raw_q, qs.q_pos, r)
        check_rope(qs.q.view(torch.bfloat16), raw_iq, qs.q_pos, r)
        assert torch.equal(step.topk, M.dagger_topk(cache, qs, step.heads, wl.k_prime, wl.k))
        c.check(step.attention.out, step.attention.lse)
    assert kv.device_status() == 0 and cache.device_status() == 0
    with pytest.raises(ValueError):
        A.SparseAttention(kv, aq, *new, pos, wl.k, rotate=[(raw_q, qs.q_pos, q)])


def test_decode_step_over_e4m3_index_keys():
    """The step of an e4m3 index cache: its new keys rotated and written before it in one graph, its own append left out
    by positions of -1."""
    from long_context_misa_b200 import inputs as G
    wl = G.WORKLOADS["misa_dagger_decode_128k"].scaled(n_seq=2, L=8192, k=256, k_prime=1024, needles_per_seq=2)
    inp = G.make_inputs(wl, 0)
    cache, qs = M.device_inputs(inp)
    n, H_kv, H, d = wl.n_seq, 2, 16, 128
    g, pos, none = gen(71), ints((inp.seq_len - 1).tolist()), ints([-1] * wl.n_seq)
    cache.seq_len.copy_(pos)
    M.pool_keys(cache)
    r = A.Rope(64, base=500000.0)
    raw_iq, raw_ik = qs.q.clone().view(torch.bfloat16), randn(g, n, 1, 128).bfloat16()
    ik, raw_q = torch.empty_like(raw_ik), randn(g, n, H, d).bfloat16()
    q = torch.empty_like(raw_q)
    kv = A.KVCache.empty(n, cache.L_cap, H_kv, d, True)
    A.append_kv(kv, *(randn(g, n, cache.L_cap - 1, H_kv, d).bfloat16() for _ in range(2)), ints([0] * n), rope=r)
    new = [randn(g, n, 1, H_kv, d).bfloat16() for _ in range(2)]
    aq = A.AttentionQueries(q, qs.q_seq, qs.q_pos)
    unused = torch.zeros(n, 1, 128, dtype=torch.uint8, device=DEV), torch.ones(n, 1, device=DEV)
    step = M.MisaDaggerDecode(cache, qs, wl.h, wl.k_prime, wl.k, *unused, none,
                              attention=A.SparseAttention(kv, aq, *new, pos, wl.k, kv_rope=r))

    def whole():
        A.apply_rope(r, [(raw_iq, qs.q_pos, qs.q.view(torch.bfloat16)), (raw_ik, pos, ik), (raw_q, qs.q_pos, q)])
        M.append_keys_e4m3(cache, ik.view(torch.int16), pos)
        step.run()
    whole()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        whole()
    for _ in range(2):
        raw_iq.copy_(randn(g, *raw_iq.shape)), raw_ik.copy_(randn(g, *raw_ik.shape)), raw_q.copy_(randn(g, *raw_q.shape))
        graph.replay()
        torch.cuda.synchronize()
        check_rope(ik, raw_ik, pos, r)
        for s in range(n):
            codes, scale = plain_codes(ik[s])
            assert torch.equal(cache.keys[s, int(pos[s])], codes[0]) and torch.equal(cache.scale[s, int(pos[s])], scale[0])
        assert cache.seq_len.tolist() == kv.seq_len.tolist() == inp.seq_len.tolist()
        pool = cache.pool.clone()
        M.pool_keys(cache)                             # the same means of 128 keys, summed in other groups
        top = (cache.keys.view(torch.float8_e4m3fn).float() * cache.scale[..., None]).abs().max()
        assert bool(((pool - cache.pool).abs() <= 2 * 128 * 2.0 ** -24 * top).all())
        assert torch.equal(step.topk, M.dagger_topk(cache, qs, step.heads, wl.k_prime, wl.k))
        want = A.attend(kv, aq, topk=step.topk, with_lse=True)
        assert torch.equal(step.attention.out, want[0]) and torch.equal(step.attention.lse, want[1])
    assert kv.device_status() == 0 and cache.device_status() == 0
