"""Token cache on the GPU against plain float64 implementations.

Tolerances.  e = finfo(type).eps / 2 is one rounding to the rows' type, u = 2^-24 one
rounding to fp32.
  scores   x = scale * q . k in fp32: |dx| <= (d + 2) u * reach + 3 u |x| with reach = scale * sum |q k|, and for the
           exponential's argument (two products with log2 e, one subtraction, ex2 within 2 ulp) another 4 u |x|.
           With |x| <= reach: dx <= (d + 9) u * reach.
  attend   a weight is off by the factor exp(dx) exp(-dx') e^(...) <= 1 + 2 dx + few u, and rounded once to the type
           (relative e, or below the smallest normal number 2^-25 absolute, for fp16, relative to the row's largest weight); the
           result is rounded once more: |do| <= e |o| + (e + 4 dx + 64 u) S + 2^-24 sum|v| (fp16) with S = sum w |v|.
           The products' fp32 sums over L keys add at most L u S (and as much for the weights' sum).
  lse      |dl| <= 2 dx + L u + 8 u (1 + |l|)
  weigh    a key's sum of N terms: relative 2 dx + 4 u |lse| + (N + 8) u
  append   angle within 2^-25 half turns (pi 2^-25 radians) and sincospi within 2 ulp: |dy| <= e |y| + (2^-23 + 4 u) (|a| + |b|)
"""
import math

import numpy as np
import pytest
import torch

from oracle import cache_oracle as CO

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float16]
LAYOUTS = [(16, 8, 128), (20, 20, 64), (14, 2, 64), (8, 1, 128), (3, 1, 64), (40, 1, 128), (2, 2, 128)]


@pytest.fixture(scope="module")
def lm():
    import log_mel_spectrogram_logmel_b200 as lm
    return lm


class Box:
    """A cache of random rows, with NaN wherever no live slot is, and new rows for its streams."""

    def __init__(self, lm, hq, hkv, d, page, dtype, new, lens, seed=0, sharp=2.0, order="page", **plan):
        self.hq, self.hkv, self.d, self.page, self.dtype, self.new, self.lens_host = hq, hkv, d, page, dtype, new, lens
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.plan = lm.CachePlan(hq, hkv, d, page, dtype=dtype, **plan)
        need = [max(0, -(-x // page)) for x in lens]
        pages = sum(need) + 3
        perm = torch.randperm(pages, device="cuda", generator=g).tolist()
        width = max(need + [1]) + 1
        table = torch.full((len(lens), width), 123456789, dtype=torch.int32)     # past the last live page: never read
        live = torch.zeros(pages, page, dtype=torch.bool)
        at = 0
        for s, n in enumerate(need):
            table[s, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
            for j in range(n):
                live[perm[at + j], :max(0, lens[s] - j * page)] = True
            at += n
        self.table, self.live = table.cuda(), live.cuda()[:, None, :, None]
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")

        def pool():
            if order == "page":          # [page, head, slot, d]
                x = torch.randn(pages, hkv, page, d, device="cuda", generator=g)
                return torch.where(self.live, x, torch.nan).to(dtype)
            x = torch.randn(pages, page, 2, hkv, d, device="cuda", generator=g).to(dtype)[:, :, 1].transpose(1, 2)
            x.copy_(torch.where(self.live, x.float(), torch.nan))
            return x
        self.k, self.v = pool(), pool()
        self.mass = torch.rand(pages, hkv, page, device="cuda", generator=g)
        self.cache = lm.TokenCache(self.plan, self.k, self.v, self.table, self.lens, mass=self.mass)
        self.offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        self.rows = int(self.offsets[-1])
        self.qkv = torch.randn(self.rows, hq + 2 * hkv, d, device="cuda", generator=g).to(dtype)
        self.q = (self.qkv[:, :hq].float() * sharp).to(dtype)
        self.scale = d ** -0.5

    def gathered(self, pool, s):
        """Slots 0 .. len - 1 of stream s, [heads, len, d] in float64 (repeated for every query head by the caller)."""
        j = torch.arange(max(0, self.lens_host[s]), device="cuda")
        return pool[self.table[s].long()[j // self.page], :, j % self.page].double().transpose(0, 1)

    def mask(self, s, causal, window):
        n, length = self.new[s], self.lens_host[s]
        p = length - n + torch.arange(n, device="cuda")[:, None]
        j = torch.arange(max(0, length), device="cuda")
        m = (j <= p) if causal else (j >= 0).expand(n, -1)
        return m & (j > p - window) if window > 0 else m

    def attend_ref(self, causal=True, window=0, q=None):
        q = self.q if q is None else q
        out = torch.zeros(self.rows, self.hq, self.d, dtype=torch.float64, device="cuda")
        tol, lse = torch.zeros_like(out), torch.full((self.rows, self.hq), -math.inf, dtype=torch.float64, device="cuda")
        ltol = torch.zeros_like(lse)
        e = torch.finfo(self.dtype).eps / 2
        g = self.hq // self.hkv
        for s, n in enumerate(self.new):
            if not n or self.lens_host[s] <= 0:
                continue
            k, v = (self.gathered(x, s).repeat_interleave(g, 0) for x in (self.k, self.v))
            rows = slice(int(self.offsets[s]), int(self.offsets[s + 1]))
            x = q[rows].double().transpose(0, 1)
            reach = (x.abs() @ k.abs().transpose(1, 2) * self.scale)
            z = x @ k.transpose(1, 2) * self.scale
            m = self.mask(s, causal, window)
            z = z.masked_fill(~m, -math.inf)
            reach = reach.masked_fill(~m, 0).amax(-1, keepdim=True)
            l = torch.logsumexp(z, -1, keepdim=True)
            some = m.any(-1)[None, :, None]
            w = torch.where(some, torch.exp(z - l), 0.0)
            w = torch.nan_to_num(w, nan=0.0)
            o = w @ v
            dx = (self.d + 9) * U * reach
            spread = w @ v.abs()
            t = e * o.abs() + (e + 4 * dx + (64 + 2 * self.lens_host[s]) * U) * spread
            if self.dtype == torch.float16:
                t = t + U * (m.double() @ v.abs()) + 2.0 ** -25
            out[rows], tol[rows] = o.transpose(0, 1), t.transpose(0, 1)
            lse[rows] = torch.where(some, l, -math.inf)[..., 0].t()
            ltol[rows] = (2 * dx + self.lens_host[s] * U + 8 * U * (1 + torch.where(some, l, 0.0).abs()))[..., 0].t()
        return out, tol, lse, ltol

    def check_attend(self, causal=True, window=0, **kw):
        out, lse = self.cache.attend(self.q, self.offsets, causal=causal, window=window, return_lse=True, **kw)
        want, tol, wl, ltol = self.attend_ref(causal, window)
        bad = (out.double() - want).abs() > tol
        assert not bool((bad | out.isnan()).any()), (int(bad.sum()), float((out.double() - want).abs().max()),
                                                     bad.nonzero()[:4].tolist())
        empty = wl == -math.inf
        assert torch.equal(lse == -math.inf, empty)
        assert bool(((lse.double() - wl).abs() <= ltol)[~empty].all()), float((lse.double() - wl).abs()[~empty].max())
        assert torch.equal(out[empty], torch.zeros_like(out[empty]))
        return out, lse

    def weigh_ref(self, lse, causal=True, window=0, decay=1.0):
        out = self.mass.double()
        tol = torch.zeros_like(out)
        g = self.hq // self.hkv
        for s, n in enumerate(self.new):
            length = self.lens_host[s]
            if not n or length <= 0:
                continue
            k = self.gathered(self.k, s).repeat_interleave(g, 0)
            rows = slice(int(self.offsets[s]), int(self.offsets[s + 1]))
            x = self.q[rows].double().transpose(0, 1)
            l = lse[rows].double().t()[..., None]
            m = self.mask(s, causal, window)
            z = (x @ k.transpose(1, 2) * self.scale - l).masked_fill(~m, -math.inf)
            dx = (self.d + 9) * U * (x.abs() @ k.abs().transpose(1, 2) * self.scale)
            w = torch.exp(z)
            rel = 2 * dx + 4 * U * torch.where(l.isfinite(), l, 0.0).abs() + (n * g + 8) * U
            add = w.unflatten(0, (self.hkv, g)).sum((1, 2))
            err = torch.where(m, w * rel, 0.0).unflatten(0, (self.hkv, g)).sum((1, 2))
            j = torch.arange(length, device="cuda")
            p, r = self.table[s].long()[j // self.page], j % self.page
            out[p, :, r] = decay * self.mass[p, :, r].double() + add.t()
            tol[p, :, r] = err.t() + 4 * U * out[p, :, r]
        return out, tol

    def check_weigh(self, causal=True, window=0, decay=1.0):
        lse = self.attend_ref(causal, window)[2].float()
        want, tol = self.weigh_ref(lse, causal, window, decay)
        out = self.mass.clone()
        assert self.cache.weigh(self.q, lse, self.offsets, causal=causal, window=window, decay=decay, out=out) is out
        bad = (out.double() - want).abs() > tol
        assert not bool((bad | out.isnan()).any()), (int(bad.sum()), float((out.double() - want).abs().max()))
        again = self.mass.clone()
        self.cache.weigh(self.q, lse, self.offsets, causal=causal, window=window, decay=decay, out=again)
        assert torch.equal(out, again)
        return out


RAGGED = [
    ("one token each", [1, 1, 1, 1, 1, 1], [1, 2, 15, 16, 17, 300]),
    ("one token, long", [1, 1], [4097, 2048]),
    ("some streams idle", [0, 1, 0, 3, 0], [0, 5, 77, 3, 16]),
    ("few tokens", [2, 5, 1, 8], [2, 64, 129, 1000]),
    ("whole prompts", [33, 128, 129, 200], [33, 128, 129, 200]),
    ("chunks after a cache", [64, 100, 256, 17], [500, 101, 256, 1300]),
    ("one long chunk", [700], [1111]),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("name,new,lens", RAGGED, ids=[r[0] for r in RAGGED])
def test_attend(lm, name, new, lens, layout, dtype):
    for page, order in ((16, "page"), (64, "slot")):
        b = Box(lm, *layout, page, dtype, new, lens, seed=len(name) + page, order=order)
        b.check_attend()
        assert b.plan.device_status() == 0


@pytest.mark.parametrize("new,lens", [([400], [9000]), ([130, 9, 260], [5000, 3000, 2600]), ([700] * 4, [900, 800, 3000, 700]),
                                      ([1500], [1500]), ([300] * 30, [300 + 10 * i for i in range(30)])])
def test_attend_long(lm, new, lens):
    """Many tiles of keys for a CTA: the ring goes round, items are split and joined, whole items go first."""
    for layout, dtype in (((16, 8, 128), torch.bfloat16), ((4, 4, 64), torch.float16)):
        b = Box(lm, *layout, 64, dtype, new, lens, seed=1)
        b.check_attend()
        b.check_attend(window=700)
        b.check_weigh()
        assert b.plan.device_status() == 0


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("causal,window", [(True, 1), (True, 50), (True, 128), (False, 0), (False, 70), (True, 10**12)])
def test_attend_masks_and_pages(lm, page, causal, window):
    for layout, dtype in (((16, 8, 128), torch.bfloat16), ((14, 2, 64), torch.float16)):
        for new, lens in (([1, 1, 1], [1, 130, 777]), ([3, 1, 0, 7], [400, 64, 9, 7]), ([150, 1, 40], [333, 128, 1000])):
            b = Box(lm, *layout, page, dtype, new, lens, seed=page)
            b.check_attend(causal, window)
            b.check_weigh(causal, window)
            assert b.plan.device_status() == 0


@pytest.mark.parametrize("new", [[5, 1, 4, 3], [140, 1, 9, 3]])
def test_rows_that_see_nothing(lm, new):
    """Lengths shorter than the push, or zero: those rows are zero and their lse minus infinity."""
    for causal in (True, False):
        b = Box(lm, 16, 8, 128, 16, torch.bfloat16, new, [3, 0, 4, 200])
        b.check_attend(causal)
        b.check_weigh(causal)
        assert b.plan.device_status() == 0


def test_against_the_oracle(lm):
    for window in (0, 6):
        b = Box(lm, 4, 2, 64, 16, torch.float16, [2, 0, 1, 5], [20, 3, 1, 9])
        a = dict(table=b.table.cpu().numpy(), lens=b.lens.cpu().numpy(), offsets=b.offsets, scale=b.scale, window=window)
        out, lse, _, _ = CO.attend(b.q.double().cpu().numpy(), b.k.double().cpu().numpy(), b.v.double().cpu().numpy(), **a)
        want, tol, wl, _ = b.attend_ref(True, window)
        assert np.allclose(out, want.cpu().numpy(), atol=1e-12) and np.allclose(lse, wl.cpu().numpy(), atol=1e-12)
        lse32 = wl.float()
        m, _, _ = CO.weigh(b.q.double().cpu().numpy(), lse32.cpu().numpy(), b.k.double().cpu().numpy(),
                           b.mass.cpu().numpy(), decay=0.5, **a)
        assert np.allclose(m, b.weigh_ref(lse32, True, window, 0.5)[0].cpu().numpy(), atol=1e-12)
        b.check_attend(True, window)
        b.check_weigh(True, window, 0.5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("name,new,lens", RAGGED, ids=[r[0] for r in RAGGED])
def test_weigh(lm, name, new, lens, layout, dtype):
    b = Box(lm, *layout, 32, dtype, new, lens, seed=3)
    out = b.check_weigh(decay=0.75)
    idle = [s for s, n in enumerate(new) if n == 0]
    for s in idle:                                            # streams without new rows stay as they are
        p = b.table[s, :-(-lens[s] // 32)].long()
        assert torch.equal(out[p], b.mass[p])
    inplace = b.cache.mass
    lse = b.attend_ref()[2].float()
    assert b.cache.weigh(b.q, lse, b.offsets, decay=0.75) is inplace and torch.equal(inplace, out)


@pytest.mark.parametrize("new,lens", [([2, 3], [40, 35]), ([6], [300]), ([100, 40], [130, 300]), ([300], [300])])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(lm, new, lens, value):
    for window in (0, 9):
        for layout, dtype in (((16, 8, 128), torch.bfloat16), ((14, 2, 64), torch.float16)):
            b = Box(lm, *layout, 16, dtype, new, lens)
            want = b.check_attend(window=window)[0]
            for back in sorted({0, 1, new[0] // 2, new[0] - 1, min(new[0] + 3, lens[0] - 1)}):
                j = lens[0] - 1 - back                        # a slot of stream 0, dimension 5 of its last key head
                page = int(b.table[0, j // 16])
                keep = b.v[page, -1, j % 16, 5].clone()
                b.v[page, -1, j % 16, 5] = value
                out = b.cache.attend(b.q, b.offsets, window=window)
                b.v[page, -1, j % 16, 5] = keep
                sees = b.mask(0, True, window)[:, j]
                hit = torch.zeros_like(out, dtype=torch.bool)
                hit[:new[0], -(b.hq // b.hkv):, 5] = sees[:, None]
                assert torch.equal(~out.isfinite(), hit), (back, window)
                if not math.isnan(value):
                    assert bool((out[hit].float() == value).all())
                assert torch.equal(out[~hit], want[~hit])


@pytest.mark.parametrize("new,lens", [([2, 3], [40, 35]), ([100, 40], [130, 300]), ([300], [300])])
def test_keys_that_are_nan_reach_the_rows_that_see_them(lm, new, lens):
    for window in (0, 9):
        for layout, dtype in (((16, 8, 128), torch.bfloat16), ((14, 2, 64), torch.float16)):
            b = Box(lm, *layout, 16, dtype, new, lens)
            want, tol, _, _ = b.attend_ref(window=window)
            for back in sorted({0, 1, new[0] // 2, new[0] - 1, min(new[0] + 3, lens[0] - 1)}):
                j = lens[0] - 1 - back
                page = int(b.table[0, j // 16])
                keep = b.k[page, 0, j % 16, 5].clone()
                b.k[page, 0, j % 16, 5] = math.nan
                out, lse = b.cache.attend(b.q, b.offsets, window=window, return_lse=True)
                mass = b.mass.clone()
                b.cache.weigh(b.q, torch.zeros_like(lse), b.offsets, window=window, out=mass)
                b.k[page, 0, j % 16, 5] = keep
                hit = torch.zeros_like(out, dtype=torch.bool)
                hit[:new[0], :b.hq // b.hkv] = b.mask(0, True, window)[:, j][:, None, None]
                assert torch.equal(out.isnan(), hit) and torch.equal(lse.isnan(), hit[:, :, 0]), (back, window)
                assert bool((((out.double() - want).abs() <= tol) | hit).all())
                live = torch.zeros_like(mass, dtype=torch.bool)
                live[page, 0, j % 16] = True
                assert torch.equal(mass.isnan(), live)


def test_weights_past_the_largest_number(lm):
    """An lse far below the scores gives infinity, not a wrapped exponent."""
    for new, lens in (([1], [70]), ([140], [300])):
        b = Box(lm, 16, 8, 128, 16, torch.bfloat16, new, lens)
        lse = torch.full((b.rows, 16), -200.0, device="cuda")
        out = b.mass.clone()
        b.cache.weigh(b.q, lse, b.offsets, out=out)
        live = b.live[:, 0, :, 0][:, None].expand_as(out)
        assert bool((out[live] == math.inf).all()) and torch.equal(out[~live], b.mass[~live])


def test_two_plans_at_once(lm):
    """Calls on plans of their own may overlap on the GPU."""
    boxes = [Box(lm, 16, 8, 128, 16, torch.bfloat16, new, lens, seed=i)
             for i, (new, lens) in enumerate([([1] * 9, [700 + 90 * i for i in range(9)]), ([200, 40], [2000, 900]),
                                              ([130], [5000]), ([1, 1], [9000, 40])])]
    want = [b.check_attend() for b in boxes]
    streams = [torch.cuda.Stream() for _ in boxes]
    masses = [b.mass.clone() for b in boxes]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for b, st, m in zip(boxes, streams, masses):
            with torch.cuda.stream(st):
                out, lse = b.cache.attend(b.q, b.offsets, return_lse=True)
                b.cache.weigh(b.q, lse, b.offsets, out=m)
                got.append((out, lse))
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, want[i % 4][0]) and torch.equal(lse, want[i % 4][1])
    for b, m, (_, lse) in zip(boxes, masses, want):
        again = b.mass.clone()
        b.cache.weigh(b.q, lse, b.offsets, out=again)
        assert torch.equal(m, again) and b.plan.device_status() == 0


def test_many_heads_share_one(lm):
    """64 query heads over one key head: a single token fills half a tile."""
    for d, dtype in ((64, torch.float16), (128, torch.bfloat16)):
        for new, lens in (([1, 1], [300, 4000]), ([3, 0, 9], [3, 9, 500])):
            b = Box(lm, 64, 1, d, 32, dtype, new, lens)
            b.check_attend()
            b.check_attend(window=20)
            b.check_weigh()


def test_large_and_small_scores(lm):
    """One key carries everything; a key far below the others; equal scores; huge scores."""
    b = Box(lm, 16, 8, 128, 16, torch.bfloat16, [1, 20, 150], [600, 400, 300], sharp=40.0)
    b.check_attend()
    b.check_weigh()
    b = Box(lm, 16, 8, 128, 16, torch.float16, [1, 20, 150], [600, 400, 300], sharp=0.0)
    b.check_attend()
    b = Box(lm, 20, 20, 64, 16, torch.bfloat16, [1, 9, 150], [600, 400, 300])
    b.k.mul_(torch.linspace(0.01, 12.0, b.page, device="cuda")[:, None])      # the maximum rises from slot to slot
    b.check_attend()
    b.check_weigh()


def test_softmax_scale(lm):
    b = Box(lm, 16, 8, 128, 16, torch.bfloat16, [1, 40], [300, 77], softmax_scale=0.31)
    b.scale = 0.31
    b.check_attend()
    b.check_weigh()


def test_strided_rows_and_outputs(lm):
    b = Box(lm, 16, 8, 128, 16, torch.bfloat16, [1, 30, 7], [300, 77, 7])
    want, lse = b.check_attend()
    wide = torch.full((b.rows, 40, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:19] = b.q
    out = wide[:, 20:36]
    b.cache.attend(wide[:, 3:19], b.offsets, out=out)
    assert torch.equal(out, want)
    assert bool((wide[:, :3] == 7).all()) and bool((wide[:, 19] == 7).all()) and bool((wide[:, 36:] == 7).all())
    heads_first = torch.empty(16, b.rows + 5, 128, dtype=torch.bfloat16, device="cuda").fill_(3.0)
    out = heads_first[:, :b.rows].transpose(0, 1)
    b.cache.attend(b.q.transpose(0, 1).contiguous().transpose(0, 1), b.offsets, out=out)
    assert torch.equal(out, want) and bool((heads_first[:, b.rows:] == 3).all())
    a, c = b.mass.clone(), b.mass.clone()
    b.cache.weigh(b.q, lse, b.offsets, out=a)
    b.cache.weigh(wide[:, 3:19], lse, b.offsets, out=c)
    assert torch.equal(a, c)


def test_many_streams(lm):
    """More ragged streams than one launch takes, idle ones among them, and uniform ones."""
    r = np.random.default_rng(5)
    new = [int(x) for x in r.integers(0, 3, 1300)]
    lens = [n + int(x) for n, x in zip(new, r.integers(0, 60, 1300))]
    b = Box(lm, 4, 2, 64, 16, torch.bfloat16, new, lens)
    b.check_attend()
    b.check_weigh()
    one = Box(lm, 4, 2, 64, 16, torch.bfloat16, [1] * 5000, [1 + (i * 7) % 50 for i in range(5000)])
    one.check_attend()
    one.check_weigh()
    mixed = Box(lm, 4, 2, 64, 16, torch.bfloat16, [1] * 600 + [40], [30] * 600 + [50])
    mixed.check_attend()
    mixed.check_weigh()


def test_no_rows(lm):
    b = Box(lm, 4, 2, 64, 16, torch.bfloat16, [0, 0], [5, 9])
    q = b.q
    assert b.cache.attend(q, b.offsets).shape == (0, 4, 64)
    assert b.cache.append(q, b.qkv[:, :2], b.qkv[:, 2:4], b.offsets).shape == (0, 4, 64)
    before = b.mass.clone()
    b.cache.weigh(q, torch.empty(0, 4, device="cuda"), b.offsets)
    assert torch.equal(b.mass, before)


def test_same_bits_every_time(lm):
    for new, lens in (([1] * 6, [900, 10, 3000, 77, 1, 500]), ([300, 1, 60], [2000, 700, 60])):
        b = Box(lm, 16, 8, 128, 16, torch.bfloat16, new, lens)
        first = b.cache.attend(b.q, b.offsets, return_lse=True)
        for _ in range(5):
            again = b.cache.attend(b.q, b.offsets, return_lse=True)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_pages_far_apart(lm):
    """Pages whose element offsets pass 2^31 and whose byte offsets pass 2^32."""
    hkv, page, d = 8, 256, 128
    n_pages = (1 << 31) // (2 * hkv * page * d) + 40
    kv = torch.empty(n_pages, 2, hkv, page, d, dtype=torch.bfloat16, device="cuda")
    assert kv.stride(0) * (n_pages - 1) > 1 << 31
    plan = lm.CachePlan(16, hkv, d, page, rotary_dim=128)
    last = [n_pages - 1, 0, n_pages - 2, n_pages - 3, n_pages - 4]
    table = torch.tensor([last[:3], last[3:] + [0]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([600, 512], dtype=torch.int32, device="cuda")
    mass = torch.zeros(n_pages, hkv, page, device="cuda")
    kv[last] = torch.randn(5, 2, hkv, page, d, device="cuda").to(torch.bfloat16)
    small = kv[last].clone()
    small_table = torch.tensor([[0, 1, 2], [3, 4, 0]], dtype=torch.int32, device="cuda")
    small_mass = torch.zeros(5, hkv, page, device="cuda")
    for n in (1, 90):
        x = torch.randn(2 * n, 32, d, device="cuda").to(torch.bfloat16)
        got = []
        for pool, tab, ms in ((kv, table, mass), (small, small_table, small_mass)):
            c = lm.TokenCache(plan, pool[:, 0], pool[:, 1], tab, lens, mass=ms)
            q = c.append(x[:, :16], x[:, 16:24], x[:, 24:])
            out, lse = c.attend(q, return_lse=True)
            c.weigh(q, lse)
            got.append((q, out, lse, ms if ms is small_mass else ms[last]))
        for a, b in zip(*got):
            assert torch.equal(a, b)
        assert torch.equal(kv[last], small)
    to = lm.TokenCache.empty(plan, 2, 256)
    c = lm.TokenCache(plan, kv[:, 0], kv[:, 1], table, lens, mass=mass)
    kept = c.evict(to, 200, recent=20)
    s = lm.TokenCache(plan, small[:, 0], small[:, 1], small_table, lens, mass=small_mass)
    to2 = lm.TokenCache.empty(plan, 2, 256)
    assert torch.equal(kept, s.evict(to2, 200, recent=20))
    assert torch.equal(to.k_pages[:, :, :200], to2.k_pages[:, :, :200])
    assert plan.device_status() == 0


# --- append ------------------------------------------------------------------


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("layout,rot", [((16, 8, 128), 128), ((16, 8, 128), 32), ((20, 20, 64), 64), ((3, 1, 64), 16),
                                        ((14, 2, 64), 48), ((8, 1, 128), 0)])
@pytest.mark.parametrize("scaling", [{}, dict(rotary_scaling="linear", rotary_factor=4.0),
                                     dict(rotary_scaling="ramp", rotary_factor=4.0, rotary_context=2048)])
def test_append(lm, layout, rot, dtype, interleaved, scaling):
    new, lens = [1, 0, 40, 17], [1, 5, 55, 1000]
    b = Box(lm, *layout, 16, dtype, new, lens, rotary_dim=rot, rotary_base=1e5, interleaved=interleaved, **scaling)
    far = torch.tensor([0, 2**31 - 1, 1000000, 65535] * 15, device="cuda")[:b.rows].to(torch.int32)
    sc = scaling.get("rotary_scaling")
    freq, length = CO.rotary(rot, 1e5, sc, scaling.get("rotary_factor", 1.0), scaling.get("rotary_context", 0))
    hq, hkv = b.hq, b.hkv
    e = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    x = b.qkv.double().cpu().numpy()
    own = np.concatenate([lens[s] - n + np.arange(n) for s, n in enumerate(new)])
    for pos in (None, far):
        k0, v0 = b.k.clone(), b.v.clone()
        q = b.cache.append(b.qkv[:, :hq], b.qkv[:, hq:hq + hkv], b.qkv[:, hq + hkv:], b.offsets, positions=pos)
        where = own.astype(np.float64) if pos is None else pos.double().cpu().numpy()
        want = CO.turn(x[:, :hq + hkv], where, freq, length, interleaved)
        size = CO.turn(np.abs(x[:, :hq + hkv]), np.zeros(b.rows), freq, 1.0, interleaved)
        both = size.copy()                                    # |a| + |b| of every pair
        half = rot // 2
        for i in range(half):
            i0, i1 = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            both[..., i0] = both[..., i1] = size[..., i0] + size[..., i1]
        tol = e * np.abs(want) + (2.0 ** -23 + 4 * U) * length * both + tiny
        tol[..., rot:] = 0.0
        assert np.all(np.abs(q.double().cpu().numpy() - want[:, :hq]) <= tol[:, :hq])
        kd = b.k.double().cpu().numpy()
        t = 0
        touched = torch.zeros(b.k.shape[0], 16, dtype=torch.bool)
        for s, n in enumerate(new):
            p, r = CO.slots(b.table.cpu().numpy(), 16, s, lens[s] - n, lens[s])
            assert np.all(np.abs(kd[p, :, r] - want[t:t + n, hq:]) <= tol[t:t + n, hq:])
            assert torch.equal(b.v[torch.tensor(p), :, torch.tensor(r)], b.qkv[t:t + n, hq + hkv:])
            touched[p, r] = True
            t += n
        rest = ~touched.cuda()[:, None, :, None]
        same = lambda a, c: bool(((a == c) | (a.isnan() & c.isnan()) | ~rest).all())
        assert same(b.k, k0) and same(b.v, v0)               # every other slot is as it was
        inplace = b.qkv.clone()
        assert b.cache.append(inplace[:, :hq], inplace[:, hq:hq + hkv], inplace[:, hq + hkv:], b.offsets, positions=pos,
                              q_out=inplace[:, :hq]) is not None
        assert torch.equal(inplace[:, :hq], q) and torch.equal(inplace[:, hq:], b.qkv[:, hq:])
    assert b.plan.device_status() == 0


def test_append_matches_distance(lm):
    """Scores of appended rows depend on the distance alone, near and far (float32 angles would be off by 4e-3)."""
    b = Box(lm, 1, 1, 128, 16, torch.float16, [2], [2], rotary_dim=128, rotary_base=1e6)
    scores = []
    for first in (0, 1000003, 2**31 - 10):
        pos = torch.tensor([first, first + 7], dtype=torch.int32, device="cuda")
        q = b.cache.append(b.qkv[:, :1], b.qkv[:, 1:2], b.qkv[:, 2:], b.offsets, positions=pos)
        k = b.k[int(b.table[0, 0]), 0, 0]
        scores.append(float(q[1, 0].double() @ k.double()))
    a, c = b.qkv[1, 0].double(), b.qkv[0, 1].double()
    tol = 3 * torch.finfo(torch.float16).eps / 2 * float(a.abs().max() * c.abs().max()) * 128 ** 0.5 * 4
    assert max(scores) - min(scores) <= tol


# --- evict -------------------------------------------------------------------


def _evict_case(lm, lens, budget, recent, layout=(16, 8, 128), page=16, dtype=torch.bfloat16, ties=True, seed=0, mass=None):
    b = Box(lm, *layout, page, dtype, [1] * len(lens), lens, seed=seed)
    if ties:
        b.mass.copy_((b.mass * 8).floor() / 8)
    if mass is not None:
        mass(b)
    to = lm.TokenCache.empty(b.plan, len(lens), budget)
    for t in (to.k_pages, to.v_pages, to.mass):
        t.fill_(9.0)
    kept = b.cache.evict(to, budget, recent=recent)
    want = CO.evict(b.mass.cpu().numpy(), b.table.cpu().numpy(), lens, page, budget, recent)
    assert torch.equal(to.lens.cpu(), torch.tensor([min(x, budget) for x in lens], dtype=torch.int32))
    for s, length in enumerate(lens):
        m = min(length, budget)
        for h in range(b.hkv):
            assert kept[s, h, :m].tolist() == want[s][h] and bool((kept[s, h, m:] == -1).all())
            j = torch.tensor(want[s][h], dtype=torch.long, device="cuda")
            i = torch.arange(m, device="cuda")
            src = b.table[s].long()[j // page], h, j % page
            dst = to.table[s].long()[i // page], h, i % page
            for x, y in ((b.k, to.k_pages), (b.v, to.v_pages), (b.mass, to.mass)):
                assert torch.equal(x[src].nan_to_num(77.0), y[dst].nan_to_num(77.0))
        free = torch.arange(m, to.table.shape[1] * page, device="cuda")
        p, r = to.table[s].long()[free // page], free % page
        assert bool((to.k_pages[p, :, r] == 9).all()) and bool((to.mass[p, :, r] == 9).all())
    assert b.plan.device_status() == 0
    return b, to, kept


@pytest.mark.parametrize("layout,page,dtype", [((16, 8, 128), 16, torch.bfloat16), ((14, 2, 64), 64, torch.float16),
                                               ((3, 1, 64), 256, torch.bfloat16)])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (100, 0), (100, 30), (100, 100), (513, 100), (3000, 7)])
def test_evict(lm, layout, page, dtype, budget, recent):
    _evict_case(lm, [0, 1, 99, 100, 101, 600, 2500], budget, recent, layout, page, dtype)


def test_evict_orders_special_weights(lm):
    def special(b):
        flat = b.mass.view(-1)
        flat[::7], flat[1::7], flat[2::7], flat[3::7], flat[4::7] = math.nan, math.inf, 0.0, -0.0, -1.0
    _evict_case(lm, [40, 333], 20, 3, mass=special)
    _evict_case(lm, [40, 333], 35, 0, mass=lambda b: b.mass.zero_())
    _evict_case(lm, [40, 333], 35, 0, mass=lambda b: b.mass.fill_(1e-42))
    _evict_case(lm, [2000], 777, 10, ties=False)
    _evict_case(lm, [9000, 4000], 2048, 100, layout=(2, 2, 128), page=128, seed=4)


@pytest.mark.parametrize("lens,page", [([5000, 7], 16), ([8000, 4096], 64), ([16000], 16), ([33000, 20000], 256)])
def test_evict_long_streams(lm, lens, page):
    """Streams that several CTAs select from together, ties in plenty among them."""
    for ties in (True, False):
        _evict_case(lm, lens, 1500, 200, layout=(2, 1, 64), page=page, ties=ties, seed=page)
    _evict_case(lm, lens, 1500, 0, layout=(2, 1, 64), page=page, mass=lambda b: b.mass.zero_())


def test_evict_within_one_pool(lm):
    """The kept rows may go to other pages of the same tensors."""
    plan = lm.CachePlan(4, 2, 64, 16)
    k = torch.randn(40, 2, 16, 64, device="cuda").to(torch.bfloat16)
    v, mass = torch.randn_like(k), torch.rand(40, 2, 16, device="cuda")
    lens = torch.tensor([300, 170], dtype=torch.int32, device="cuda")
    table = torch.randperm(40, device="cuda", dtype=torch.int32)
    src, dst = torch.zeros(2, 19, dtype=torch.int32, device="cuda"), torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    src[0, :19], src[1, :11], dst[0], dst[1] = table[:19], table[19:30], table[30:34], table[34:38]
    c = lm.TokenCache(plan, k, v, src, lens, mass=mass)
    to = lm.TokenCache(plan, k, v, dst, torch.zeros_like(lens), mass=mass)
    before = k.clone(), mass.clone()
    kept = c.evict(to, 64, recent=5)
    want = CO.evict(before[1].cpu().numpy(), src.cpu().numpy(), [300, 170], 16, 64, 5)
    assert kept.tolist() == want
    for s in range(2):
        assert torch.equal(k[src[s, :-(-int(lens[s]) // 16)].long()], before[0][src[s, :-(-int(lens[s]) // 16)].long()])
        j = kept[s, 1].long()
        assert torch.equal(k[dst[s].long()][:, 1].reshape(64, 64), before[0][src[s].long()[j // 16], 1, j % 16])


# --- together, as they are used ----------------------------------------------


def test_a_stream_from_push_to_push(lm):
    """Pushes of ragged sizes through append, attend, weigh, with a cut in between, against one float64 stream."""
    torch.manual_seed(1)
    hq, hkv, d, page, S = 8, 4, 64, 16, 3
    plan = lm.CachePlan(hq, hkv, d, page, rotary_dim=32, rotary_base=1e4)
    cache = lm.TokenCache.empty(plan, S, 400)
    freq, _ = CO.rotary(32, 1e4)
    hist = [[[] for _ in range(hkv)] for _ in range(S)]       # (turned key, value, weight) per kept slot, float64
    seen_so_far = [0] * S
    e = torch.finfo(torch.bfloat16).eps / 2
    for step, new in enumerate([[5, 1, 30], [1, 1, 1], [0, 40, 2], [1, 1, 1], [17, 3, 0], [1, 1, 1]]):
        off = np.concatenate([[0], np.cumsum(new)])
        rows = int(off[-1])
        x = torch.randn(rows, hq + 2 * hkv, d, device="cuda").to(torch.bfloat16)
        x[:, :hq] *= 2
        pos = np.concatenate([seen_so_far[s] + np.arange(n) for s, n in enumerate(new)])
        cache.lens.add_(torch.tensor(new, dtype=torch.int32, device="cuda"))
        q = cache.append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], off,
                         positions=torch.tensor(pos, dtype=torch.int32, device="cuda"))
        out, lse = cache.attend(q, off, return_lse=True)
        cache.weigh(q, lse, off)
        # rows as the cache holds them (one rounding), then everything in float64
        turned = torch.from_numpy(CO.turn(x[:, :hq + hkv].double().cpu().numpy(), pos.astype(float), freq, 1.0, False))
        assert bool(((q.double().cpu() - turned[:, :hq]).abs() <= e * turned[:, :hq].abs() + 2e-6 * 8).all())
        turned = turned.to(torch.bfloat16).double()
        xd = x.double().cpu()
        for s, n in enumerate(new):
            seen_so_far[s] += n
            for i in range(n):
                t = int(off[s]) + i
                for h in range(hkv):
                    hist[s][h].append([turned[t, hq + h], xd[t, hq + hkv + h], 0.0])
                    k = torch.stack([r[0] for r in hist[s][h]])
                    v = torch.stack([r[1] for r in hist[s][h]])
                    for g in range(2):
                        z = k @ q[t, 2 * h + g].double().cpu() * d ** -0.5
                        w = z.softmax(0)
                        # a turned key may round the other way (relative 2 e of a pair), which moves a score by up to
                        # 2 e * scale * sum|q k|; that bounds the weights' relative change by twice as much
                        dz = 2 * e * float((k.abs() @ q[t, 2 * h + g].double().cpu().abs()).max()) * d ** -0.5
                        spread = w @ v.abs()
                        assert bool(((out[t, 2 * h + g].double().cpu() - w @ v).abs()
                                     <= (2 * e + 2 * dz + 1e-5) * spread + e * spread).all())
                        for r, y in zip(hist[s][h], w.tolist()):
                            r[2] += y
        for s in range(S):
            for h in range(hkv):
                length = len(hist[s][h])
                p, r = CO.slots(cache.table.cpu().numpy(), page, s, 0, length)
                got = cache.mass[torch.tensor(p, device="cuda"), h, torch.tensor(r, device="cuda")].double().cpu()
                want = torch.tensor([y[2] for y in hist[s][h]], dtype=torch.float64)
                assert bool(((got - want).abs() <= 0.1 * want + 1e-6).all())     # keys' other roundings, as above
        if step == 3:
            to = lm.TokenCache.empty(plan, S, 400)
            kept = cache.evict(to, 20, recent=6)
            for s in range(S):
                for h in range(hkv):
                    rows_kept = [j for j in kept[s, h].tolist() if j >= 0]
                    assert len(rows_kept) == min(20, len(hist[s][h]))
                    hist[s][h] = [hist[s][h][j] for j in rows_kept]
                    p, r = CO.slots(to.table.cpu().numpy(), page, s, 0, len(rows_kept))
                    got = to.mass[torch.tensor(p, device="cuda"), h, torch.tensor(r, device="cuda")].tolist()
                    for y, m in zip(hist[s][h], got):
                        y[2] = m
            cache = to
    assert plan.device_status() == 0


def test_beside_the_spectrogram_stream(lm):
    """Rows of a streaming push become tokens of the cache: one push, one ragged attend, the counts of the push."""
    plan, st_n = lm.Plan(), 3
    st = lm.Stream(plan, st_n)
    cp = lm.CachePlan(2, 1, 64, 16, dtype=torch.float16, rotary_dim=64)
    cache = lm.TokenCache.empty(cp, st_n, 200)
    proj = torch.randn(128, 4 * 64, device="cuda") * 0.02
    for push in range(4):
        lens = [1280, 400 + 160 * push, 0 if push == 1 else 2000]
        off = np.concatenate([[0], np.cumsum(lens)])
        rows, n = st.push_batch_ragged(torch.randn(int(off[-1]), device="cuda"), off)
        x = torch.cat([rows[s, :n[s]] for s in range(st_n)]) @ proj
        x = x.view(-1, 4, 64).to(torch.float16)
        cache.lens.add_(torch.from_numpy(n).to(torch.int32).cuda())
        o = np.concatenate([[0], np.cumsum(n)])
        q = cache.append(x[:, :2], x[:, 2:3], x[:, 3:], o)
        out = cache.attend(q, o, window=50)
        assert out.shape[0] == int(n.sum()) and bool(out.isfinite().all())
        assert torch.equal(out, cache.attend(q, o, window=50))
    assert cp.device_status() == 0


# --- streams, graphs, refusals, bad tables ------------------------------------


def test_captured_step_follows_lengths(lm):
    """A captured decode step replays with the lengths, tables and rows of the moment."""
    for n in (1, 3, 40):
        b = Box(lm, 16, 8, 128, 16, torch.bfloat16, [n] * 4, [40, 200, 41, 640], rotary_dim=128)
        for p in (b.k, b.v):
            p.copy_(torch.randn(p.shape, device="cuda").to(p.dtype))
        x = torch.randn(4 * n, 32, 128, device="cuda").to(torch.bfloat16)
        out_mass = b.mass.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(g, stream=side):
                q = b.cache.append(x[:, :16], x[:, 16:24], x[:, 24:])
                out, lse = b.cache.attend(q, return_lse=True)
                b.cache.weigh(q, lse, out=out_mass)
        torch.cuda.current_stream().wait_stream(side)
        g2 = torch.cuda.CUDAGraph()                            # a second graph on the same plan
        with torch.cuda.graph(g2):
            out2 = b.cache.attend(q, window=33)
        for lens in ([40, 200, 41, 640], [n, n, n, n], [640 - 600, 150, 39, 500]):
            b.lens.copy_(torch.tensor(lens, dtype=torch.int32))
            x.copy_(torch.randn_like(x))
            g.replay()
            g2.replay()
            g.replay()
            got = out.clone(), lse.clone(), out_mass.clone(), out2.clone()
            b.lens_host, b.q = lens, q
            want = b.check_attend()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert torch.equal(got[3], b.cache.attend(q, window=33))
            again = out_mass.clone()
            b.cache.weigh(q, lse, out=again)
            assert torch.equal(again, got[2])
            # append reports a row whose slot would lie below zero (39 tokens cannot hold a push of 40)
            assert b.plan.device_status() == (4 if min(lens) < n else 0)


def test_given_streams(lm):
    """Work goes to the stream that is given, whichever is current."""
    b = Box(lm, 16, 8, 128, 16, torch.bfloat16, [1, 40], [300, 77], rotary_dim=128)
    want, lse = b.check_attend()
    side = torch.cuda.Stream()
    x = torch.empty_like(b.q)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        x.copy_(b.q)                                           # the rows arrive late, on the other stream
    out, got_lse = b.cache.attend(x, b.offsets, return_lse=True, stream=side)
    m = b.mass.clone()
    side.wait_stream(torch.cuda.current_stream())
    b.cache.weigh(x, got_lse, b.offsets, out=m, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(got_lse, lse)
    m2 = b.mass.clone()
    b.cache.weigh(b.q, lse, b.offsets, out=m2)
    assert torch.equal(m, m2)


@pytest.mark.parametrize("new", [[1, 1, 1], [90, 1, 20]])
def test_bad_tables_and_lengths_are_reported_not_followed(lm, new):
    """A page id or a length out of range: the status word says so, other streams are right, nothing else is written."""
    for what in ("high page", "negative page", "long", "negative"):
        b = Box(lm, 16, 8, 128, 16, torch.bfloat16, new, [300, 120, 77], rotary_dim=128)
        want, _ = b.check_attend()
        lse = b.attend_ref()[2].float()
        good = b.mass.clone()
        b.cache.weigh(b.q, lse, b.offsets, out=good)
        if what == "high page":
            b.table[1, 3] = b.k.shape[0]
        elif what == "negative page":
            b.table[1, 3] = -1
        else:
            b.lens[1] = b.table.shape[1] * 16 + 1 if what == "long" else -5
        if what == "long":
            b.table[1] = b.table[1, 0]
        assert b.plan.device_status() == 0
        out = b.cache.attend(b.q, b.offsets)
        assert b.plan.device_status() == 4, what
        rows = np.r_[0:b.offsets[1], b.offsets[2]:b.rows]
        assert torch.equal(out[rows], want[rows]), what
        m = b.mass.clone()
        b.cache.weigh(b.q, lse, b.offsets, out=m)
        assert b.plan.device_status() == 4, what
        for s in (0, 2):
            p = b.table[s, :-(-b.lens_host[s] // 16)].long()
            assert torch.equal(m[p], good[p]), what
        if what in ("long", "negative"):
            before = b.k.clone()
            b.cache.append(b.qkv[:, :16], b.qkv[:, 16:24], b.qkv[:, 24:], b.offsets)
            assert b.plan.device_status() == 4, what
            if what == "negative":
                own = b.table[1, :8].long()
                assert torch.equal(b.k[own].nan_to_num(1.0), before[own].nan_to_num(1.0))
        to = lm.TokenCache.empty(b.plan, 3, 50)
        b.cache.evict(to, 50)
        assert b.plan.device_status() == 4, what
        assert b.plan.device_status() == 0
    b = Box(lm, 16, 8, 128, 16, torch.bfloat16, new, [300, 120, 77])
    to = lm.TokenCache.empty(b.plan, 3, 50)
    to.table[1, 0] = 10 ** 6
    b.cache.evict(to, 50)
    assert b.plan.device_status() == 4


def test_waits_that_run_out_are_reported(lm):
    """Copies that never complete a barrier: the calls end, the status word says so, the next calls are right."""
    b = Box(lm, 16, 8, 128, 16, torch.bfloat16, [90, 1, 20], [300, 120, 777])
    want, lse = b.check_attend()
    masses = b.mass.clone()
    b.cache.weigh(b.q, lse, b.offsets, out=masses)
    for bad in (-16, 8, (1 << 19) + 16):
        with pytest.raises(lm.LogMelError):
            b.plan.set_wait_test(bad)
    for call in (lambda: b.cache.attend(b.q, b.offsets), lambda: b.cache.weigh(b.q, lse, b.offsets, out=b.mass.clone())):
        b.plan.set_wait_test(16)
        call()
        b.plan.set_wait_test(0)
        assert b.plan.device_status() == 5
        assert b.plan.device_status() == 0
        out, got = b.cache.attend(b.q, b.offsets, return_lse=True)
        again = b.mass.clone()
        b.cache.weigh(b.q, lse, b.offsets, out=again)
        assert torch.equal(out, want) and torch.equal(got, lse) and torch.equal(again, masses)
        assert b.plan.device_status() == 0
    # a bad length after it does not hide it
    b.plan.set_wait_test(16)
    b.cache.attend(b.q, b.offsets)
    b.plan.set_wait_test(0)
    good = b.cache.lens.clone()
    b.cache.lens[0] = -1
    b.cache.attend(b.q, b.offsets)
    b.cache.lens.copy_(good)
    assert b.plan.device_status() == 5
    assert torch.equal(b.cache.attend(b.q, b.offsets), want)


def test_refusals(lm):
    b = Box(lm, 16, 8, 128, 16, torch.bfloat16, [1, 2], [30, 40], rotary_dim=128)
    c, q = b.cache, b.q
    k, v = b.qkv[:, 16:24], b.qkv[:, 24:]
    lse = torch.zeros(3, 16, device="cuda")
    cases = [
        (TypeError, lambda: c.attend(q.half(), b.offsets)), (TypeError, lambda: c.attend(q.cpu(), b.offsets)),
        (ValueError, lambda: c.attend(q[:, :8], b.offsets)), (ValueError, lambda: c.attend(q[..., :64], b.offsets)),
        (ValueError, lambda: c.attend(q)), (ValueError, lambda: c.attend(q, [0, 1])),
        (ValueError, lambda: c.attend(q, [0, 1, 2])), (ValueError, lambda: c.attend(q, [1, 1, 3])),
        (lm.LogMelError, lambda: c.attend(q, [0, 5, 3])), (lm.LogMelError, lambda: c.attend(q, b.offsets, window=-1)),
        (lm.LogMelError, lambda: c.attend(q, b.offsets, out=q)),
        (ValueError, lambda: c.attend(q, b.offsets, out=q[:2])),
        (ValueError, lambda: c.attend(q.transpose(1, 2).contiguous().transpose(1, 2), b.offsets)),
        (lm.LogMelError, lambda: c.attend(q, b.offsets, out=q[:1].expand(3, -1, -1).clone()[:1].expand(3, -1, -1))),
        (lm.LogMelError, lambda: c.attend(torch.zeros(3 * 16 * 128 + 1, dtype=torch.bfloat16, device="cuda")[1:]
                                          .view(3, 16, 128), b.offsets)),
        (lm.LogMelError, lambda: c.attend(torch.zeros(3, 16, 132, dtype=torch.bfloat16, device="cuda")[..., :128],
                                          b.offsets)),
        (TypeError, lambda: c.append(q, k, v, b.offsets, positions=torch.zeros(3, device="cuda"))),
        (ValueError, lambda: c.append(q, k, v, b.offsets, positions=torch.zeros(2, device="cuda", dtype=torch.int32))),
        (ValueError, lambda: c.append(q, k[:2], v, b.offsets)), (ValueError, lambda: c.append(q, k, v[:, :4], b.offsets)),
        (ValueError, lambda: c.weigh(q, lse[:2], b.offsets)), (TypeError, lambda: c.weigh(q, lse.double(), b.offsets)),
        (lm.LogMelError, lambda: c.weigh(q, lse, b.offsets, decay=math.inf)),
        (ValueError, lambda: c.weigh(q, lse, b.offsets, out=torch.zeros(3, device="cuda"))),
        (lm.LogMelError, lambda: c.evict(lm.TokenCache.empty(b.plan, 2, 32), 33)),
        (lm.LogMelError, lambda: c.evict(lm.TokenCache.empty(b.plan, 2, 32), 0)),
        (lm.LogMelError, lambda: c.evict(lm.TokenCache.empty(b.plan, 2, 32), 32, recent=33)),
        (lm.LogMelError, lambda: c.evict(lm.TokenCache.empty(b.plan, 2, 32), 32, recent=-1)),
        (lm.LogMelError, lambda: c.evict(lm.TokenCache.empty(b.plan, 3, 32), 32)),
        (lm.LogMelError, lambda: c.evict(lm.TokenCache(b.plan, b.k, b.v, b.table.clone(), b.lens, mass=b.mass), 32)),
        (lm.LogMelError, lambda: c.evict(lm.TokenCache(b.plan, b.k, b.v, b.table, torch.zeros_like(b.lens), mass=b.mass), 32)),
        (lm.LogMelError, lambda: c.evict(lm.TokenCache.empty(b.plan, 2, 32), 10 ** 30)),
        (lm.LogMelError, lambda: c.attend(q, b.offsets, window=-10 ** 30)),
        (lm.LogMelError, lambda: c.attend(q[:1].expand(3, -1, -1), b.offsets)),
        (TypeError, lambda: c.evict(None, 3)),
        (ValueError, lambda: c.evict(lm.TokenCache.empty(lm.CachePlan(16, 8, 64, 16), 2, 32), 3)),
        (TypeError, lambda: lm.TokenCache(b.plan, b.k.float(), b.v, b.table, b.lens)),
        (TypeError, lambda: lm.TokenCache(b.plan, b.k, b.v, b.table.long(), b.lens)),
        (ValueError, lambda: lm.TokenCache(b.plan, b.k[:, :4], b.v, b.table, b.lens)),
        (ValueError, lambda: lm.TokenCache(b.plan, b.k, b.v, b.table[:1], b.lens)),
        (ValueError, lambda: lm.TokenCache(b.plan, b.k, b.v, b.table, b.lens, mass=b.mass[:1])),
        (ValueError, lambda: lm.TokenCache(b.plan, b.k, b.v, b.table, b.lens).weigh(q, lse, b.offsets)),
        (lm.LogMelError, lambda: lm.TokenCache(b.plan, b.k[:1].expand(4, -1, -1, -1), b.v[:4], b.table, b.lens)
         .attend(q, b.offsets)),
        (lm.LogMelError, lambda: lm.TokenCache(b.plan, b.k, b.v, b.table, b.lens)
         .evict(lm.TokenCache.empty(b.plan, 2, 32), 5)),
    ]
    before = b.k.clone(), b.mass.clone()
    for i, (kind, call) in enumerate(cases):
        with pytest.raises(kind):
            call()
            print("case", i)
    torch.cuda.synchronize()
    assert torch.equal(b.k.nan_to_num(5.0), before[0].nan_to_num(5.0)) and torch.equal(b.mass, before[1])
    b.check_attend()
