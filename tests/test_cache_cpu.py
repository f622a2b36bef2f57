"""Token cache without a GPU: the rotary table, refusals that precede any CUDA
call, and the float64 oracle against independent facts."""
import ctypes
import math

import numpy as np
import pytest
import torch

import log_mel_spectrogram_logmel_b200 as lm
from oracle import cache_oracle as CO

CONFIG = dict(n_q_heads=16, n_kv_heads=8, head_dim=128, page_size=64, dtype=0, rotary_dim=128, interleaved=0,
              rotary_scaling=0, rotary_context=0, rotary_base=10000.0, rotary_factor=1.0, softmax_scale=0.0)


def _rotary(**change):
    c = lm._CacheConfig(**{**CONFIG, **change})
    inv = np.full(64, np.nan)
    length = ctypes.c_double(np.nan)
    code = lm._lib.logmel_cache_rotary(ctypes.addressof(c), inv.ctypes.data, ctypes.addressof(length))
    return code, inv, length.value


@pytest.mark.parametrize("dim", [0, 16, 64, 128])
@pytest.mark.parametrize("scaling,factor,context", [(None, 1.0, 0), ("linear", 4.0, 0), ("ramp", 4.0, 32768),
                                                    ("ramp", 8.0, 64), ("ramp", 1.0, 4096)])
@pytest.mark.parametrize("base", [500.0, 10000.0, 1e6])
def test_rotary_table(dim, scaling, factor, context, base):
    code, inv, length = _rotary(rotary_dim=dim, rotary_base=base, rotary_factor=factor, rotary_context=context,
                                rotary_scaling={None: 0, "linear": 1, "ramp": 2}[scaling])
    assert code == 0
    want, want_length = CO.rotary(dim, base, scaling, factor, context)
    # a handful of float64 operations each
    assert np.allclose(inv[:dim // 2], want, rtol=1e-13, atol=0) and np.all(np.isnan(inv[dim // 2:]))
    assert length == pytest.approx(want_length if dim else length, rel=1e-14)


def test_ramp_keeps_fast_pairs_and_slows_the_slow_ones():
    _, plain, _ = _rotary(rotary_base=1e6)
    _, ramp, _ = _rotary(rotary_base=1e6, rotary_scaling=2, rotary_factor=4.0, rotary_context=32768)
    turns = 32768 * plain / (2 * math.pi)
    ratio = ramp / plain
    assert np.allclose(ratio[turns > 40], 1.0, rtol=1e-12) and np.allclose(ratio[turns < 0.5], 0.25, rtol=1e-12)
    assert np.all(np.diff(ratio) <= 1e-12)


@pytest.mark.parametrize("change,code", [
    (dict(n_q_heads=15), 2), (dict(n_q_heads=0), 1), (dict(n_kv_heads=0), 1), (dict(n_q_heads=65, n_kv_heads=1), 2),
    (dict(head_dim=96), 2), (dict(head_dim=256), 2), (dict(page_size=8), 2), (dict(page_size=48), 2),
    (dict(page_size=512), 2), (dict(dtype=2), 2), (dict(rotary_dim=24), 2), (dict(rotary_dim=144), 2),
    (dict(rotary_dim=-16), 2), (dict(rotary_scaling=3), 2), (dict(rotary_base=1.0), 1),
    (dict(rotary_base=math.inf), 1), (dict(rotary_base=math.nan), 1), (dict(rotary_scaling=1, rotary_factor=0.5), 1),
    (dict(rotary_scaling=2, rotary_factor=2.0, rotary_context=0), 1), (dict(softmax_scale=-1.0), 1),
    (dict(softmax_scale=math.nan), 1), (dict(softmax_scale=1e39), 1), (dict(softmax_scale=3e38), 1),
    (dict(softmax_scale=1e-46), 1)])
def test_bad_configurations_are_refused(change, code):
    assert _rotary(**change)[0] == code
    c = lm._CacheConfig(**{**CONFIG, **change})
    h = ctypes.c_void_p()
    assert lm._lib.logmel_cache_plan_create(ctypes.addressof(c), ctypes.byref(h)) == code and not h.value


def test_null_arguments_are_refused():
    h = ctypes.c_void_p()
    assert lm._lib.logmel_cache_plan_create(None, ctypes.byref(h)) == 1
    assert lm._lib.logmel_cache_rotary(None, None, None) == 1
    assert lm._lib.logmel_cache_append(None, None, None, None, None, None, None, None, None) == 1
    assert lm._lib.logmel_cache_attend(None, None, None, None, None, None, 1, 0, None) == 1
    assert lm._lib.logmel_cache_weigh(None, None, None, None, None, 1, 0, 1.0, None, None) == 1
    assert lm._lib.logmel_cache_evict(None, None, None, 1, 0, None, None) == 1
    assert lm._lib.logmel_cache_plan_set_wait_test(None, 0) == 1
    lm._lib.logmel_cache_plan_destroy(None)


def test_binding_refuses_before_cuda():
    with pytest.raises(TypeError):
        lm.CachePlan(16, 8, 128, dtype=torch.float32)
    with pytest.raises(ValueError):
        lm.CachePlan(16, 8, 128, rotary_scaling="other")
    with pytest.raises(ValueError):
        lm.CachePlan(16, 8, 128, softmax_scale=0.0)
    with pytest.raises(lm.LogMelError) as e:
        lm.CachePlan(16, 8, 96)
    assert e.value.code == 2
    with pytest.raises(lm.LogMelError) as e:
        lm.CachePlan(16, 8, 128, rotary_dim=1000)
    assert e.value.code == 2
    with pytest.raises(lm.LogMelError) as e:   # a C int would hold 128
        lm.CachePlan(16, 8, 128, rotary_dim=128 - (1 << 32))
    assert e.value.code == 2


# --- the oracle ------------------------------------------------------------


def test_oracle_turn_is_a_rotation_by_relative_position():
    """Scores of turned rows depend on the distance of positions alone; lengths are kept."""
    r = np.random.default_rng(0)
    freq, _ = CO.rotary(16, 10000.0)
    q, k = r.standard_normal((1, 1, 24)), r.standard_normal((1, 1, 24))
    for inter in (False, True):
        def score(a, b):
            return float((CO.turn(q, np.array([a]), freq, 1.0, inter) * CO.turn(k, np.array([b]), freq, 1.0, inter)).sum())
        assert score(105, 100) == pytest.approx(score(7, 2), abs=1e-9)
        y = CO.turn(q, np.array([12345]), freq, 1.0, inter)
        assert np.linalg.norm(y) == pytest.approx(np.linalg.norm(q), rel=1e-12)
        assert np.array_equal(y[..., 16:], q[..., 16:])
        assert not np.allclose(y[..., :16], q[..., :16])


def test_oracle_seen_by_hand():
    assert CO.seen(5, 2, 0, True, 0) == [0, 1, 2, 3]
    assert CO.seen(5, 2, 1, True, 0) == [0, 1, 2, 3, 4]
    assert CO.seen(5, 2, 0, True, 2) == [2, 3]
    assert CO.seen(5, 2, 0, False, 0) == [0, 1, 2, 3, 4]
    assert CO.seen(5, 2, 0, False, 2) == [2, 3, 4]
    assert CO.seen(1, 3, 0, True, 0) == [] and CO.seen(1, 3, 2, True, 0) == [0]
    assert CO.seen(0, 1, 0, True, 0) == []


def test_oracle_attend_and_weigh_against_torch():
    torch.manual_seed(0)
    q, k, v = torch.randn(3, 4, 8).double(), torch.randn(2, 2, 4, 8).double(), torch.randn(2, 2, 4, 8).double()
    table, lens, off = np.array([[1, 0]]), np.array([7]), np.array([0, 3])
    out, lse, spread, _ = CO.attend(q.numpy(), k.numpy(), v.numpy(), table, lens, off, 0.3)
    kk = torch.cat([k[1], k[0]], 1)[:, :7].repeat_interleave(2, 0)
    vv = torch.cat([v[1], v[0]], 1)[:, :7].repeat_interleave(2, 0)
    mask = torch.ones(3, 7, dtype=torch.bool).tril(4)
    x = (q.transpose(0, 1) @ kk.transpose(1, 2) * 0.3).masked_fill(~mask, -math.inf)
    w = x.softmax(-1)
    assert np.allclose(out, (w @ vv).transpose(0, 1).numpy()) and np.allclose(lse, x.logsumexp(-1).t().numpy())
    assert np.all(spread >= np.abs(out) - 1e-12)
    mass = np.ones((2, 2, 4))
    m, added, terms = CO.weigh(q.numpy(), lse, k.numpy(), mass, table, lens, off, 0.3, decay=0.5)
    total = w.view(2, 2, 3, 7).sum((1, 2)).numpy()
    assert np.allclose(added[1], total[:, :4]) and np.allclose(added[0][:, :3], total[:, 4:])
    assert m[0, 0, 3] == 1.0 and np.allclose(m[1], 0.5 + added[1])        # slot 7 is not live
    assert added.sum() == pytest.approx(3 * 4)                            # every row hands out a weight of one


def test_oracle_evict_by_hand():
    mass = np.array([[[5, 1, 5, 0]], [[2, 9, 7, 8]]], np.float32)          # pages [2, 1 head, 4 slots]
    table = np.array([[1, 0]])                                            # slots: 2 9 7 8 | 5 1 5 0
    assert CO.evict(mass, table, [8], 4, 4, 1) == [[[1, 2, 3, 7]]]
    assert CO.evict(mass, table, [8], 4, 5, 0) == [[[1, 2, 3, 4, 6]]]
    assert CO.evict(mass, table, [8], 4, 4, 0) == [[[1, 2, 3, 4]]]         # the tie of slots 4 and 6 goes to 4
    assert CO.evict(mass, table, [3], 4, 5, 1) == [[[0, 1, 2]]]
    assert CO.evict(mass, table, [8], 4, 3, 3) == [[[5, 6, 7]]]
    assert CO.evict(mass, table, [0], 4, 3, 3) == [[[]]]
