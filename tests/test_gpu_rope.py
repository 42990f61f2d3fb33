"""Rotated append on the GPU: kvd_rope_append / kvd_paged_rope_append.

The reference takes each angle exactly (a frequency is a rational number, the
phase of position times frequency is reduced in integers against 1 / (2 pi) to
256 bits) and rotates in fp64.

Tolerance per element of the pair (x, y) with exact result r: cos and sin are
off by at most 2^-23 (the phase to fp32: pi/4 2^-24; sinpif / cospif: one unit
in the last place, at most 2^-24), so x cos and y sin by 2^-23 (|x| + |y|); the
product's and the sum's fp32 roundings add 2^-24 (|y| + |r|) <= 2^-23 (|x| + |y|);
together at most 2^-22 (|x| + |y|).  Rounding to the cache's type adds half a
step: eps / 2 |r| (and half the smallest fp16 step, 2^-25).
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

import kv_cache_decode_append_gb300 as kvd
from helpers import to_np

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# 1 / (2 pi) to 256 bits and more
_PI = Fraction(314159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798,
               10 ** 101)
_INV_2PI = Fraction(int(2 ** 300 / (2 * _PI)), 2 ** 300)


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def _cos_sin(positions, inv_freq):
    """cos and sin of every position (list of int) times every frequency, through the exact phase."""
    turns = [Fraction(f) * _INV_2PI for f in inv_freq]
    phase = np.array([[float((t * p) % 1) for t in turns] for p in positions])
    phase = np.where(phase > 0.5, phase - 1.0, phase)
    return np.cos(2 * np.pi * phase), np.sin(2 * np.pi * phase)


def _rotate(x, cos, sin, rot, interleaved):
    """Rows [H, N, D] (fp64) with cos, sin [N, rot / 2]; also |x| + |y| of every element's pair."""
    y, size = x.copy(), np.zeros_like(x)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, size


def _near(got, ref, size, dtype):
    step = 0.0 if dtype == "f32" else torch.finfo(DT[dtype]).eps / 2
    tol = 2.0 ** -22 * size + step * np.abs(ref) * (1 + 2.0 ** -20) + (2.0 ** -25 if dtype == "f16" else 0.0)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.abs(got - ref)[bad].max(), np.argwhere(bad)[:3])


def _bits(t):
    return to_np(t).view(np.uint8)


def _inputs(B, H_q, H_kv, D, N, T, dtype, fused, seed, page=0):
    g = torch.Generator("cpu").manual_seed(seed)
    rows = lambda *s: torch.randn(s, generator=g).to(DT[dtype]).to(DEV)
    if fused:
        qkv = rows(B, N, H_q + 2 * H_kv, D).transpose(1, 2)
        q, k, v = qkv[:, :H_q], qkv[:, H_q:H_q + H_kv], qkv[:, H_q + H_kv:]
    else:
        q, k, v = rows(B, H_q, N, D), rows(B, H_kv, N, D), rows(B, H_kv, N, D)
    if not page:
        return q, k, v, rows(B, H_kv, T, D), rows(B, H_kv, T, D), None
    n = -(-T // page)
    table = torch.randperm(B * n + 2, generator=g)[:B * n].to(torch.int32).view(B, n).to(DEV)
    return q, k, v, rows(B * n + 2, H_kv, page, D), rows(B * n + 2, H_kv, page, D), table


def _call(q, q_out, kc, vc, k, v, table, past, max_past, freq, **more):
    if table is None:
        kvd.kvd_rope_append(q, q_out, kc, vc, k, v, past, max_past, freq, **more)
    else:
        kvd.kvd_paged_rope_append(q, q_out, kc, vc, k, v, table, past, max_past, freq, **more)


def _slot(table, page, b, t):
    return (b, slice(None), t) if table is None else (int(table[b, t // page]), slice(None), t % page)


def _check(q, q_out, kc0, vc0, kc, vc, k, v, table, page, past, pos, freq, rot, interleaved, dtype, skip=()):
    """q_out and the caches after the call against the reference; every other slot unchanged."""
    N = q.shape[2]
    want_v, touched = vc0.clone(), torch.zeros(kc.shape[:3], dtype=torch.bool)
    for b, P in enumerate(past):
        if b in skip:
            continue
        cos, sin = _cos_sin(pos[b], freq)
        ref, size = _rotate(q[b].double().cpu().numpy(), cos, sin, rot, interleaved)
        _near(q_out[b].double().cpu().numpy(), ref, size, dtype)
        assert np.array_equal(_bits(q_out[b][..., rot:]), _bits(q[b][..., rot:]))
        ref, size = _rotate(k[b].double().cpu().numpy(), cos, sin, rot, interleaved)
        for i in range(N):
            at = _slot(table, page, b, P + i)
            _near(kc[at].double().cpu().numpy(), ref[:, i], size[:, i], dtype)
            assert np.array_equal(_bits(kc[at][..., rot:]), _bits(k[b, :, i, rot:]))
            want_v[at] = v[b, :, i]
            touched[at] = True
    assert np.array_equal(_bits(vc), _bits(want_v))
    rest = ~touched.to(DEV)
    assert np.array_equal(_bits(kc[rest]), _bits(kc0[rest]))


CASES = [  # B, H_q, H_kv, D, N, T, past, dtype, rot, interleaved, page, fused
    (1, 12, 12, 64, 1, 64, [63], "f32", 64, False, 0, False),
    (1, 1, 1, 64, 1, 1, [0], "bf16", 64, False, 0, False),
    (3, 8, 2, 128, 1, 200, [0, 199, 64], "bf16", 128, False, 64, False),
    (2, 6, 2, 64, 5, 200, [62, 195], "f16", 32, False, 64, True),
    (2, 6, 2, 64, 5, 200, [62, 195], "f16", 16, True, 128, True),
    (2, 4, 4, 128, 33, 300, [100, 0], "f32", 32, True, 0, True),
    (2, 4, 1, 128, 7, 100, [93, 1], "bf16", 64, True, 0, False),
    (40, 3, 1, 64, 4, 70, list(range(40)), "f16", 64, False, 0, True),
    (2, 2, 1, 256, 3, 10, [7, 0], "bf16", 256, False, 0, False),
    (1, 2, 2, 8, 3, 10, [7], "f32", 8, False, 0, False),
]


@pytest.mark.parametrize("case", CASES, ids=[f"rope{i}" for i in range(len(CASES))])
def test_parity(case):
    B, H_q, H_kv, D, N, T, past, dtype, rot, interleaved, page, fused = case
    q, k, v, kc0, vc0, table = _inputs(B, H_q, H_kv, D, N, T, dtype, fused, 500 + D + N + rot, page)
    freq = [10000.0 ** (-2 * f / rot) for f in range(rot // 2)]
    kc, vc, q_out = kc0.clone(), vc0.clone(), torch.full((B, H_q, N, D), float("nan"), dtype=DT[dtype], device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    _call(q, q_out, kc, vc, k, v, table, torch.tensor(past, dtype=torch.int32, device=DEV), max(past),
          torch.tensor(freq, dtype=torch.float64, device=DEV), interleaved=interleaved, err_word=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    pos = [[P + i for i in range(N)] for P in past]
    _check(q, q_out, kc0, vc0, kc, vc, k, v, table, page, past, pos, freq, rot, interleaved, dtype)


@pytest.mark.parametrize("pos_base,positions", [(1 << 20, None), ((1 << 31) - 1, None), (-5, None),
                                                (0, [[0, 2147483647, -2147483648], [7, 7, 100001]]),
                                                (-(1 << 31), [[5, -1, 0], [2147483647, 1, -9]])])
@pytest.mark.parametrize("freqs", ["usual", "odd"])
def test_far_positions(pos_base, positions, freqs):
    """Angles are exact at any position, for frequencies of any size and sign."""
    B, H_q, H_kv, D, N, rot = 2, 2, 1, 64, 3, 32
    q, k, v, kc0, vc0, _ = _inputs(B, H_q, H_kv, D, N, 16, "f32", False, 77)
    freq = [500000.0 ** (-2 * f / rot) for f in range(rot // 2)]
    if freqs == "odd":
        freq[:8] = [0.0, -0.3, 6.5, 1e-30, 123456.789, np.pi, 2.0 ** -60, -1e9]
    past = [4, 9]
    kc, vc, q_out = kc0.clone(), vc0.clone(), torch.empty_like(q)
    more = {} if positions is None else {"positions": torch.tensor(positions, dtype=torch.int32, device=DEV)}
    kvd.kvd_rope_append(q, q_out, kc, vc, k, v, torch.tensor(past, dtype=torch.int32, device=DEV), 9,
                        torch.tensor(freq, dtype=torch.float64, device=DEV), pos_base=pos_base, **more)
    torch.cuda.synchronize()
    pos = [[pos_base + (positions[b][i] if positions else P + i) for i in range(N)] for b, P in enumerate(past)]
    _check(q, q_out, kc0, vc0, kc, vc, k, v, None, 0, past, pos, freq, rot, False, "f32")


def test_q_in_place_and_side_stream_and_graph():
    """q_out may be q; the call follows its stream and can be captured and replayed."""
    B, H_q, H_kv, D, N = 3, 8, 2, 64, 2
    q, k, v, kc0, vc0, _ = _inputs(B, H_q, H_kv, D, N, 40, "bf16", False, 5)
    past = torch.tensor([0, 17, 38], dtype=torch.int32, device=DEV)
    freq = torch.tensor([10000.0 ** (-f / 32) for f in range(32)], dtype=torch.float64, device=DEV)
    kc, vc, out = kc0.clone(), vc0.clone(), torch.empty_like(q)
    kvd.kvd_rope_append(q, out, kc, vc, k, v, past, 38, freq)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    q2, kc2, vc2 = q.clone(), kc0.clone(), vc0.clone()
    torch.cuda.synchronize()
    kvd.kvd_rope_append(q2, q2, kc2, vc2, k, v, past, 38, freq, stream=side)
    side.synchronize()
    assert np.array_equal(_bits(q2), _bits(out)) and np.array_equal(_bits(kc2), _bits(kc)) and np.array_equal(_bits(vc2), _bits(vc))
    out3, kc3, vc3 = torch.zeros_like(q), kc0.clone(), vc0.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvd.kvd_rope_append(q, out3, kc3, vc3, k, v, past, 38, freq)
    for _ in range(2):
        out3.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(_bits(out3), _bits(out)) and np.array_equal(_bits(kc3), _bits(kc)) and np.array_equal(_bits(vc3), _bits(vc))


def test_bad_past_len_and_bad_page_write_nothing():
    B, H_q, H_kv, D, N, page = 4, 4, 2, 64, 3, 64
    q, k, v, kc0, vc0, table = _inputs(B, H_q, H_kv, D, N, 128, "bf16", False, 9, page)
    freq = [10000.0 ** (-f / 32) for f in range(32)]
    past = [62, -1, 126, 70]          # the second and third are out of range
    table[3, 1] = kc0.shape[0]        # a page outside the pool, for the fourth
    fill = torch.full_like(q, 3.0)
    kc, vc, q_out = kc0.clone(), vc0.clone(), fill.clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    kvd.kvd_paged_rope_append(q, q_out, kc, vc, k, v, table, torch.tensor(past, dtype=torch.int32, device=DEV), 125,
                              torch.tensor(freq, dtype=torch.float64, device=DEV), err_word=err)
    torch.cuda.synchronize()
    assert int(err) == kvd.KVD_DEVERR_PAST_LEN | kvd.KVD_DEVERR_PAGE
    assert np.array_equal(_bits(q_out[1:3]), _bits(fill[1:3]))
    pos = [[P + i for i in range(N)] for P in past]
    _check(q, q_out, kc0, vc0, kc, vc, k, v, table, page, past, pos, freq, 64, False, "bf16", skip=(1, 2, 3))
    cos, sin = _cos_sin(pos[3], freq)
    ref, size = _rotate(q[3].double().cpu().numpy(), cos, sin, 64, False)
    _near(q_out[3].double().cpu().numpy(), ref, size, "bf16")


def test_binding_refuses():
    q, k, v, kc, vc, _ = _inputs(2, 4, 2, 64, 3, 16, "bf16", True, 3)
    past = torch.zeros(2, dtype=torch.int32, device=DEV)
    freq = torch.ones(32, dtype=torch.float64, device=DEV)
    out = torch.empty(2, 4, 3, 64, dtype=torch.bfloat16, device=DEV)
    ok = dict(q=q, q_out=out, k_cache=kc, v_cache=vc, k_new=k, v_new=v, past_len=past, max_past_len=0, inv_freq=freq)
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(inv_freq=freq.float()), dict(q_out=out.transpose(1, 2)),
                dict(k_new=k[:, :1]), dict(past_len=past[:1]), dict(q=q.transpose(2, 3)), dict(pos_base=1 << 31),
                dict(positions=past), dict(k_cache=kc[:1], v_cache=vc[:1])):
        with pytest.raises(ValueError):
            kvd.kvd_rope_append(**{**ok, **bad})
    with pytest.raises(kvd.KvdError) as e:
        kvd.kvd_rope_append(**{**ok, "max_past_len": 14})
    assert e.value.status == kvd.KVD_ERR_CAPACITY
