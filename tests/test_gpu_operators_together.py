"""Rotated append, scored attention and shared-prefix attention as a decoder uses
them: together, on streams of their own, captured, with many sequences, and
with a stalled copy.

Rows in the caches are checked with test_gpu_rope's bound, outputs against fp64
attention over the rows that the caches then hold (attn_reference's bound).
"""
import ctypes

import numpy as np
import pytest
import torch

import kv_cache_decode_append_gb300 as kvd
import kv_cache_decode_append_gb300.build as kbuild
import kv_cache_decode_append_gb300.kvd as binding
from attn_reference import DT, assert_near, attention64, seen_mask
from helpers import to_np
from test_gpu_rope import _cos_sin, _near, _rotate

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(900)]

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def _bits(t):
    return to_np(t).view(np.uint8)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rotated_decode_with_window_sinks_and_cap(dtype):
    """A prompt chunk, then captured single-token steps, over a paged cache: rotated append and scored
    attention read the lengths that the graph itself advances."""
    B, H_q, H_kv, D, page, T = 3, 8, 2, 64, 64, 320
    window, sinks, cap = 100, 4, 15.0
    g = torch.Generator("cpu").manual_seed(11)
    rows = lambda *s: torch.randn(s, generator=g).to(DT[dtype]).to(DEV)
    table = torch.randperm(B * T // page + 1, generator=g)[:B * T // page].to(torch.int32).view(B, -1).to(DEV)
    kp, vp = (torch.full((B * T // page + 1, H_kv, page, D), float("nan"), dtype=DT[dtype], device=DEV) for _ in range(2))
    freq = [10000.0 ** (-f / 32) for f in range(32)]
    freq_d = torch.tensor(freq, dtype=torch.float64, device=DEV)
    lens, err = _i32([0, 0, 0]), _i32([0])
    sink_d = _i32([sinks] * B)
    ws = kvd.alloc_scored_workspace(B, H_q, H_kv, D, 150, T - 150, DT[dtype])  # (both shapes in turn)

    def step(x, q_out, out, max_past):
        q, k, v = x.transpose(1, 2).split([H_q, H_kv, H_kv], dim=1)
        kvd.kvd_paged_rope_append(q, q_out, kp, vp, k, v, table, lens, max_past, freq_d, err_word=err)
        kvd.kvd_paged_decode_attention_scored(q_out, kp, vp, out, table, lens, max_past, softcap=cap, window=window,
                                              prefix_len=sink_d, workspace=ws, err_word=err)

    def check(x, q_out, out, P):
        N = x.shape[1]
        q, k, v = x.transpose(1, 2).split([H_q, H_kv, H_kv], dim=1)
        cos, sin = _cos_sin(range(P, P + N), freq)
        n = P + N
        for b in range(B):
            _near(_f64(q_out[b]), *_rotate(_f64(q[b]), cos, sin, D, False), dtype)
            kc, vc = (p[table[b].long()].transpose(0, 1).reshape(H_kv, T, D)[:, :n] for p in (kp, vp))
            _near(_f64(kc[:, P:]), *_rotate(_f64(k[b]), cos, sin, D, False), dtype)
            assert np.array_equal(_bits(vc[:, P:].contiguous()), _bits(v[b].contiguous()))
            ref, tol = attention64(_f64(q_out[b]), _f64(kc), _f64(vc), D ** -0.5, seen_mask(P, N, window, sinks, None),
                                   cap, None, P, dtype)
            assert_near(_f64(out[b]), ref, tol, f"sequence {b} at {P}")

    N = 150
    x, q_out = rows(B, N, H_q + 2 * H_kv, D), torch.empty(B, H_q, N, D, dtype=DT[dtype], device=DEV)
    out = torch.empty_like(q_out)
    step(x, q_out, out, 0)
    torch.cuda.synchronize()
    check(x, q_out, out, 0)

    lens += N
    x, q_out = rows(B, 1, H_q + 2 * H_kv, D), torch.empty(B, H_q, 1, D, dtype=DT[dtype], device=DEV)
    out = torch.empty_like(q_out)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(x, q_out, out, T - 1)
        lens += 1
    for i in range(4):
        x.copy_(rows(*x.shape))
        graph.replay()
        torch.cuda.synchronize()
        check(x, q_out, out, N + i)
    assert int(err) == 0 and lens.tolist() == [N + 4] * B


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rotated_decode_behind_a_shared_prefix(dtype):
    """The prefix rotated and cached once, as a batch of one; the sequences' positions go on behind it."""
    B, H_q, H_kv, D, S, T = 9, 8, 2, 128, 517, 40
    g = torch.Generator("cpu").manual_seed(12)
    rows = lambda *s: torch.randn(s, generator=g).to(DT[dtype]).to(DEV)
    freq = [500000.0 ** (-f / 64) for f in range(64)]
    freq_d = torch.tensor(freq, dtype=torch.float64, device=DEV)
    k_pre, v_pre = (torch.full((1, H_kv, S, D), float("nan"), dtype=DT[dtype], device=DEV) for _ in range(2))
    q, k, v = rows(1, H_q, S, D), rows(1, H_kv, S, D), rows(1, H_kv, S, D)
    kvd.kvd_rope_append(q, torch.empty_like(q), k_pre, v_pre, k, v, _i32([0]), 0, freq_d, interleaved=True)
    kc, vc = (torch.full((B, H_kv, T, D), float("nan"), dtype=DT[dtype], device=DEV) for _ in range(2))
    lens, past, err = _i32([0] * B), 0, _i32([0])
    ws = kvd.alloc_shared_prefix_workspace(B, H_q, H_kv, D, 5, S, T - 5, DT[dtype])
    for N in (5, 1, 1):
        q, k, v = rows(B, H_q, N, D), rows(B, H_kv, N, D), rows(B, H_kv, N, D)
        q_out, out = torch.empty_like(q), torch.full_like(q, float("nan"))
        kvd.kvd_rope_append(q, q_out, kc, vc, k, v, lens, past, freq_d, interleaved=True, pos_base=S, err_word=err)
        kvd.kvd_shared_prefix_attention(q_out, k_pre[0], v_pre[0], S, kc, vc, out, lens, past, workspace=ws, err_word=err)
        torch.cuda.synchronize()
        cos, sin = _cos_sin(range(S + past, S + past + N), freq)
        for b in range(B):
            _near(_f64(q_out[b]), *_rotate(_f64(q[b]), cos, sin, D, True), dtype)
            _near(_f64(kc[b, :, past:past + N]), *_rotate(_f64(k[b]), cos, sin, D, True), dtype)
            kk, vv = (torch.cat([p[0], c[b, :, :past + N]], dim=1) for p, c in ((k_pre, kc), (v_pre, vc)))
            ref, tol = attention64(_f64(q_out[b]), _f64(kk), _f64(vv), D ** -0.5,
                                   seen_mask(S + past, N, 0, 0, None), dtype=dtype)
            assert_near(_f64(out[b]), ref, tol, f"sequence {b} at {past}")
        lens += N
        past += N
    assert int(err) == 0


def test_calls_at_once():
    """Three streams, a workspace each, nothing waited for in between: the same bits as alone."""
    g = torch.Generator("cpu").manual_seed(13)
    rows = lambda *s: torch.randn(s, generator=g).bfloat16().to(DEV)
    B, H_q, H_kv, D, S, T = 4, 16, 2, 128, 900, 700
    k, v, kp, vp = rows(B, H_kv, T, D), rows(B, H_kv, T, D), rows(H_kv, S, D), rows(H_kv, S, D)
    q1, q4 = rows(B, H_q, 1, D), rows(B, H_q, 4, D)
    past = _i32([600, 3, 0, 77])
    w = [kvd.alloc_scored_workspace(B, H_q, H_kv, D, n, 600, torch.bfloat16) for n in (1, 4)]
    w.append(kvd.alloc_shared_prefix_workspace(B, H_q, H_kv, D, 4, S, 600, torch.bfloat16))
    streams = [torch.cuda.Stream() for _ in range(3)]

    def calls(i, out, stream):
        if i < 2:
            kvd.kvd_decode_attention_scored((q1, q4)[i], k, v, out, past, 600, softcap=20.0, window=300,
                                            workspace=w[i], stream=stream)
        else:
            kvd.kvd_shared_prefix_attention(q4, kp, vp, S, k, v, out, past, 600, workspace=w[2], stream=stream)

    want = [torch.empty_like(x) for x in (q1, q4, q4)]
    for i in range(3):
        calls(i, want[i], streams[0])
        streams[0].synchronize()
    outs = [[torch.full_like(x, float("nan")) for x in want] for _ in range(8)]
    torch.cuda.synchronize()
    for out in outs:
        for i in range(3):
            calls(i, out[i], streams[i])
    torch.cuda.synchronize()
    for out in outs:
        for a, b in zip(out, want):
            assert np.array_equal(_bits(a), _bits(b))


@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "bf16"), (128, "f32")])
def test_many_sequences(D, dtype):
    """2048 sequences of many rows, 16384 of one row (fp32: 2048); what is too many is refused before a launch."""
    g = torch.Generator("cpu").manual_seed(14)
    for B, H_q in ((2048, 17), (16384 if dtype != "f32" else 2048, 2)):
        rows = lambda *s: torch.randn(s, generator=g).to(DT[dtype])
        q, k, v = rows(B, H_q, 1, D), rows(B, 1, 70, D), rows(B, 1, 70, D)
        past = [(7 * b) % 69 for b in range(B)]
        kd, vd, qd, out = k.to(DEV), v.to(DEV), q.to(DEV), torch.full_like(q, float("nan"), device=DEV)
        err = _i32([0])
        kvd.kvd_decode_attention_scored(qd, kd, vd, out, _i32(past), 69, softcap=8.0, err_word=err,
                                        workspace=kvd.alloc_scored_workspace(B, H_q, 1, D, 1, 69, DT[dtype]))
        two = torch.full_like(out, float("nan"))
        kvd.kvd_shared_prefix_attention(qd, kd[0], vd[0], 70, kd, vd, two, _i32(past), 69, err_word=err,
                                        workspace=kvd.alloc_shared_prefix_workspace(B, H_q, 1, D, 1, 70, 69, DT[dtype]))
        torch.cuda.synchronize()
        assert int(err) == 0
        for b in (0, 1, 9, 10, B // 2, B - 1):
            n = past[b] + 1
            args = (_f64(q[b]), _f64(k[b, :, :n]), _f64(v[b, :, :n]), D ** -0.5)
            assert_near(_f64(out[b]), *attention64(*args, np.ones((1, n), bool), 8.0, dtype=dtype), f"sequence {b}")
            kk, vv = (_f64(torch.cat([x[0], x[b, :, :n]], dim=1)) for x in (k, v))
            assert_near(_f64(two[b]), *attention64(args[0], kk, vv, D ** -0.5, np.ones((1, 70 + n), bool), dtype=dtype),
                        f"sequence {b} and prefix")
    B, H_q = 20000, 17
    assert kvd.alloc_scored_workspace(B, H_q, 1, D, 1, 0, DT[dtype]) is None
    x, y = (torch.zeros(B, h, 1, D, dtype=DT[dtype], device=DEV) for h in (H_q, 1))
    with pytest.raises(kvd.KvdError) as e:
        kvd.kvd_decode_attention_scored(x, y, y, x.clone(), _i32([0] * B), 0, workspace=torch.zeros(1 << 20, dtype=torch.uint8, device=DEV))
    assert e.value.status == kvd.KVD_ERR_UNSUPPORTED


# ---- a copy that never completes (test builds of the library) ----
@pytest.fixture(scope="module")
def tlib():
    lib = binding._Lib(kbuild.build(extra_flags=["-DKVD_TIMEOUT_TEST"], variant="timeout_test"))
    lib.kvd_test_inject_stall.restype = None
    lib.kvd_test_inject_stall.argtypes = [ctypes.c_int]
    return lib


STALLS = [  # H_q, H_kv, D, N, past, prefix length (None: scored attention), dtype
    ("scored_tcgen05", 8, 2, 128, 5, [700, 130], None, "bf16"),
    ("scored_f32", 8, 8, 128, 1, [4000, 3100], None, "f32"),
    ("prefix_tcgen05", 8, 2, 128, 1, [60, 130], 900, "bf16"),
    ("prefix_tcgen05_both", 8, 2, 64, 5, [600, 130], 900, "f16"),
    ("prefix_own_f32", 4, 4, 64, 1, [3000, 1], 300, "f32"),
]


@pytest.mark.parametrize("case", STALLS, ids=[c[0] for c in STALLS])
def test_stall_is_flagged_and_the_next_call_is_exact(tlib, case):
    """The workspace holds leftovers of anything outside the zeroed part: what a call that gave up did not
    write is not taken for a place to read."""
    _, H_q, H_kv, D, N, past, S, dtype = case
    B, T, code = len(past), max(past) + N, {"f32": kvd.KVD_F32, "bf16": kvd.KVD_BF16, "f16": kvd.KVD_F16}[dtype]
    g = torch.Generator("cpu").manual_seed(15)
    rows = lambda *s: torch.randn(s, generator=g).to(DT[dtype]).to(DEV)
    q, k, v = rows(B, H_q, N, D), rows(B, H_kv, T, D), rows(B, H_kv, T, D)
    past_d, err, out = _i32(past), _i32([0]), torch.full((B, H_q, N, D), float("nan"), dtype=DT[dtype], device=DEV)
    stream = torch.cuda.current_stream().cuda_stream
    if S is None:
        size = tlib.kvd_decode_scored_workspace_bytes(B, H_q, H_kv, D, N, max(past), code)
        score = binding.Score(12.0, None, 0, None, None)
    else:
        size = tlib.kvd_shared_prefix_workspace_bytes(B, H_q, H_kv, D, N, S, max(past), code)
        kp, vp = rows(H_kv, S, D), rows(H_kv, S, D)
    ws = torch.randint(0, 256, (size,), dtype=torch.uint8, device=DEV)

    def call():
        if S is None:
            ws[:min(size, 256 * 1024)] = 0
            return tlib.kvd_decode_attention_scored(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                                    past_d.data_ptr(), ctypes.byref(score), B, H_q, H_kv, T, D, N,
                                                    max(past), 0.0, code, ws.data_ptr(), size, err.data_ptr(), stream)
        return tlib.kvd_shared_prefix_attention(q.data_ptr(), kp.data_ptr(), vp.data_ptr(), k.data_ptr(), v.data_ptr(),
                                                out.data_ptr(), past_d.data_ptr(), B, H_q, H_kv, S, T, D, N, S,
                                                max(past), 0.0, code, ws.data_ptr(), size, err.data_ptr(), stream)

    tlib.kvd_test_inject_stall(1)
    try:
        assert call() == kvd.KVD_OK
        torch.cuda.synchronize()
    finally:
        tlib.kvd_test_inject_stall(0)
    assert int(err) & kvd.KVD_DEVERR_TIMEOUT
    err.zero_()
    out.fill_(float("nan"))
    assert call() == kvd.KVD_OK
    torch.cuda.synchronize()
    assert int(err) == 0
    for b, P in enumerate(past):
        kk, vv, mask = k[b, :, :P + N], v[b, :, :P + N], seen_mask(P, N, 0, 0, None)
        if S is not None:
            kk, vv = torch.cat([kp, kk], dim=1), torch.cat([vp, vv], dim=1)
            mask = np.concatenate([np.ones((N, S), bool), mask], axis=1)
        ref, tol = attention64(_f64(q[b]), _f64(kk), _f64(vv), D ** -0.5, mask, 12.0 if S is None else 0.0, dtype=dtype)
        assert_near(_f64(out[b]), ref, tol, f"sequence {b}")
