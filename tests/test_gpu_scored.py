"""Attention with modified scores on the GPU (kvd_decode_attention_scored and
kvd_paged_decode_attention_scored) against fp64, with the bound of
attn_reference.  Every slot that no row sees holds NaN, and pages of such slots
alone have no valid block-table entry.
"""
import numpy as np
import pytest
import torch

import kv_cache_decode_append_gb300 as kvd
from attn_reference import DT, assert_near, attention64, seen_mask
from helpers import to_np

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def _bits(t):
    return to_np(t).view(np.uint8)


class Case:
    """Inputs of one call; contiguous and paged caches over the same rows."""

    def __init__(self, B, H_q, H_kv, D, N, past, dtype, cap=0.0, slopes=False, window=0, prefix=None, docs=None,
                 page=64, seed=0, T_extra=3):
        self.__dict__.update(B=B, H_q=H_q, H_kv=H_kv, D=D, N=N, past=past, dtype=dtype, cap=cap, window=window,
                             prefix=prefix, docs=docs, page=page, dt=DT[dtype])
        g = torch.Generator("cpu").manual_seed(1000 + seed)
        T = max(past) + N + T_extra
        rnd = lambda *s: torch.randn(s, generator=g).to(self.dt)
        self.q = (rnd(B, H_q, N, D).float() * 2).to(self.dt)
        self.k, self.v = rnd(B, H_kv, T, D), rnd(B, H_kv, T, D)
        self.slopes = (2.0 ** -torch.arange(1, H_q + 1).float()) if slopes else None
        self.masks = [seen_mask(P, N, window, prefix[b] if prefix else 0, docs[b] if docs else None)
                      for b, P in enumerate(past)]
        for b, P in enumerate(past):  # what no row sees is NaN
            hidden = torch.ones(T, dtype=torch.bool)
            hidden[:P + N] = torch.from_numpy(~self.masks[b].any(0))
            self.k[b, :, hidden] = float("nan")
            self.v[b, :, hidden] = float("nan")
        n = -(-T // page)
        total = B * n + 2
        perm = torch.randperm(total, generator=g)[:B * n].to(torch.int32)
        self.table = perm.view(B, n).clone()
        self.kp = torch.full((total, H_kv, page, D), float("nan"), dtype=self.dt)
        self.vp = self.kp.clone()
        for b, P in enumerate(past):
            seen = np.zeros(n * page, bool)
            seen[:P + N] = self.masks[b].any(0)
            for j in range(n):
                rows = slice(j * page, min(T, (j + 1) * page))
                m = rows.stop - rows.start
                self.kp[self.table[b, j].item(), :, :m] = self.k[b, :, rows]
                self.vp[self.table[b, j].item(), :, :m] = self.v[b, :, rows]
            # entries of pages that lie wholly in tiles no row sees (64 keys: no larger than any tile)
            for j in range(n):
                lo, hi = j * page, (j + 1) * page
                if not seen[lo:hi].any() and seen.any():
                    self.table[b, j] = -1

    def more(self):
        m = {"softcap": self.cap, "window": self.window}
        if self.slopes is not None:
            m["slopes"] = self.slopes.to(DEV)
        if self.prefix is not None:
            m["prefix_len"] = torch.tensor(self.prefix, dtype=torch.int32, device=DEV)
        if self.docs is not None:
            m["doc_start"] = torch.tensor(self.docs, dtype=torch.int32, device=DEV)
        return m

    def workspace(self):
        return kvd.alloc_scored_workspace(self.B, self.H_q, self.H_kv, self.D, self.N, max(self.past), self.dt)

    def run(self, paged, stream=None, **over):
        out = torch.full(self.q.shape, float("nan"), dtype=self.dt, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        past = torch.tensor(self.past, dtype=torch.int32, device=DEV)
        more = {**self.more(), "workspace": self.workspace(), "err_word": err, "stream": stream, **over}
        q = self.q.to(DEV)
        torch.cuda.synchronize()
        if paged:
            kvd.kvd_paged_decode_attention_scored(q, self.kp.to(DEV), self.vp.to(DEV), out, self.table.to(DEV), past,
                                                  max(self.past), **more)
        else:
            kvd.kvd_decode_attention_scored(q, self.k.to(DEV), self.v.to(DEV), out, past, max(self.past), **more)
        torch.cuda.synchronize()
        return out, int(err)

    def check(self, out):
        q, k, v = (x.double().numpy() for x in (self.q, self.k, self.v))
        sl = None if self.slopes is None else self.slopes.double().numpy()
        got = out.double().cpu().numpy()
        for b, P in enumerate(self.past):
            n = P + self.N
            ref, tol = attention64(q[b], k[b, :, :n], v[b, :, :n], self.D ** -0.5, self.masks[b], self.cap, sl, P,
                                   self.dtype)
            assert_near(got[b], ref, tol, f"sequence {b}")


def _docs(past, N, at):
    """A document begun in the cache at `at[b]`, and another from the middle of the chunk on."""
    return [[a if i < max(1, N // 2) else P + N // 2 for i in range(N)] for P, a in zip(past, at)]


# rows per KV head (g N) and the type pick the kernel: fp32 the CUDA cores, 16-bit
# types the streaming kernel up to 16 rows, tcgen05 in pairs of blocks from 17 on
CASES = {
    # plain: the same call as kvd_decode_attention
    "plain": dict(B=2, H_q=4, H_kv=2, D=64, N=1, past=[100, 0], dtype="bf16"),
    "cap_f32": dict(B=2, H_q=4, H_kv=2, D=64, N=3, past=[130, 5], dtype="f32", cap=3.0),
    "slopes_f32": dict(B=1, H_q=3, H_kv=3, D=128, N=1, past=[300], dtype="f32", slopes=True),
    "window1": dict(B=2, H_q=4, H_kv=4, D=64, N=2, past=[77, 0], dtype="bf16", window=1),
    "window_one_row": dict(B=3, H_q=2, H_kv=2, D=64, N=1, past=[1000, 63, 64], dtype="f16", window=65),
    "window_f32_d128": dict(B=2, H_q=8, H_kv=2, D=128, N=2, past=[500, 33], dtype="f32", window=40, slopes=True),
    "sinks_mma": dict(B=3, H_q=8, H_kv=2, D=128, N=1, past=[700, 100, 3], dtype="bf16", window=64, prefix=[4, 4, 4], cap=5.0),
    "sinks_wide": dict(B=2, H_q=4, H_kv=1, D=128, N=2, past=[900, 400], dtype="f16", window=100, prefix=[200, 330]),
    "prefix_both_ways": dict(B=2, H_q=4, H_kv=2, D=64, N=6, past=[0, 40], dtype="f16", prefix=[4, 43]),
    "prefix_past_end": dict(B=2, H_q=4, H_kv=2, D=64, N=6, past=[10, 64], dtype="bf16", prefix=[1000, -3]),
    "docs_mma": dict(B=3, H_q=8, H_kv=1, D=64, N=2, past=[200, 64, 1], dtype="bf16", slopes=True,
                     docs=_docs([200, 64, 1], 2, [130, 64, 0])),
    "docs_window_prefix": dict(B=2, H_q=4, H_kv=2, D=128, N=8, past=[600, 130], dtype="f16", window=50,
                               prefix=[140, 70], docs=_docs([600, 130], 8, [70, 65]), cap=10.0, slopes=True),
    "empty_rows": dict(B=3, H_q=4, H_kv=2, D=64, N=3, past=[90, 200, 0], dtype="bf16",
                       docs=[[95, 95, 95], [0, 300, 202], [0, 2, 2]]),
    "empty_rows_f32": dict(B=2, H_q=2, H_kv=2, D=64, N=2, past=[90, 500], dtype="f32", docs=[[95, 95], [501, 501]]),
    "empty_rows_tc5": dict(B=2, H_q=16, H_kv=2, D=64, N=4, past=[90, 200], dtype="f16", docs=[[95] * 4, [0, 300, 203, 203]]),
    "tc5_cap": dict(B=2, H_q=8, H_kv=2, D=128, N=16, past=[333, 0], dtype="bf16", cap=4.0),
    "tc5_all": dict(B=2, H_q=4, H_kv=2, D=64, N=40, past=[500, 77], dtype="f16", cap=20.0, slopes=True, window=90,
                    prefix=[70, 100], docs=_docs([500, 77], 40, [64, 3])),
    "tc5_prefix": dict(B=1, H_q=4, H_kv=2, D=128, N=130, past=[70], dtype="bf16", prefix=[150]),
    "tc5_window_blocks": dict(B=2, H_q=6, H_kv=2, D=128, N=50, past=[700, 10], dtype="bf16", window=33, slopes=True),
    "many_seqs": dict(B=70, H_q=2, H_kv=1, D=64, N=1, past=[(37 * b) % 300 for b in range(70)], dtype="bf16", window=20,
                      prefix=[b % 7 for b in range(70)]),
    "page512": dict(B=2, H_q=8, H_kv=2, D=128, N=1, past=[1500, 600], dtype="bf16", window=200, prefix=[3, 3], page=512),
    "rows3_d128": dict(B=1, H_q=3, H_kv=1, D=128, N=1, past=[2000], dtype="bf16", cap=2.0, slopes=True),
    "rows7_d64": dict(B=2, H_q=7, H_kv=1, D=64, N=1, past=[300, 1], dtype="f16", slopes=True, window=128),
}


@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "paged"])
@pytest.mark.parametrize("name", CASES)
def test_parity(name, paged):
    c = Case(**CASES[name], seed=sorted(CASES).index(name))
    out, err = c.run(paged)
    assert err == 0
    c.check(out)


def test_long_split_merge_pass_and_short_window():
    """Long ranges (heads split over CTAs, the separate merge pass), with a window that leaves few tiles."""
    past = [9000, 5000, 7001, 8192]
    for more in (dict(cap=30.0), dict(window=3000, prefix=[4] * 4), dict(window=300, prefix=[4] * 4, slopes=True)):
        c = Case(4, 8, 8, 128, 1, past, "f32", **more)
        out, err = c.run(True)
        assert err == 0
        c.check(out)


def test_no_modification_is_the_plain_call():
    """fp32 runs the plain call's kernels: the same bits.  16-bit caches have kernels of their own, which
    sum in another order: both calls within the bound of the exact result."""
    for dtype, N in (("f32", 2), ("bf16", 1), ("bf16", 8), ("f16", 24)):
        c = Case(2, 8, 4, 128, N, [400, 61], dtype)
        out, _ = c.run(False)
        plain = torch.empty_like(out)
        ws = kvd.alloc_workspace(2, 8, 4, 128, N, 400, c.dt)
        kvd.kvd_decode_attention(c.q.to(DEV), c.k.to(DEV), c.v.to(DEV), plain,
                                 torch.tensor(c.past, dtype=torch.int32, device=DEV), 400, workspace=ws)
        torch.cuda.synchronize()
        if dtype == "f32":
            assert np.array_equal(_bits(out), _bits(plain))
        else:
            c.check(out)
            c.check(plain)


def test_streams_graph_and_workspace_reuse():
    """Calls on two streams with their own workspaces, a captured call replayed, one workspace used by
    different modifications in turn: the same bits as alone."""
    a = Case(**CASES["sinks_mma"])
    b = Case(**CASES["tc5_all"])
    want_a, want_b = a.run(False)[0], b.run(True)[0]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ws = a.workspace()
    for _ in range(3):
        out_a, _ = a.run(False, stream=s1, workspace=ws)
        out_b, _ = b.run(True, stream=s2)
        assert np.array_equal(_bits(out_a), _bits(want_a)) and np.array_equal(_bits(out_b), _bits(want_b))
        a.run(False, workspace=ws, softcap=0.0)
    args = [x.to(DEV) for x in (a.q, a.k, a.v)]
    past = torch.tensor(a.past, dtype=torch.int32, device=DEV)
    more, out = a.more(), torch.zeros_like(args[0])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kvd.kvd_decode_attention_scored(*args, out, past, max(a.past), workspace=ws, **more)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(_bits(out), _bits(want_a))


def test_bad_sequences_are_skipped_and_flagged():
    c = Case(3, 8, 2, 128, 1, [200, 100, 50], "bf16", window=64, prefix=[4, 4, 4])
    q, k, v = (x.to(DEV) for x in (c.q, c.k, c.v))
    out = torch.full_like(q, 7.0)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    past = torch.tensor([200, -1, 50], dtype=torch.int32, device=DEV)
    kvd.kvd_decode_attention_scored(q, k, v, out, past, 200, workspace=c.workspace(), err_word=err, **c.more())
    torch.cuda.synchronize()
    assert int(err) == kvd.KVD_DEVERR_PAST_LEN
    assert bool((out[1] == 7.0).all())
    good, _ = c.run(False)
    assert np.array_equal(_bits(out[0]), _bits(good[0])) and np.array_equal(_bits(out[2]), _bits(good[2]))
    c.table[0, 3] = c.kp.shape[0]  # the last page of the first sequence: outside the pool
    out, err = c.run(True)
    assert err == kvd.KVD_DEVERR_PAGE
    assert np.array_equal(_bits(out[1]), _bits(good[1]))


def test_binding_refuses():
    c = Case(**CASES["sinks_mma"])
    for bad in (dict(window=-1), dict(window=1 << 31), dict(slopes=torch.ones(3, device=DEV)),
                dict(slopes=torch.ones(8, dtype=torch.float64, device=DEV)),
                dict(prefix_len=torch.ones(1, dtype=torch.int32, device=DEV)),
                dict(doc_start=torch.ones(3, dtype=torch.int32, device=DEV))):
        with pytest.raises(ValueError):
            c.run(False, **bad)
    for bad, status in ((dict(softcap=-1.0), kvd.KVD_ERR_INVALID_ARG), (dict(softcap=float("nan")), kvd.KVD_ERR_INVALID_ARG),
                        (dict(workspace=None), kvd.KVD_ERR_WORKSPACE)):
        with pytest.raises(kvd.KvdError) as e:
            c.run(False, **bad)
        assert e.value.status == status


@pytest.mark.parametrize("order", ["rising", "mixed"])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64), ("f32", 64)])
def test_maxima_that_jump(dtype, D, order):
    """Every 32 keys a row's scores lie some 2^40 higher (or elsewhere at random): the maximum moves inside
    tiles, far beyond what a weight may exceed it by."""
    for N, past in ((40, [333, 77]), (1, [700, 64])):
        c = Case(2, 4, 2, D, N, past, dtype, window=10 ** 6, seed=300)
        steps = np.arange(-(-c.k.shape[2] // 32)) * 28.0 * (D / 64) ** 0.5
        if order == "mixed":
            np.random.default_rng(3).shuffle(steps)
        u = torch.full((D,), D ** -0.5)
        c.q = (c.q.float() / 2 + 8 * u).to(c.dt)
        c.k = (c.k.float() + torch.from_numpy(np.repeat(steps, 32)[:c.k.shape[2]]).float()[None, None, :, None] * u).to(c.dt)
        out, err = c.run(False)
        assert err == 0
        c.check(out)
