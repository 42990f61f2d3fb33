"""Attention over a shared prefix on the GPU (kvd_shared_prefix_attention and
kvd_paged_shared_prefix_attention) against fp64, with the bound of
attn_reference (the join of a row's parts adds roundings of 2^-24 each, within
its count of sums).  Rows past the prefix and past the sequences' ends hold NaN.
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
    def __init__(self, B, H_q, H_kv, D, N, S, past, dtype, page=64, seed=0, peak=1.0):
        self.__dict__.update(B=B, H_q=H_q, H_kv=H_kv, D=D, N=N, S=S, past=past, dtype=dtype, page=page, dt=DT[dtype])
        g = torch.Generator("cpu").manual_seed(3000 + seed)
        rnd = lambda *s: torch.randn(s, generator=g).to(self.dt)
        T = max(past) + N + 5
        self.q = (rnd(B, H_q, N, D).float() * 2 * peak).to(self.dt)
        self.kp, self.vp = rnd(H_kv, S + 3, D), rnd(H_kv, S + 3, D)
        self.kp[:, S:] = float("nan")
        self.vp[:, S:] = float("nan")
        self.k, self.v = rnd(B, H_kv, T, D), rnd(B, H_kv, T, D)
        for b, P in enumerate(past):
            self.k[b, :, P + N:] = float("nan")
            self.v[b, :, P + N:] = float("nan")
        n, first = -(-T // page), -(-S // page)
        total = B * n + first + 2
        perm = torch.randperm(total, generator=g).to(torch.int32)
        self.table, self.ptable = perm[:B * n].view(B, n).clone(), perm[B * n:B * n + first].clone()
        self.pool_k = torch.full((total, H_kv, page, D), float("nan"), dtype=self.dt)
        self.pool_v = self.pool_k.clone()
        for pool, own, pre in ((self.pool_k, self.k, self.kp), (self.pool_v, self.v, self.vp)):
            for j in range(first):
                rows = slice(j * page, min(S, (j + 1) * page))
                pool[self.ptable[j].item(), :, :rows.stop - rows.start] = pre[:, rows]
            for b in range(B):
                for j in range(n):
                    rows = slice(j * page, min(T, (j + 1) * page))
                    pool[self.table[b, j].item(), :, :rows.stop - rows.start] = own[b, :, rows]

    def workspace(self):
        ws = kvd.alloc_shared_prefix_workspace(self.B, self.H_q, self.H_kv, self.D, self.N, self.S, max(self.past), self.dt)
        return ws.fill_(0xff)  # (NaN: it needs no initial contents)

    def inputs(self):
        return {n: getattr(self, n).to(DEV) for n in ("q", "kp", "vp", "k", "v", "pool_k", "pool_v", "table", "ptable")}

    def call(self, x, out, past, paged, **more):
        if paged:
            kvd.kvd_paged_shared_prefix_attention(x["q"], x["pool_k"], x["pool_v"], x["ptable"], self.S, out, x["table"],
                                                  past, max(self.past), **more)
        else:
            kvd.kvd_shared_prefix_attention(x["q"], x["kp"], x["vp"], self.S, x["k"], x["v"], out, past,
                                            max(self.past), **more)

    def run(self, paged, past=None, **over):
        x = self.inputs()
        out = torch.full(self.q.shape, float("nan"), dtype=self.dt, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        past = torch.tensor(self.past if past is None else past, dtype=torch.int32, device=DEV)
        more = {"workspace": self.workspace(), "err_word": err, **over}
        torch.cuda.synchronize()
        self.call(x, out, past, paged, **more)
        torch.cuda.synchronize()
        return out, int(err)

    def check(self, out, heads=None, seqs=None):
        got = out.double().cpu().numpy()
        q, k, v, kp, vp = (x.double().numpy() for x in (self.q, self.k, self.v, self.kp, self.vp))
        g = self.H_q // self.H_kv
        for b in range(self.B) if seqs is None else seqs:
            P, S = self.past[b], self.S
            mask = np.concatenate([np.ones((self.N, S), bool), seen_mask(P, self.N, 0, 0, None)], axis=1)
            for h in range(self.H_kv) if heads is None else heads:
                kk = np.concatenate([kp[h, :S], k[b, h, :P + self.N]])[None]
                vv = np.concatenate([vp[h, :S], v[b, h, :P + self.N]])[None]
                rows = slice(h * g, (h + 1) * g)
                ref, tol = attention64(q[b, rows], kk, vv, self.D ** -0.5, mask, dtype=self.dtype)
                assert_near(got[b, rows], ref, tol, f"sequence {b} head {h}")


CASES = {
    "one_row": dict(B=1, H_q=1, H_kv=1, D=64, N=1, S=1, past=[0], dtype="bf16"),
    "short_prefix": dict(B=3, H_q=4, H_kv=2, D=64, N=1, S=63, past=[0, 5, 100], dtype="f16"),
    "tile_exact": dict(B=2, H_q=4, H_kv=2, D=128, N=2, S=256, past=[64, 0], dtype="bf16"),
    "tile_plus_one": dict(B=2, H_q=4, H_kv=2, D=128, N=1, S=257, past=[63, 300], dtype="f16"),
    "odd_group": dict(B=30, H_q=5, H_kv=1, D=64, N=1, S=1000, past=[(31 * b) % 200 for b in range(30)], dtype="bf16"),
    "two_blocks": dict(B=50, H_q=8, H_kv=2, D=128, N=1, S=700, past=[b % 9 for b in range(50)], dtype="bf16"),
    "three_blocks": dict(B=70, H_q=8, H_kv=2, D=64, N=1, S=300, past=[b for b in range(70)], dtype="f16"),
    "rows_65": dict(B=3, H_q=5, H_kv=1, D=128, N=13, S=333, past=[200, 0, 64], dtype="bf16"),
    "rows_128": dict(B=3, H_q=8, H_kv=1, D=64, N=16, S=129, past=[10, 0, 64], dtype="bf16"),
    "rows_200": dict(B=2, H_q=8, H_kv=1, D=128, N=25, S=400, past=[10, 90], dtype="f16"),
    "rows_1000": dict(B=2, H_q=8, H_kv=1, D=64, N=125, S=190, past=[3, 77], dtype="bf16"),
    "many_heads": dict(B=4, H_q=24, H_kv=24, D=64, N=1, S=2000, past=[0, 1, 64, 65], dtype="f16", page=128),
    "peaked": dict(B=5, H_q=4, H_kv=2, D=128, N=1, S=1500, past=[7, 30, 0, 200, 64], dtype="bf16", peak=6.0),
    "f32": dict(B=3, H_q=4, H_kv=2, D=64, N=2, S=200, past=[0, 64, 33], dtype="f32"),
    "f32_d128": dict(B=40, H_q=4, H_kv=1, D=128, N=1, S=321, past=[b % 5 for b in range(40)], dtype="f32"),
    "f32_rows_130": dict(B=2, H_q=2, H_kv=1, D=64, N=65, S=65, past=[9, 70], dtype="f32", page=128),
    "no_prefix": dict(B=3, H_q=4, H_kv=2, D=128, N=1, S=0, past=[100, 0, 64], dtype="bf16"),
    "no_prefix_f32": dict(B=2, H_q=4, H_kv=2, D=64, N=3, S=0, past=[100, 0], dtype="f32"),
}


@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "paged"])
@pytest.mark.parametrize("name", CASES)
def test_parity(name, paged):
    c = Case(**CASES[name], seed=sorted(CASES).index(name))
    out, err = c.run(paged)
    assert err == 0
    c.check(out)


def test_long_prefix():
    """A prefix split over every SM, several pieces a row, rows in every block; long own caches beside."""
    c = Case(40, 16, 4, 128, 1, 9001, [(577 * b) % 1500 for b in range(40)], "bf16", seed=90)
    for paged in (False, True):
        out, err = c.run(paged)
        assert err == 0
        c.check(out, heads=[0, 3], seqs=[0, 1, 31, 32, 39])


def test_is_the_one_cache_call():
    """Against kvd_decode_attention over caches that hold the prefix in front, within both calls' bounds."""
    c = Case(6, 8, 2, 128, 2, 130, [0, 5, 64, 70, 1, 200], "f16", seed=5)
    out, _ = c.run(False)
    T = c.S + c.k.shape[2]
    k = torch.cat([c.kp[None, :, :c.S].expand(6, -1, -1, -1), c.k], dim=2).contiguous().to(DEV)
    v = torch.cat([c.vp[None, :, :c.S].expand(6, -1, -1, -1), c.v], dim=2).contiguous().to(DEV)
    past = torch.tensor([c.S + P for P in c.past], dtype=torch.int32, device=DEV)
    one = torch.empty_like(out)
    kvd.kvd_decode_attention(c.q.to(DEV), k, v, one, past, T - c.N, workspace=kvd.alloc_workspace(6, 8, 2, 128, 2, T - c.N, c.dt))
    torch.cuda.synchronize()
    c.check(out)
    c.check(one)


def test_streams_graph_and_workspace_reuse():
    """The same bits eager, on another stream, replayed, and on a workspace that another shape used."""
    c = Case(**CASES["two_blocks"])
    want, _ = c.run(False)
    side = torch.cuda.Stream()
    out, _ = c.run(False, stream=side)
    assert np.array_equal(_bits(out), _bits(want))
    ws = c.workspace()
    c.run(True, workspace=ws)
    small = Case(**CASES["no_prefix"])
    ref, _ = small.run(False)
    assert np.array_equal(_bits(small.run(False, workspace=ws)[0]), _bits(ref))
    x, past = c.inputs(), torch.tensor(c.past, dtype=torch.int32, device=DEV)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for _ in range(3):  # back to back: each call's launches overlap its neighbours'
            c.call(x, out, past, False, workspace=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(_bits(out), _bits(want))


def test_bad_sequences_and_pages():
    c = Case(3, 8, 2, 128, 1, 300, [100, 50, 20], "bf16", seed=8)
    good, _ = c.run(False)
    out, err = c.run(False, past=[100, -1, 20])
    assert err == kvd.KVD_DEVERR_PAST_LEN
    assert bool(torch.isnan(out[1]).all())  # (left as it was)
    assert np.array_equal(_bits(out[0]), _bits(good[0])) and np.array_equal(_bits(out[2]), _bits(good[2]))
    c.table[1, 0] = -7
    out, err = c.run(True)
    assert err == kvd.KVD_DEVERR_PAGE
    paged = out
    c.table[1, 0] = 0
    c.ptable[2] = c.pool_k.shape[0]
    out, err = c.run(True)
    assert err == kvd.KVD_DEVERR_PAGE
    assert np.array_equal(_bits(paged[0]), _bits(good[0]))


def test_binding_and_library_refuse():
    c = Case(**CASES["tile_exact"])
    x = c.inputs()
    out, past = torch.empty_like(x["q"]), torch.tensor(c.past, dtype=torch.int32, device=DEV)
    ws = c.workspace()
    for bad in (dict(kp=x["kp"][:1]), dict(kp=x["kp"].float()), dict(vp=x["vp"][:, :5]), dict(k=x["k"][:1])):
        with pytest.raises(ValueError):
            c.call({**x, **bad}, out, past, False, workspace=ws)
    with pytest.raises(ValueError):
        c.call({**x, "ptable": x["ptable"][:1]}, out, past, True, workspace=ws)
    for S, w, status in ((c.S + 4, ws, kvd.KVD_ERR_CAPACITY), (-1, ws, kvd.KVD_ERR_INVALID_ARG), (c.S, None, kvd.KVD_ERR_WORKSPACE),
                         (c.S, ws[:-256], kvd.KVD_ERR_WORKSPACE)):
        with pytest.raises(kvd.KvdError) as e:
            kvd.kvd_shared_prefix_attention(x["q"], x["kp"], x["vp"], S, x["k"], x["v"], out, past, max(c.past), workspace=w)
        assert e.value.status == status


@pytest.mark.parametrize("order", ["rising", "mixed"])
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("f16", 128), ("f32", 64)])
def test_maxima_that_jump(dtype, D, order):
    """Every 32 keys of the prefix a row's scores lie some 2^40 higher (or elsewhere at random): the maximum
    moves inside tiles, far beyond what a weight may exceed it by."""
    c = Case(5, 8, 2, D, 3, 500, [70, 0, 3, 64, 200], dtype, seed=301)
    steps = np.arange(-(-c.kp.shape[1] // 32)) * 28.0 * (D / 64) ** 0.5
    if order == "mixed":
        np.random.default_rng(4).shuffle(steps)
    u = torch.full((D,), D ** -0.5)
    c.q = (c.q.float() / 2 + 8 * u).to(c.dt)
    c.kp = (c.kp.float() + torch.from_numpy(np.repeat(steps, 32)[:c.kp.shape[1]]).float()[None, :, None] * u).to(c.dt)
    # (the sequences' own keys: about where the prefix ends)
    c.k = (c.k.float() + float(steps.max()) * u).to(c.dt)
    out, err = c.run(False)
    assert err == 0
    c.check(out)
