"""Cases for the serving operators around the KV cache: rotating and appending a
step's new rows, decode attention with modified scores, and decode attention of
a batch that shares one long prefix.

Each case names its operator in ``op``:

* ``rope``   -- q and the new keys of N tokens per sequence are rotated by their
  positions, the rotated keys and the values written into the cache
  (contiguous [B, H_kv, T_max, D], or pages of ``page`` tokens);
* ``scored`` -- attention of the N appended rows with any of: scores capped by
  a tanh, a per-head penalty on the distance, a sliding window, a prefix that
  every row sees, documents packed into one sequence;
* ``prefix`` -- attention of the N appended rows over one prefix common to all
  sequences, followed by each sequence's own cache.

``run`` computes the plain form (elementary torch operations in fp32, angles in
fp64) while ``own`` is false, and calls the framework's entry points while it
is true.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------------
# cases
def _rope(name, B, H_q, H_kv, D, N, dtype, past, T_max, rot, pairs="halves", page=0, fused=False, pos_base=0):
    return {"name": name, "op": "rope", "B": B, "H_q": H_q, "H_kv": H_kv, "D": D, "N": N, "dtype": dtype, "lo": past[0],
            "hi": past[1], "T_max": T_max, "rot": rot, "pairs": pairs, "page": page, "fused": fused,
            "pos_base": pos_base}


def _scored(name, B, H_q, H_kv, D, N, dtype, past, page=0, cap=0.0, slopes=False, window=0, prefix="none", docs=False):
    return {"name": name, "op": "scored", "B": B, "H_q": H_q, "H_kv": H_kv, "D": D, "N": N, "dtype": dtype, "lo": past[0],
            "hi": past[1], "page": page, "cap": cap, "slopes": slopes, "window": window, "prefix": prefix, "docs": docs}


def _prefix(name, B, H_q, H_kv, D, N, dtype, S, past, page=0):
    return {"name": name, "op": "prefix", "B": B, "H_q": H_q, "H_kv": H_kv, "D": D, "N": N, "dtype": dtype, "S": S,
            "lo": past[0], "hi": past[1], "page": page}


def listed():
    return [
        # one token of one sequence, fp32, interleaved pairs, a rotation of half the head: bare latency
        _rope("rope_one_token_f32", 1, 12, 12, 64, 1, "f32", (1000, 1000), 1024, 32, pairs="neighbours"),
        # a decode step of a grouped-query batch on pages, far positions
        _rope("rope_step_b32_paged", 32, 32, 8, 128, 1, "bf16", (100, 500), 512, 128, page=64, pos_base=100000),
        # an odd chunk on pages, fp16, straight from a fused projection's rows
        _rope("rope_chunk_333_f16", 5, 12, 4, 64, 333, "f16", (0, 600), 1024, 64, page=128, fused=True),
        # a long prefill chunk of two sequences, from a fused projection's rows
        _rope("rope_prefill_2048", 2, 32, 8, 128, 2048, "bf16", (0, 2000), 4160, 128, fused=True),
        # one token of one sequence, fp32, distance penalty: bare latency
        _scored("scored_one_token_f32", 1, 12, 12, 64, 1, "f32", (1000, 1000), slopes=True),
        # the long-context decode step with capped scores on pages
        _scored("scored_step_cap_paged", 32, 32, 8, 128, 1, "bf16", (1024, 8192), page=64, cap=30.0),
        # the same batch in a sliding-window layer that keeps its first tokens in sight
        _scored("scored_step_window", 32, 32, 8, 128, 1, "bf16", (1024, 8192), cap=50.0, window=1024, prefix="sinks"),
        # a chunk of 16 new tokens in packed documents, fp16, distance penalty
        _scored("scored_docs_n16_f16", 16, 12, 12, 64, 16, "f16", (700, 4001), slopes=True, docs=True),
        # a prefill chunk whose prompt prefix attends both ways, capped
        _scored("scored_chunk_128_prefix", 4, 32, 8, 128, 128, "bf16", (1500, 8000), cap=50.0, prefix="chunk"),
        # a small batch over a short system prompt
        _prefix("prefix_b8_s1000", 8, 12, 12, 64, 1, "bf16", 1000, (0, 64)),
        # a serving batch over a long shared prompt
        _prefix("prefix_b128_s16384", 128, 32, 8, 128, 1, "bf16", 16384, (16, 512)),
        # four tokens a step on pages, odd prefix, fp16
        _prefix("prefix_n4_paged_f16", 16, 32, 8, 128, 4, "f16", 5003, (100, 1500), page=64),
    ]


def _log(rng, lo, hi):
    """A whole number in lo..hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        m = most.setdefault(c["op"], [0, 0])
        m[0], m[1] = max(m[0], w["bytes"]), max(m[1], w["flops"])
    while True:
        op = rng.choice(("rope", "scored", "prefix"))
        D = rng.choice((64, 128))
        H_kv = rng.choice((1, 2, 4, 8, 12))
        H_q = H_kv * rng.choice((1, 2, 3, 4, 8))
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        page = rng.choice((0, 0, 64, 128))
        if op == "rope":
            B, N = _log(rng, 1, 64), rng.choice((1, 1, _log(rng, 2, 2048)))
            hi = _log(rng, 1, 2000)
            c = _rope("", B, H_q, H_kv, D, N, dtype, (rng.randint(0, hi), hi), hi + N + rng.randint(0, 200),
                      rng.choice((D, D, D // 2, D // 4)), rng.choice(("halves", "neighbours")), page,
                      rng.random() < 0.5, rng.choice((0, 0, _log(rng, 1, 1000000))))
        elif op == "scored":
            B, N = _log(rng, 1, 64), rng.choice((1, 1, 2, 3, 5, _log(rng, 2, 128)))
            hi = _log(rng, 1, 8192)
            c = _scored("", B, H_q, H_kv, D, N, dtype, (rng.randint(0, hi), hi), page, rng.choice((0.0, 20.0, 50.0)),
                        rng.random() < 0.4, rng.choice((0, 0, _log(rng, 1, 4096))),
                        rng.choice(("none", "none", "sinks", "chunk")), rng.random() < 0.3)
        else:
            B, N = _log(rng, 1, 128), rng.choice((1, 1, 2, 3, _log(rng, 2, 16)))
            hi = _log(rng, 1, 1500)
            c = _prefix("", B, H_q, H_kv, D, N, dtype, _log(rng, 1, 16384), (rng.randint(0, hi), hi), page)
        if H_q // H_kv * N > 1024:
            continue
        w = work(c)
        if w["bytes"] <= most[op][0] and w["flops"] <= most[op][1] and _cache_values(c) <= 300e6 and _score_values(c) <= 300e6:
            if dtype != "f32" or op == "rope" or w["flops"] <= 2e9:
                del c["name"]
                return c


def _lens(c):
    """The sequences' cached tokens, spread over lo..hi (their order is the seed's)."""
    B = c["B"]
    return [c["lo"] + (c["hi"] - c["lo"]) * b // max(1, B - 1) if B > 1 else c["hi"] for b in range(B)]


def _slots(c):
    """Tokens that a sequence's cache has room for, and pages of it (0: not paged)."""
    T = c["T_max"] if c["op"] == "rope" else c["hi"] + c["N"] + 17
    if not c["page"]:
        return T, 0
    n = -(-T // c["page"])
    return n * c["page"], n


def _cache_values(c):
    return 2.0 * (c["B"] * c["H_kv"] * _slots(c)[0] * c["D"] + (c["H_kv"] * c.get("S", 0) * c["D"]))


def _score_values(c):
    return float(c["B"]) * c["H_q"] * c["N"] * (c["hi"] + c["N"] + c.get("S", 0)) if c["op"] != "rope" else 0.0


def _prefix_of(c, P):
    """How many of the first keys every row of a sequence with P cached tokens sees."""
    return {"none": 0, "sinks": 4, "chunk": P + c["N"] // 2}[c["prefix"]]


def _docs_of(c, P):
    """The first key of each new row's document: one began in the cache, another begins inside the chunk."""
    N = c["N"]
    if not c["docs"]:
        return [0] * N
    return [3 * P // 8 if i < max(1, N // 2) else P + N // 2 for i in range(N)]


def _visible(c, P):
    """(keys that any row of the sequence sees, pairs of row and key in sight) of a sequence with P cached tokens."""
    N, W, pre = c["N"], c["window"], min(_prefix_of(c, P), P + c["N"])
    docs, pairs = _docs_of(c, P), 0
    lo_all = P + N
    for i in range(N):
        p = P + i
        lo = max(0, p - W + 1) if W else 0
        a, b = max(lo, pre), p + 1                      # the causal or windowed part past the prefix
        pairs += max(0, b - max(a, docs[i])) + max(0, pre - docs[i])
        lo_all = min(lo_all, max(lo, docs[i]))
    keys = max(0, P + N - max(lo_all, min(pre, P + N))) + max(0, pre - docs[0])
    return keys, pairs


def work(case):
    c, es = case, 4 if case["dtype"] == "f32" else 2
    rows = c["B"] * c["N"] * c["D"]
    if c["op"] == "rope":
        return {"bytes": rows * es * (2 * c["H_q"] + 4 * c["H_kv"]),
                "flops": 3.0 * c["B"] * c["N"] * c["rot"] * (c["H_q"] + c["H_kv"])}
    q_out = 2 * rows * c["H_q"] * es
    if c["op"] == "scored":
        seen = [_visible(c, P) for P in _lens(c)]
        return {"bytes": q_out + 2 * es * c["H_kv"] * c["D"] * sum(k for k, _ in seen),
                "flops": 4.0 * c["D"] * c["H_q"] * sum(p for _, p in seen)}
    N, S = c["N"], c["S"]
    return {"bytes": q_out + 2 * es * c["H_kv"] * c["D"] * (S + sum(P + N for P in _lens(c))),
            "flops": 4.0 * c["D"] * c["H_q"] * sum(N * (S + P) + N * (N + 1) // 2 for P in _lens(c))}


# ---------------------------------------------------------------------------------
# inputs
def prepare(case, seed):
    c, dev = dict(case), "cuda"
    dt = DTYPES[c["dtype"]]
    g = torch.Generator(dev).manual_seed(int(seed) * 7919 + 17)
    host = torch.Generator("cpu").manual_seed(int(seed) * 104729 + 29)
    B, H_q, H_kv, D, N = c["B"], c["H_q"], c["H_kv"], c["D"], c["N"]

    def randn(*shape, by=1.0):
        return (torch.randn(shape, generator=g, device=dev) * by).to(dt)

    past_cpu = torch.tensor(_lens(c), dtype=torch.int32)[torch.randperm(B, generator=host)]
    s = {"case": c, "past_len": past_cpu.to(dev), "max_past": c["hi"]}
    slots, n_pages = _slots(c)
    if n_pages:
        # one pool; the sequences' pages (and a shared prefix's) lie in it in any order, a few are spare
        first = -(-c["S"] // c["page"]) if c["op"] == "prefix" else 0
        total = B * n_pages + first + 3
        order = torch.randperm(total, generator=host).to(torch.int32)
        s["table"] = order[:B * n_pages].view(B, n_pages).contiguous().to(dev)
        s["prefix_table"] = order[B * n_pages:B * n_pages + first].contiguous().to(dev)
        s["k"], s["v"] = randn(total, H_kv, c["page"], D), randn(total, H_kv, c["page"], D)
    else:
        s["k"], s["v"] = randn(B, H_kv, slots, D), randn(B, H_kv, slots, D)
        if c["op"] == "prefix":
            s["k_prefix"], s["v_prefix"] = randn(H_kv, c["S"], D), randn(H_kv, c["S"], D)
    if c["op"] == "rope":
        if c["fused"]:  # the rows of one projection: [B, N, H_q + 2 H_kv, D]
            qkv = randn(B, N, H_q + 2 * H_kv, D).transpose(1, 2)
            s["q"], s["k_new"], s["v_new"] = qkv[:, :H_q], qkv[:, H_q:H_q + H_kv], qkv[:, H_q + H_kv:]
        else:
            s["q"], s["k_new"], s["v_new"] = randn(B, H_q, N, D), randn(B, H_kv, N, D), randn(B, H_kv, N, D)
        half = c["rot"] // 2
        s["inv_freq"] = torch.tensor([10000.0 ** (-f / half) for f in range(half)], dtype=torch.float64).to(dev)
        s["q_out"] = torch.empty(B, H_q, N, D, dtype=dt, device=dev)
        return s
    # queries whose scores spread as a trained layer's do (a few keys take most of the weight)
    s["q"] = randn(B, H_q, N, D, by=2.5)
    s["out"] = torch.empty_like(s["q"])
    if c["op"] == "scored":
        lens = past_cpu.tolist()
        s["slopes"] = (2.0 ** (-8.0 * torch.arange(1, H_q + 1, dtype=torch.float64) / H_q)).float().to(dev) if c["slopes"] else None
        s["doc_start"] = torch.tensor([_docs_of(c, P) for P in lens], dtype=torch.int32).to(dev) if c["docs"] else None
        s["prefix_len"] = torch.tensor([_prefix_of(c, P) for P in lens], dtype=torch.int32).to(dev) if c["prefix"] != "none" else None
    return s


# ---------------------------------------------------------------------------------
# one pass
def run(state):
    return {"rope": _run_rope, "scored": _run_scored, "prefix": _run_prefix}[state["case"]["op"]](state)


def _run_rope(s):
    c = s["case"]
    if own:
        import kv_cache_decode_append_gb300 as kvd
        more = {"interleaved": c["pairs"] == "neighbours", "pos_base": c["pos_base"]}
        if c["page"]:
            kvd.kvd_paged_rope_append(s["q"], s["q_out"], s["k"], s["v"], s["k_new"], s["v_new"], s["table"],
                                      s["past_len"], s["max_past"], s["inv_freq"], **more)
        else:
            kvd.kvd_rope_append(s["q"], s["q_out"], s["k"], s["v"], s["k_new"], s["v_new"], s["past_len"],
                                s["max_past"], s["inv_freq"], **more)
        return s["q_out"], s["k"], s["v"]
    dt, N = s["q"].dtype, c["N"]
    t = s["past_len"].long()[:, None] + torch.arange(N, device="cuda")
    angle = (t + c["pos_base"]).double()[:, None, :, None] * s["inv_freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    q, k = _plain_rotate(s["q"], cos, sin, c), _plain_rotate(s["k_new"], cos, sin, c)
    at = torch.arange(c["B"], device="cuda")[:, None]
    slot = t
    if c["page"]:
        at, slot = s["table"].long().gather(1, t // c["page"]), t % c["page"]
    s["k"][at, :, slot] = k.to(dt).transpose(1, 2)
    s["v"][at, :, slot] = s["v_new"].transpose(1, 2)
    return q.to(dt), s["k"], s["v"]


def _plain_rotate(x, cos, sin, c):
    """Rows [B, H, N, D] in fp32 with their first `rot` elements rotated in pairs."""
    x, rot = x.float(), c["rot"]
    if c["pairs"] == "neighbours":
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((turned, x[..., rot:]), dim=-1)


def _plain_cache(s, which, T):
    """The first T keys or values of every sequence, [B, H_kv, T, D] in fp32."""
    c, x = s["case"], s[which]
    if c["page"]:
        n = -(-T // c["page"])
        x = x[s["table"][:, :n].long()].transpose(1, 2).reshape(c["B"], c["H_kv"], n * c["page"], c["D"])
    return x[:, :, :T].float()


def _run_scored(s):
    c = s["case"]
    B, H_q, H_kv, D, N = c["B"], c["H_q"], c["H_kv"], c["D"], c["N"]
    if own:
        import kv_cache_decode_append_gb300 as kvd
        if "workspace" not in s:
            s["workspace"] = kvd.alloc_scored_workspace(B, H_q, H_kv, D, N, s["max_past"], s["q"].dtype)
        more = {"softcap": c["cap"], "slopes": s["slopes"], "window": c["window"], "doc_start": s["doc_start"],
                "prefix_len": s["prefix_len"], "workspace": s["workspace"]}
        if c["page"]:
            kvd.kvd_paged_decode_attention_scored(s["q"], s["k"], s["v"], s["out"], s["table"], s["past_len"],
                                                  s["max_past"], **more)
        else:
            kvd.kvd_decode_attention_scored(s["q"], s["k"], s["v"], s["out"], s["past_len"], s["max_past"], **more)
        return s["out"]
    T = s["max_past"] + N
    k, v = _plain_cache(s, "k", T), _plain_cache(s, "v", T)
    scores = (s["q"].float().view(B, H_kv, H_q // H_kv * N, D) @ k.transpose(2, 3)).view(B, H_q, N, T) / math.sqrt(D)
    if c["cap"]:
        scores = c["cap"] * torch.tanh(scores / c["cap"])
    p = (s["past_len"].long()[:, None] + torch.arange(N, device="cuda"))[:, None, :, None]
    j = torch.arange(T, device="cuda")
    if c["slopes"]:
        scores = scores - s["slopes"][:, None, None] * (p - j).abs()
    seen = j <= p
    if c["window"]:
        seen = seen & (j > p - c["window"])
    if s["prefix_len"] is not None:
        seen = seen | (j < s["prefix_len"].long()[:, None, None, None])
    if c["docs"]:
        seen = seen & (j >= s["doc_start"].long()[:, None, :, None])
    seen = seen & (j < s["past_len"].long()[:, None, None, None] + N)
    scores = torch.where(seen, scores, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    w = torch.exp(scores - torch.where(top == float("-inf"), 0.0, top))
    total = w.sum(-1, keepdim=True)
    o = (w.view(B, H_kv, -1, T) @ v).view(B, H_q, N, D)
    return torch.where(total > 0, o / total, 0.0).to(s["q"].dtype)


def _run_prefix(s):
    c = s["case"]
    B, H_q, H_kv, D, N, S = c["B"], c["H_q"], c["H_kv"], c["D"], c["N"], c["S"]
    if own:
        import kv_cache_decode_append_gb300 as kvd
        if "workspace" not in s:
            s["workspace"] = kvd.alloc_shared_prefix_workspace(B, H_q, H_kv, D, N, S, s["max_past"], s["q"].dtype)
        if c["page"]:
            kvd.kvd_paged_shared_prefix_attention(s["q"], s["k"], s["v"], s["prefix_table"], S, s["out"], s["table"],
                                                  s["past_len"], s["max_past"], workspace=s["workspace"])
        else:
            kvd.kvd_shared_prefix_attention(s["q"], s["k_prefix"], s["v_prefix"], S, s["k"], s["v"], s["out"],
                                            s["past_len"], s["max_past"], workspace=s["workspace"])
        return s["out"]
    if c["page"]:
        kp, vp = (s[x][s["prefix_table"].long()].transpose(0, 1).reshape(H_kv, -1, D)[:, :S].float() for x in ("k", "v"))
    else:
        kp, vp = s["k_prefix"].float(), s["v_prefix"].float()
    T, R = s["max_past"] + N, H_q // H_kv * N
    k, v = _plain_cache(s, "k", T), _plain_cache(s, "v", T)
    q = s["q"].float().view(B, H_kv, R, D) / math.sqrt(D)
    far = (q.transpose(0, 1).reshape(H_kv, B * R, D) @ kp.transpose(1, 2)).view(H_kv, B, R, S).transpose(0, 1)
    near = (q @ k.transpose(2, 3)).view(B, H_q, N, T)
    p = (s["past_len"].long()[:, None] + torch.arange(N, device="cuda"))[:, None, :, None]
    near = torch.where(torch.arange(T, device="cuda") <= p, near, float("-inf")).view(B, H_kv, R, T)
    top = torch.maximum(far.amax(-1, keepdim=True), near.amax(-1, keepdim=True))
    w_far, w_near = torch.exp(far - top), torch.exp(near - top)
    total = w_far.sum(-1, keepdim=True) + w_near.sum(-1, keepdim=True)
    o = (w_far.transpose(0, 1).reshape(H_kv, B * R, S) @ vp).view(H_kv, B, R, D).transpose(0, 1) + w_near @ v
    return (o / total).reshape(B, H_q, N, D).to(s["q"].dtype)


# ---------------------------------------------------------------------------------
# the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    lens = s["past_len"].tolist()
    return {"rope": _exact_rope, "scored": _exact_scored, "prefix": _exact_prefix}[c["op"]](s, c, lens)


def _exact_rope(s, c, lens):
    half = c["rot"] // 2
    first, second = (slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["pairs"] == "neighbours" else (slice(0, half), slice(half, c["rot"]))
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    new_k, new_v = s["k_new"].double(), s["v_new"].double()
    q_out = q.clone()
    for b, P in enumerate(lens):
        z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                        torch.outer(torch.arange(P, P + c["N"], device="cuda", dtype=torch.float64) + c["pos_base"], s["inv_freq"]))
        rows = []
        for x in (q[b], new_k[b]):
            y, turned = x.clone(), torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * z
            y[..., first], y[..., second] = turned.real, turned.imag
            rows.append(y)
        q_out[b] = rows[0]
        if c["page"]:
            t = torch.arange(P, P + c["N"], device="cuda")
            pages = s["table"][b].long()[t // c["page"]]
            k[pages, :, t % c["page"]] = rows[1].transpose(0, 1)
            v[pages, :, t % c["page"]] = new_v[b].transpose(0, 1)
        else:
            k[b, :, P:P + c["N"]] = rows[1]
            v[b, :, P:P + c["N"]] = new_v[b]
    return q_out, k, v


def _rows_of(s, c, b, n, which):
    """The first n keys or values of sequence b, [H_kv, n, D] in fp64."""
    if not c["page"]:
        return s[which][b, :, :n].double()
    t = torch.arange(n, device="cuda")
    return s[which][s["table"][b].long()[t // c["page"]], :, t % c["page"]].transpose(0, 1).double()


def _exact_scored(s, c, lens):
    N, group = c["N"], c["H_q"] // c["H_kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, P in enumerate(lens):
        n = P + N
        k, v = (_rows_of(s, c, b, n, x).repeat_interleave(group, 0) for x in ("k", "v"))
        a = torch.einsum("hid,hjd->hij", s["q"][b].double(), k) * c["D"] ** -0.5
        if c["cap"]:
            a = c["cap"] * torch.tanh(a / c["cap"])
        keys = torch.arange(n, device="cuda")
        pre, docs = _prefix_of(c, P), _docs_of(c, P)
        hidden = torch.empty(N, n, dtype=torch.bool, device="cuda")
        for i in range(N):
            low = P + i - c["window"] if c["window"] else -1
            hidden[i] = (((keys > P + i) | (keys <= low)) & (keys >= pre)) | (keys < docs[i])
        if c["slopes"]:
            away = (torch.arange(P, n, device="cuda")[:, None] - keys).abs().double()
            a = a - s["slopes"].double()[:, None, None] * away
        a = a.masked_fill(hidden, float("-inf"))
        w = torch.softmax(a, dim=-1).masked_fill(hidden.all(-1)[None, :, None], 0.0)
        out[b] = torch.einsum("hij,hjd->hid", w, v)
    return out


def _exact_prefix(s, c, lens):
    N, S, group = c["N"], c["S"], c["H_q"] // c["H_kv"]
    if c["page"]:
        t = torch.arange(S, device="cuda")
        pages = s["prefix_table"].long()[t // c["page"]]
        kp, vp = (s[x][pages, :, t % c["page"]].transpose(0, 1).double() for x in ("k", "v"))
    else:
        kp, vp = s["k_prefix"].double(), s["v_prefix"].double()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, P in enumerate(lens):
        k = torch.cat((kp, _rows_of(s, c, b, P + N, "k")), dim=1).repeat_interleave(group, 0)
        v = torch.cat((vp, _rows_of(s, c, b, P + N, "v")), dim=1).repeat_interleave(group, 0)
        a = torch.einsum("hid,hjd->hij", s["q"][b].double(), k) * c["D"] ** -0.5
        later = torch.arange(S + P + N, device="cuda") > S + P + torch.arange(N, device="cuda")[:, None]
        w = torch.softmax(a.masked_fill(later, float("-inf")), dim=-1)
        out[b] = torch.einsum("hij,hjd->hid", w, v)
    return out
