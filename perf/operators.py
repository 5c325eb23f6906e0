"""Cases of the attention half of a test-time-training block: the per-head norm and rotation of
queries and keys with the cache write, causal attention over packed prompts, and one-token steps
over a paged cache.

`run` computes a case in its plain form (elementary torch operations in 32 bits, rounded once), or
through the framework's entry points where `own` is true. `exact` gives the 64-bit results.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_TYPES = {BF16: torch.bfloat16, F32: torch.float32}


# ------------------------------------------------------------------------------------- the cases
def _rope(**kw):
    return dict(dict(op="rope", dtype=BF16, Hq=32, Hkv=8, dh=128, rot=128, layout="half",
                     base=1e6, factor=1.0, norm=True, cache=True, far=0), **kw)


def _packed(**kw):
    return dict(dict(op="packed", Hq=32, Hkv=8, dh=128, docs=1, past=0, window=0), **kw)


def _decode(**kw):
    return dict(dict(op="decode", Hq=32, Hkv=8, dh=128, window=0, page=64, ragged=False), **kw)


def listed():
    return [
        # one token of one sequence: the smallest call of a generating loop
        _rope(name="rope_1", N=1, far=40000),
        # a short prompt in fp32, adjacent pairs, a quarter of the head rotated, no norm, no cache
        _rope(name="rope_1023_f32", N=1023, dtype=F32, Hq=16, Hkv=16, dh=64, rot=16,
              layout="interleaved", base=1e4, norm=False, cache=False),
        # a prompt of the scan's length at the 2560 / 9728 block's heads, far positions, cached
        _rope(name="rope_32768", N=32768, factor=4.0, far=1 << 20),
        # a prompt shorter than a tile, the routing workload's heads
        _packed(name="packed_77", N=77, Hq=16, Hkv=16, dh=64),
        # documents of different lengths packed into one sequence
        _packed(name="packed_8192_docs", N=8192, docs=11),
        # the sliding window that some blocks keep beside the fast weights, TTT-Linear's heads
        _packed(name="packed_8191_window", N=8191, Hq=32, Hkv=32, dh=64, window=2048),
        # a piece of a prompt whose earlier part is in the cache already
        _packed(name="packed_512_past", N=512, past=15872),
        # one long document
        _packed(name="packed_16384", N=16384),
        # a single stream
        _decode(name="decode_1", S=1, L=4096),
        # an ordinary serving batch of ragged lengths in small pages
        _decode(name="decode_33_ragged", S=33, L=5000, Hq=16, Hkv=4, dh=64, page=16, ragged=True),
        # many streams of long contexts
        _decode(name="decode_16_long", S=16, L=32768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "packed", "packed", "decode"])
    dh = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    Hq = Hkv * rng.choice([g for g in (1, 2, 3, 4, 7, 8) if g * Hkv <= 32])
    if op == "rope":
        dh = rng.choice([64, 80, 96, 128, 256])
        rot = 16 * rng.randint(1, dh // 16)
        dtype = rng.choice([BF16, BF16, F32])
        most = 32768 * 40 * 128 * 2 // ((Hq + 2 * Hkv) * dh * (2 if dtype == BF16 else 4))
        return _rope(N=_log(rng, 1, min(32768, most)), dtype=dtype, Hq=Hq, Hkv=Hkv, dh=dh, rot=rot,
                     layout=rng.choice(["half", "interleaved"]), base=rng.choice([1e4, 5e5, 1e6]),
                     factor=rng.choice([1.0, 4.0, 8.0]), norm=rng.random() < 0.7,
                     cache=rng.random() < 0.7, far=rng.choice([0, 5000, 100000, 1 << 20]))
    if op == "packed":
        N = _log(rng, 1, 12000)
        past = _log(rng, 1, 16000 - N) if rng.random() < 0.3 else 0
        docs = 1 if past or N < 64 else rng.choice([1, 1, 2, 5, 16, 40])
        return _packed(N=N, Hq=Hq, Hkv=Hkv, dh=dh, docs=docs, past=past,
                       window=rng.choice([0, 0, 0, 128, 1000, 4096]))
    S = _log(rng, 1, 64)
    most = 500000 * 8 * 128 // (S * Hkv * dh)
    return _decode(S=S, L=_log(rng, 1, min(32768, most)), Hq=Hq, Hkv=Hkv, dh=dh,
                   window=rng.choice([0, 0, 0, 1024]), page=rng.choice([16, 64, 256]),
                   ragged=rng.random() < 0.6)


# ------------------------------------------------------------------------------------ the inputs
def _lengths(case, seed):
    """Host lengths of a case: [(queries, keys)] of the packed sequences, or the cached lengths.
    They belong to the case's seed, so they are drawn on the host."""
    g = torch.Generator().manual_seed(7919 * seed + 13)
    if case["op"] == "packed":
        N, docs = case["N"], case["docs"]
        cuts = sorted(torch.randint(0, N + 1, (docs - 1,), generator=g).tolist())
        cuts = [0] + cuts + [N]
        return [(b - a, b - a + case["past"]) for a, b in zip(cuts, cuts[1:])]
    if not case["ragged"]:
        return [case["L"]] * case["S"]
    # the longest is there every time, and one sequence holds nothing yet
    lens = torch.randint(1, case["L"] + 1, (case["S"],), generator=g).tolist()
    lens[0] = case["L"]
    if len(lens) > 2:
        lens[-1] = 0
    return lens


def _cumulative(lens, device):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=device)


def prepare(case, seed):
    d = torch.device("cuda:0")
    g = torch.Generator(device=d).manual_seed(seed)
    Hq, Hkv, dh = case["Hq"], case["Hkv"], case["dh"]

    def normal(*shape, dtype=torch.bfloat16, by=1.0):
        return (torch.randn(shape, generator=g, device=d) * by).to(dtype)

    if case["op"] == "rope":
        N, t = case["N"], _TYPES[case["dtype"]]
        # one buffer as a fused projection leaves it: queries, keys and values of a token in a row
        row = normal(N, (Hq + 2 * Hkv) * dh, dtype=t, by=1.5)
        half = case["rot"] // 2
        j = torch.arange(half, dtype=torch.float64, device=d)
        s = dict(case=case, Q=row[:, :Hq * dh].view(N, Hq, dh),
                 K=row[:, Hq * dh:(Hq + Hkv) * dh].view(N, Hkv, dh),
                 V=row[:, (Hq + Hkv) * dh:].view(N, Hkv, dh),
                 pos=torch.arange(N, dtype=torch.int32, device=d) + case["far"],
                 inv_freq=case["base"] ** (-2.0 * j / case["rot"]) / case["factor"],
                 rope_scale=0.1 * math.log(case["factor"]) + 1.0, q_w=None, k_w=None)
        if case["norm"]:
            s["q_w"] = 1.0 + 0.2 * torch.randn(dh, generator=g, device=d)
            s["k_w"] = 1.0 + 0.2 * torch.randn(dh, generator=g, device=d)
        if case["cache"]:
            n_slots = -(-(N + N // 8 + 1) // 64) * 64
            s["slots"] = torch.randperm(n_slots, generator=g, device=d)[:N].to(torch.int32)
            s["Kc"], s["Vc"] = normal(n_slots, Hkv, dh, dtype=t), normal(n_slots, Hkv, dh, dtype=t)
        return s
    if case["op"] == "packed":
        lens = _lengths(case, seed)
        nk = sum(b for _, b in lens)
        return dict(case=case, Q=normal(case["N"], Hq, dh), K=normal(nk, Hkv, dh),
                    V=normal(nk, Hkv, dh), cu_q=_cumulative([a for a, _ in lens], d),
                    cu_k=_cumulative([b for _, b in lens], d), scale=dh ** -0.5)
    lens, page = _lengths(case, seed), case["page"]
    most = max(1, -(-max(lens) // page))
    n_pages = sum(-(-n // page) for n in lens) + 3
    order = torch.randperm(n_pages, generator=g, device=d).to(torch.int32)
    held = torch.tensor([-(-n // page) for n in lens], device=d)
    at = torch.cumsum(held, 0) - held
    k = torch.arange(most, device=d)
    table = order[(at[:, None] + k[None]).clamp(max=n_pages - 1)]
    table = torch.where(k[None] < held[:, None], table, torch.full_like(table, -1))
    return dict(case=case, Q=normal(case["S"], Hq, dh), Kc=normal(n_pages * page, Hkv, dh),
                Vc=normal(n_pages * page, Hkv, dh), table=table.contiguous(),
                lens=torch.tensor(lens, dtype=torch.int32, device=d), scale=dh ** -0.5)


# --------------------------------------------------------------------------------- plain forms
def _plain_norm_rope(x, w, s):
    """One head's norm and rotation, in fp32 with the angles in fp64."""
    case = s["case"]
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w
    angle = s["pos"].double()[:, None] * s["inv_freq"]
    c = (angle.cos() * s["rope_scale"]).float()[:, None]
    n = (angle.sin() * s["rope_scale"]).float()[:, None]
    r, rest = y[..., :case["rot"]], y[..., case["rot"]:]
    if case["layout"] == "half":
        a, b = r.chunk(2, -1)
        r = torch.cat((a * c - b * n, a * n + b * c), -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * c - b * n, a * n + b * c), -1).flatten(-2)
    return torch.cat((r, rest), -1).to(x.dtype)


def _plain_rope(s):
    q, k = _plain_norm_rope(s["Q"], s["q_w"], s), _plain_norm_rope(s["K"], s["k_w"], s)
    if not s["case"]["cache"]:
        return q, k
    at = s["slots"].long()
    s["Kc"].index_copy_(0, at, k)
    s["Vc"].index_copy_(0, at, s["V"])
    return q, k, s["Kc"], s["Vc"]


def _plain_softmax(z, v):
    """(P V) and the log of the sum of exponentials for logits z (masked ones -inf, overwritten)."""
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = z.sub_(m).exp_()
    n = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(n == 0, torch.ones_like(n), n)
    return o, (m + n.log()).squeeze(-1)


def _plain_packed(s):
    case = s["case"]
    Hkv, G, dh, N, nk = case["Hkv"], case["Hq"] // case["Hkv"], case["dh"], case["N"], len(s["K"])
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    i, j = torch.arange(N, device=cu_q.device), torch.arange(nk, device=cu_q.device)
    of_q, of_k = (torch.bucketize(x, c[1:], right=True) for x, c in ((i, cu_q), (j, cu_k)))
    # the key that stands at a query's own place, counted from the packed keys' start
    at = i + (cu_k[1:] - cu_q[1:])[of_q]
    see = (of_q[:, None] == of_k[None]) & (j[None] <= at[:, None])
    if case["window"]:
        see &= j[None] > at[:, None] - case["window"]
    q = s["Q"].float().mul(s["scale"]).view(N, Hkv, G, dh).permute(1, 2, 0, 3).reshape(Hkv, G * N, dh)
    k = s["K"].float().permute(1, 2, 0).contiguous()
    v = s["V"].float().permute(1, 0, 2).contiguous()
    z = torch.matmul(q, k).view(Hkv, G, N, nk).masked_fill_(~see, -math.inf).view(Hkv, G * N, nk)
    o, lse = _plain_softmax(z, v)
    o = o.view(Hkv, G, N, dh).permute(2, 0, 1, 3).reshape(N, Hkv * G, dh)
    return o.to(s["Q"].dtype), lse.view(Hkv * G, N).t().contiguous()


def _plain_decode(s):
    case = s["case"]
    Hkv, G, dh, S, page = case["Hkv"], case["Hq"] // case["Hkv"], case["dh"], case["S"], case["page"]
    most = s["table"].shape[1] * page
    j = torch.arange(most, device=s["Q"].device)
    at = s["table"].long()[:, j // page].clamp(min=0) * page + j % page  # [S, most]
    lens = s["lens"][:, None]
    see = j[None] < lens
    if case["window"]:
        see &= j[None] >= lens - case["window"]
    k = s["Kc"][at].permute(0, 2, 3, 1).float()
    z = torch.matmul(s["Q"].float().mul(s["scale"]).view(S, Hkv, G, dh), k)
    z.masked_fill_(~see[:, None, None], -math.inf)
    o, lse = _plain_softmax(z, s["Vc"][at].permute(0, 2, 1, 3).float())
    return o.reshape(S, Hkv * G, dh).to(s["Q"].dtype), lse.reshape(S, Hkv * G)


# ----------------------------------------------------------------------------- the framework's
def _own_rope(s):
    import chunked_weight_sequence_amd as ttt
    kw = dict(q_weight=s["q_w"], k_weight=s["k_w"], eps=1e-6, layout=s["case"]["layout"],
              rope_scale=s["rope_scale"])
    if not s["case"]["cache"]:
        return ttt.qk_norm_rope(s["Q"], s["K"], s["pos"], s["inv_freq"], **kw)
    q, k = ttt.qk_norm_rope(s["Q"], s["K"], s["pos"], s["inv_freq"], V=s["V"], K_cache=s["Kc"],
                            V_cache=s["Vc"], slots=s["slots"], **kw)
    return q, k, s["Kc"], s["Vc"]


def _own_packed(s):
    import chunked_weight_sequence_amd as ttt
    return ttt.attention_packed(s["Q"], s["K"], s["V"], s["cu_q"], s["cu_k"], scale=s["scale"],
                                window=s["case"]["window"], with_lse=True)


def _own_decode(s):
    import chunked_weight_sequence_amd as ttt
    return ttt.attention_decode(s["Q"], s["Kc"], s["Vc"], s["table"], s["lens"], s["case"]["page"],
                                scale=s["scale"], window=s["case"]["window"], with_lse=True)


def run(state):
    op = state["case"]["op"]
    if op == "rope":
        return _own_rope(state) if own else _plain_rope(state)
    if op == "packed":
        return _own_packed(state) if own else _plain_packed(state)
    return _own_decode(state) if own else _plain_decode(state)


# ---------------------------------------------------------------------------------------- work
def _visible(lq, lk, window):
    """Keys seen by all the queries of one sequence: query i sees the last min(i + 1 + lk - lq,
    window) of the keys up to its own place."""
    a, b = lk - lq + 1, lk  # the first and the last query's counts (lk >= lq here)
    if not window or window >= b:
        return lq * (a + b) // 2
    if window <= a:
        return lq * window
    ramp = window - a  # queries that see fewer than a window
    return ramp * (a + window - 1) // 2 + (lq - ramp) * window


def work(case):
    Hq, Hkv, dh = case["Hq"], case["Hkv"], case["dh"]
    if case["op"] == "rope":
        e = 2 if case["dtype"] == BF16 else 4
        heads = 2 * (Hq + Hkv) + (3 * Hkv if case["cache"] else 0)
        return {"bytes": case["N"] * (heads * dh * e + (8 if case["cache"] else 4)),
                "flops": case["N"] * (Hq + Hkv) * (3 * case["rot"] + (4 * dh if case["norm"] else 0))}
    if case["op"] == "packed":
        # the lengths of another seed differ a little; seed 0's stand for them
        lens = _lengths(case, 0)
        seen = sum(_visible(a, b, case["window"]) for a, b in lens)
        keys = sum(min(b, case["window"] + a - 1) if case["window"] and a else b for a, b in lens)
        return {"bytes": 2 * dh * (2 * case["N"] * Hq + 2 * keys * Hkv) + 4 * case["N"] * Hq,
                "flops": 4 * dh * Hq * seen}
    lens = _lengths(case, 0)
    seen = sum(min(n, case["window"]) if case["window"] else n for n in lens)
    return {"bytes": 2 * dh * (2 * case["S"] * Hq + 2 * seen * Hkv) + 4 * case["S"] * Hq,
            "flops": 4 * dh * Hq * seen}


# --------------------------------------------------------------------------------- in 64 bits
def _exact_rotated(x, w, s):
    """Norm, then each pair as a complex number times e^(i angle)."""
    case, y = s["case"], x.double()
    if w is not None:
        y = y / ((y * y).sum(-1, keepdim=True) / case["dh"] + 1e-6).sqrt() * w.double()
    angle = s["pos"].double()[:, None, None] * s["inv_freq"]
    turn = torch.polar(torch.full_like(angle, s["rope_scale"]), angle)
    half, out = case["rot"] // 2, y.clone()
    lo = slice(0, half) if case["layout"] == "half" else slice(0, case["rot"], 2)
    hi = slice(half, case["rot"]) if case["layout"] == "half" else slice(1, case["rot"], 2)
    z = torch.complex(y[..., lo].contiguous(), y[..., hi].contiguous()) * turn
    out[..., lo], out[..., hi] = z.real, z.imag
    return out


def _exact_rows(q, k, v, first, scale, window):
    """Attention of rows q [n, Hq, dh] over k, v [m, Hkv, dh]; row i stands at key first + i."""
    n, Hq, dh = q.shape
    G = Hq // k.shape[1]
    o = torch.zeros(n, Hq, dh, dtype=torch.float64, device=q.device)
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64, device=q.device)
    if n == 0 or len(k) == 0:
        return o, lse
    place = first + torch.arange(n, device=q.device)[:, None]
    behind = place - torch.arange(len(k), device=q.device)[None]
    hidden = behind < 0
    if window:
        hidden |= behind >= window
    for h in range(Hq):
        x = q[:, h].double() @ k[:, h // G].double().t() * scale
        x[hidden] = -math.inf
        lse[:, h] = torch.logsumexp(x, 1)
        o[:, h] = torch.exp(x - lse[:, h, None]).nan_to_num(0.0) @ v[:, h // G].double()
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        q, k = _exact_rotated(s["Q"], s["q_w"], s), _exact_rotated(s["K"], s["k_w"], s)
        if not case["cache"]:
            return q, k
        Kc, Vc, at = s["Kc"].double(), s["Vc"].double(), s["slots"].long()
        Kc[at], Vc[at] = k, s["V"].double()
        return q, k, Kc, Vc
    parts = []
    if case["op"] == "packed":
        a0 = b0 = 0
        for a, b in _lengths(case, seed):
            parts.append(_exact_rows(s["Q"][a0:a0 + a], s["K"][b0:b0 + b], s["V"][b0:b0 + b], b - a,
                                     s["scale"], case["window"]))
            a0, b0 = a0 + a, b0 + b
    else:
        page = case["page"]
        for r, n in enumerate(_lengths(case, seed)):
            rows = [int(p) * page + i for p in s["table"][r].tolist() for i in range(page)][:n]
            at = torch.tensor(rows, dtype=torch.long, device=s["Q"].device)
            parts.append(_exact_rows(s["Q"][r:r + 1], s["Kc"][at], s["Vc"][at], n - 1, s["scale"],
                                     case["window"]))
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
