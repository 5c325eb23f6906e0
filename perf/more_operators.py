"""Cases of what a step of a serving loop takes beside the scan: the norm between the halves of a block,
attention of new tokens over a paged cache, and the gated delta rule over a prompt and token by token.

`run` computes a case in its plain form (elementary torch operations in 32 bits, rounded once), or
through the framework's entry points where `own` is true. `exact` gives the 64-bit results.
"""
import math

import torch

own = False

BF16, F32, E4M3 = "bf16", "f32", "e4m3"
_TYPES = {BF16: torch.bfloat16, F32: torch.float32}
EPS = 1e-6
CHUNK = 64  # tokens that the plain form of the delta rule takes at a time


# ------------------------------------------------------------------------------------- the cases
def _norm(**kw):
    return dict(dict(op="norm", dtype=BF16, out=BF16, group=0, residual=True), **kw)


def _paged(**kw):
    return dict(dict(op="paged", Hq=32, Hkv=8, dh=128, S=1, window=0, page=64, lengths="alike"), **kw)


def _delta(**kw):
    return dict(dict(op="delta", Hk=16, Hv=32, dk=128, dv=128, docs=1, fresh=False), **kw)


def _step(**kw):
    return dict(dict(op="step", Hk=16, Hv=32, dk=128, dv=128), **kw)


def listed():
    return [
        # one token of the 2560 / 9728 block: the smallest call of a generating loop
        _norm(name="norm_1", N=1, D=2560),
        # the tokens of an fp32 model whose width is no multiple of a workgroup's share
        _norm(name="norm_4099_f32", N=4099, D=1000, dtype=F32, out=F32),
        # a prompt of the scan's length, made ready for a product in 8 bits
        _norm(name="norm8_32768", N=32768, D=2560, out=E4M3, group=128),
        # a few drafted tokens of each of 16 streams, to be checked at once, in small pages
        _paged(name="paged_drafts", S=16, new=5, L=8000, Hq=16, Hkv=4, dh=64, page=16, lengths="ragged"),
        # one piece of a long prompt
        _paged(name="paged_512_past", new=512, L=16384),
        # a serving batch: a piece of a prompt beside streams that take one token each, one of them idle
        _paged(name="paged_mixed", S=16, new=512, L=12000, page=32, lengths="mixed"),
        # pieces of four prompts under a sliding window
        _paged(name="paged_window", S=4, new=2000, L=8000, Hq=32, Hkv=32, dh=64, window=2048, page=256),
        # a short prompt at the routing workload's heads
        _delta(name="delta_77", N=77, Hk=16, Hv=16, dk=64, dv=64, fresh=True),
        # documents of different lengths, packed
        _delta(name="delta_8192_docs", N=8192, docs=11),
        # one long document that goes on from a state
        _delta(name="delta_32768", N=32768, Hk=32),
        # a single stream
        _step(name="step_1", S=1),
        # a serving batch
        _step(name="step_64", S=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "paged", "paged", "delta", "delta", "step"])
    if op == "norm":
        D = 8 * _log(rng, 16, 1280)
        dtype, out = rng.choice([(BF16, BF16), (F32, F32), (BF16, E4M3), (F32, E4M3)])
        group = rng.choice([0, 32, 128]) if out == E4M3 else 0
        if group:
            D = -(-D // group) * group
        N = _log(rng, 1, 32768 * 2560 // D // (2 if dtype == F32 else 1))
        return _norm(N=N, D=D, dtype=dtype, out=out, group=group, residual=rng.random() < 0.8)
    if op == "paged":
        dh = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8, 16])
        Hq = Hkv * rng.choice([g for g in (1, 2, 3, 4, 7, 8) if g * Hkv <= 32])
        S = _log(rng, 1, 32)
        lengths = rng.choice(["alike", "ragged", "mixed"]) if S > 1 else "alike"
        new = _log(rng, 1, 8000 // (1 if lengths == "mixed" else S))
        L = max(new, _log(rng, 16, min(16384, 100000000 // (S * new))))
        return _paged(S=S, new=new, L=L, Hq=Hq, Hkv=Hkv, dh=dh, lengths=lengths,
                      window=rng.choice([0, 0, 0, 128, 1000, 4096]), page=rng.choice([16, 32, 64, 256]))
    dk, dv = rng.choice([(64, 64), (128, 128), (128, 128), (64, 128), (128, 64)])
    Hk = rng.choice([1, 2, 4, 8, 16])
    Hv = Hk * rng.choice([1, 1, 2])
    if op == "delta":
        N = _log(rng, 1, 32768 * 16 // max(16, Hv))
        return _delta(N=N, Hk=Hk, Hv=Hv, dk=dk, dv=dv, docs=1 if N < 64 else rng.choice([1, 1, 2, 5, 16, 40]),
                      fresh=rng.random() < 0.5)
    return _step(S=_log(rng, 1, 2048 // Hv), Hk=Hk, Hv=Hv, dk=dk, dv=dv)


# ------------------------------------------------------------------------------------ the inputs
def _lengths(case, seed):
    """Host lengths of a case, from its seed: [(new tokens, tokens with them)] of the paged sequences (how many
    are new goes by the case alone), or the tokens of the packed documents."""
    g = torch.Generator().manual_seed(7919 * seed + 29)

    def some(lo, hi):
        return int(torch.randint(lo, hi + 1, (1,), generator=g))

    if case["op"] == "delta":
        cuts = sorted(some(0, case["N"]) for _ in range(case["docs"] - 1))
        cuts = [0] + cuts + [case["N"]]
        return [b - a for a, b in zip(cuts, cuts[1:])]
    S, new, L = case["S"], case["new"], case["L"]
    if case["lengths"] == "alike":
        return [(new, L)] * S
    if case["lengths"] == "mixed":  # one piece, single tokens, and (of several) one with nothing new
        lens = [(new, L)] + [(1, some(1, L)) for _ in range(S - 1)]
        return lens[:-1] + [(0, lens[-1][1])] if S > 2 else lens
    fixed = torch.Generator().manual_seed(31 * new + S)
    counts = torch.randint(1, new + 1, (S,), generator=fixed).tolist()
    return [(new, L)] + [(n, some(n, L)) for n in counts[1:]]


def _cumulative(lens, device):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=device)


def prepare(case, seed):
    d = torch.device("cuda:0")
    g = torch.Generator(device=d).manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, by=1.0):
        return (torch.randn(shape, generator=g, device=d) * by).to(dtype)

    if case["op"] == "norm":
        N, D, t = case["N"], case["D"], _TYPES[case["dtype"]]
        # some channels of a residual stream are far larger than the others
        size = 1.0 + 20.0 * (torch.rand(D, generator=g, device=d) < 0.005)
        return dict(case=case, X=normal(N, D, dtype=t, by=0.5),
                    R=(torch.randn(N, D, generator=g, device=d) * size).to(t) if case["residual"] else None,
                    w=1.0 + 0.2 * torch.randn(D, generator=g, device=d))
    if case["op"] == "paged":
        Hq, Hkv, dh, page = case["Hq"], case["Hkv"], case["dh"], case["page"]
        lens = _lengths(case, seed)
        most = -(-max(n for _, n in lens) // page)
        held = [-(-n // page) for _, n in lens]
        n_pages = sum(held) + 3
        order = torch.randperm(n_pages, generator=g, device=d).to(torch.int32)
        held = torch.tensor(held, device=d)
        at, k = torch.cumsum(held, 0) - held, torch.arange(most, device=d)
        table = order[(at[:, None] + k[None]).clamp(max=n_pages - 1)]
        table = torch.where(k[None] < held[:, None], table, torch.full_like(table, -1))
        return dict(case=case, Q=normal(sum(n for n, _ in lens), Hq, dh),
                    Kc=normal(n_pages * page, Hkv, dh), Vc=normal(n_pages * page, Hkv, dh),
                    table=table.contiguous(), cu=_cumulative([n for n, _ in lens], d), most_new=max(n for n, _ in lens),
                    lens=torch.tensor([n for _, n in lens], dtype=torch.int32, device=d), scale=dh ** -0.5)
    Hk, Hv, dk, dv = case["Hk"], case["Hv"], case["dk"], case["dv"]
    lens = _lengths(case, seed) if case["op"] == "delta" else [1] * case["S"]
    N, S = sum(lens), len(lens)
    # queries, keys and values of a token in a row, as the projections leave them; the keys of a head have
    # a direction in common
    row = torch.randn(N, 2 * Hk * dk + Hv * dv, generator=g, device=d)
    row[:, Hk * dk:2 * Hk * dk] += 0.5 * torch.randn(Hk * dk, generator=g, device=d)
    row = row.to(torch.bfloat16)
    # heads forget at rates from 1e-3 to 1 a token
    rate = torch.exp(torch.rand(Hv, generator=g, device=d) * math.log(1e3) - math.log(1e3))
    s = dict(case=case, Q=row[:, :Hk * dk].view(N, Hk, dk), K=row[:, Hk * dk:2 * Hk * dk].view(N, Hk, dk),
             V=row[:, 2 * Hk * dk:].view(N, Hv, dv),
             g=-rate * torch.nn.functional.softplus(torch.randn(N, Hv, generator=g, device=d)),
             beta=torch.sigmoid(torch.randn(N, Hv, generator=g, device=d)), scale=dk ** -0.5, state=None)
    # a pool of states and its copy for the step in flight, so that a step can be taken back
    n_slots = S + 2
    s["slots"] = torch.randperm(n_slots, generator=g, device=d)[:S].to(torch.int32)
    if case["op"] == "step" or not case["fresh"]:
        s["state"] = 0.3 * torch.randn(n_slots, Hv, dk, dv, generator=g, device=d)
    s["state_out"] = torch.zeros(n_slots, Hv, dk, dv, device=d)
    if case["op"] == "delta":
        s["cu"], s["most"] = _cumulative(lens, d), max(lens)
    return s


# --------------------------------------------------------------------------------- plain forms
def _plain_norm(s):
    case, X, R = s["case"], s["X"], s["R"]
    h = X.float() if R is None else X.float() + R.float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["w"]
    total = [] if R is None else [h.to(X.dtype)]
    if case["out"] != E4M3:
        return [y.to(X.dtype)] + total
    N, D = y.shape
    y = y.view(N, -1, case["group"] or D)
    scales = (y.abs().amax(-1) / 448.0).clamp(min=2.0 ** -126)
    return [(y / scales[..., None]).view(N, D).to(torch.float8_e4m3fn), scales] + total


def _plain_paged(s):
    case = s["case"]
    Hkv, G, dh, S, page = case["Hkv"], case["Hq"] // case["Hkv"], case["dh"], case["S"], case["page"]
    nq, cu, lens = s["most_new"], s["cu"].long(), s["lens"].long()
    most = s["table"].shape[1] * page
    i, j = torch.arange(nq, device=cu.device), torch.arange(most, device=cu.device)
    new = cu[1:] - cu[:-1]
    here = i[None] < new[:, None]  # [S, nq]
    place = i[None] + (lens - new)[:, None]  # of a query among its sequence's tokens
    see = (j[None, None] <= place[..., None]) & (j[None, None] < lens[:, None, None])
    if case["window"]:
        see &= j[None, None] > place[..., None] - case["window"]
    at_q = (cu[:-1, None] + i[None]).clamp(max=len(s["Q"]) - 1)
    at = s["table"].long()[:, j // page].clamp(min=0) * page + j % page  # [S, most]
    q = s["Q"][at_q].float().mul(s["scale"]).view(S, nq, Hkv, G, dh).permute(0, 2, 3, 1, 4)
    q = q.reshape(S * Hkv, G * nq, dh)
    k = s["Kc"][at].permute(0, 2, 3, 1).float().contiguous().view(S * Hkv, dh, most)
    v = s["Vc"][at].permute(0, 2, 1, 3).float().contiguous().view(S * Hkv, most, dh)
    z = torch.matmul(q, k).view(S, Hkv, G, nq, most).masked_fill_(~see[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = z.sub_(m).exp_()
    n = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(S * Hkv, G * nq, most), v).view(S, Hkv, G, nq, dh)
    o = (o / torch.where(n == 0, torch.ones_like(n), n)).permute(0, 3, 1, 2, 4)
    lse = (m + n.log()).squeeze(-1).permute(0, 3, 1, 2)
    return o[here].reshape(-1, Hkv * G, dh).to(s["Q"].dtype), lse[here].reshape(-1, Hkv * G).contiguous()


def _unit(x):
    x = x.float()
    return x * torch.rsqrt(x.square().sum(-1, keepdim=True) + EPS)


def _unit_lower_inverse(a):
    """The inverse of 1 + a, a [.., n, n] strictly lower triangular, n a power of two: of blocks of twice the
    size each time, whose lower left part is - (lower right) a (upper left)."""
    *lead, n, _ = a.shape
    out = torch.eye(n, device=a.device).expand(a.shape).contiguous()
    size = 1
    while size < n:
        blocks = out.view(*lead, n // (2 * size), 2 * size, n // (2 * size), 2 * size)
        src = a.view(*lead, n // (2 * size), 2 * size, n // (2 * size), 2 * size)
        k = torch.arange(n // (2 * size), device=a.device)
        dims = len(lead)
        x = blocks.movedim(dims + 2, dims + 1)[..., k, k, :, :]
        y = src.movedim(dims + 2, dims + 1)[..., k, k, size:, :size]
        low = -torch.matmul(torch.matmul(x[..., size:, size:], y), x[..., :size, :size])
        blocks.movedim(dims + 2, dims + 1)[..., k, k, size:, :size] = low
        size *= 2
    return out


def _plain_delta(s):
    """Chunk by chunk: inside a chunk the updates u solve a triangular system, so that only the state goes
    from chunk to chunk. Sequences side by side, padded with tokens that change nothing."""
    case = s["case"]
    Hk, Hv, dk, dv, S = case["Hk"], case["Hv"], case["dk"], case["dv"], len(s["cu"]) - 1
    cu, dev, C = s["cu"].long(), s["cu"].device, CHUNK
    nc = max(1, -(-s["most"] // C))
    i = torch.arange(nc * C, device=dev)
    here = i[None] < (cu[1:] - cu[:-1])[:, None]  # [S, nc C]
    at = (cu[:-1, None] + i[None]).clamp(max=case["N"] - 1)

    def laid(x, heads):  # [N, heads, w] -> [S, Hv, nc, C, w]
        x = x.repeat_interleave(Hv // heads, 1) if heads != Hv else x
        x = torch.where(here[..., None, None], x[at], torch.zeros((), device=dev))
        return x.view(S, nc, C, Hv, -1).permute(0, 3, 1, 2, 4).contiguous()

    q, k = laid(_unit(s["Q"]) * s["scale"], Hk), laid(_unit(s["K"]), Hk)
    v, beta = laid(s["V"].float(), Hv), laid(s["beta"][..., None], Hv)
    # sums of a chunk's gates in 64 bits, since their differences are what counts
    G = laid(s["g"][..., None].double(), Hv).squeeze(-1).cumsum(-1)
    low = torch.ones(C, C, dtype=torch.bool, device=dev).tril()
    decay = torch.where(low, (G[..., :, None] - G[..., None, :]).float(), -math.inf).exp()
    kt = k.transpose(-1, -2).contiguous()
    inner = torch.matmul(q, kt) * decay
    a = torch.matmul(k, kt).mul_(decay).mul_(beta).tril_(-1)
    solve = _unit_lower_inverse(a) * beta.transpose(-1, -2)
    since, left = G.float().exp()[..., None], (G[..., -1:] - G).float().exp()[..., None]
    whole = G[..., -1].float().exp()[..., None, None]
    kt = kt * left.transpose(-1, -2)
    at_slot = s["slots"].long()
    W = torch.zeros(S, Hv, dk, dv, device=dev) if s["state"] is None else s["state"][at_slot]
    o = torch.empty(S, Hv, nc, C, dv, device=dev)
    for c in range(nc):
        u = torch.matmul(solve[:, :, c], v[:, :, c] - since[:, :, c] * torch.matmul(k[:, :, c], W))
        o[:, :, c] = since[:, :, c] * torch.matmul(q[:, :, c], W) + torch.matmul(inner[:, :, c], u)
        W = whole[:, :, c] * W + torch.matmul(kt[:, :, c], u)
    s["state_out"].index_copy_(0, at_slot, W)
    o = o.view(S, Hv, nc * C, dv).transpose(1, 2)[here]
    return o.to(s["Q"].dtype), s["state_out"]


def _plain_step(s):
    case, at = s["case"], s["slots"].long()
    rep = case["Hv"] // case["Hk"]
    q = (_unit(s["Q"]) * s["scale"]).repeat_interleave(rep, 1)[:, :, None]
    k = _unit(s["K"]).repeat_interleave(rep, 1)
    W = s["state"][at] * s["g"].exp()[..., None, None]
    u = s["beta"][..., None] * (s["V"].float() - torch.matmul(k[:, :, None], W).squeeze(2))
    W = W + k[..., None] * u[:, :, None]
    s["state_out"].index_copy_(0, at, W)
    return torch.matmul(q, W).squeeze(2).to(s["Q"].dtype), s["state_out"]


# ----------------------------------------------------------------------------- the framework's
def _own_norm(s):
    import chunked_weight_sequence_amd as ttt
    case = s["case"]
    got = ttt.add_rms_norm(s["X"], s["w"], residual=s["R"], eps=EPS, e4m3=case["out"] == E4M3,
                           group=case["group"])
    # one scale a row comes as [N]; the plain form's are [N, groups]
    return [x if x.dim() == 2 else x[:, None] for x in got if x is not None]


def _own_paged(s):
    import chunked_weight_sequence_amd as ttt
    return ttt.attention_paged(s["Q"], s["Kc"], s["Vc"], s["cu"], s["table"], s["lens"], s["case"]["page"],
                               scale=s["scale"], window=s["case"]["window"], with_lse=True)


def _own_delta(s):
    import chunked_weight_sequence_amd as ttt
    return ttt.gated_delta_packed(s["Q"], s["K"], s["V"], s["g"], s["beta"], s["cu"], state=s["state"],
                                  state_out=s["state_out"], slots=s["slots"], scale=s["scale"], norm_eps=EPS)


def _own_step(s):
    import chunked_weight_sequence_amd as ttt
    return ttt.gated_delta_decode(s["Q"], s["K"], s["V"], s["g"], s["beta"], s["state"],
                                  state_out=s["state_out"], slots=s["slots"], scale=s["scale"], norm_eps=EPS)


def run(state):
    op = state["case"]["op"]
    if op == "norm":
        return _own_norm(state) if own else _plain_norm(state)
    if op == "paged":
        return _own_paged(state) if own else _plain_paged(state)
    if op == "delta":
        return _own_delta(state) if own else _plain_delta(state)
    return _own_step(state) if own else _plain_step(state)


# ---------------------------------------------------------------------------------------- work
def _visible(lq, lk, window):
    """Keys seen by all the queries of one sequence whose last query stands at its last key."""
    a, b = lk - lq + 1, lk  # the first and the last query's counts (lk >= lq here)
    if not window or window >= b:
        return lq * (a + b) // 2
    if window <= a:
        return lq * window
    ramp = window - a  # queries that see fewer than a window
    return ramp * (a + window - 1) // 2 + (lq - ramp) * window


def work(case):
    if case["op"] == "norm":
        N, D, e = case["N"], case["D"], 2 if case["dtype"] == BF16 else 4
        out = D + 4 * (D // case["group"] if case["group"] else 1) if case["out"] == E4M3 else D * e
        return {"bytes": N * (D * e * (3 if case["residual"] else 1) + out) + 4 * D,
                "flops": N * D * (7 if case["out"] == E4M3 else 5)}
    if case["op"] == "paged":
        # the lengths of another seed differ a little; seed 0's stand for them
        Hq, Hkv, dh, w, lens = case["Hq"], case["Hkv"], case["dh"], case["window"], _lengths(case, 0)
        seen = sum(_visible(a, b, w) for a, b in lens)
        keys = sum(min(b, w + a - 1) if w else b for a, b in lens if a)
        rows = sum(a for a, _ in lens)
        return {"bytes": 2 * dh * (2 * rows * Hq + 2 * keys * Hkv) + 4 * rows * Hq, "flops": 4 * dh * Hq * seen}
    Hk, Hv, dk, dv = case["Hk"], case["Hv"], case["dk"], case["dv"]
    N, S = (case["S"],) * 2 if case["op"] == "step" else (case["N"], case["docs"])
    states = 1 if case["op"] == "delta" and case["fresh"] else 2
    # a token: the decay, the state's answer to the key, its update, its answer to the query
    return {"bytes": N * (4 * Hk * dk + 4 * Hv * dv + 8 * Hv) + 4 * states * S * Hv * dk * dv,
            "flops": 7 * N * Hv * dk * dv}


# --------------------------------------------------------------------------------- in 64 bits
def _exact_paged(s, case, lens):
    Hq, G, page, parts, a0 = case["Hq"], case["Hq"] // case["Hkv"], case["page"], [], 0
    for r, (a, n) in enumerate(lens):
        pages = s["table"][r, :-(-n // page)].long()
        rows = (pages[:, None] * page + torch.arange(page, device=pages.device)).flatten()[:n]
        k, v, q = s["Kc"][rows], s["Vc"][rows], s["Q"][a0:a0 + a]
        behind = (n - a + torch.arange(a, device=rows.device))[:, None] - torch.arange(n, device=rows.device)
        hidden = behind < 0
        if case["window"]:
            hidden |= behind >= case["window"]
        o = torch.zeros(a, Hq, case["dh"], dtype=torch.float64, device=rows.device)
        lse = torch.zeros(a, Hq, dtype=torch.float64, device=rows.device)
        for h in range(Hq):
            x = (q[:, h].double() @ k[:, h // G].double().t() * s["scale"]).masked_fill_(hidden, -math.inf)
            lse[:, h] = torch.logsumexp(x, 1)
            o[:, h] = torch.exp(x - lse[:, h, None]) @ v[:, h // G].double()
        parts.append((o, lse))
        a0 += a
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def _exact_delta(s, case, lens):
    """Token by token, the sequences side by side."""
    rep, at = case["Hv"] // case["Hk"], s["slots"].long()
    q, k = s["Q"].double(), s["K"].double()
    q = (q / ((q * q).sum(-1, keepdim=True) + EPS).sqrt()).repeat_interleave(rep, 1) * s["scale"]
    k = (k / ((k * k).sum(-1, keepdim=True) + EPS).sqrt()).repeat_interleave(rep, 1)
    v, beta, keep = s["V"].double(), s["beta"].double(), s["g"].double().exp()
    pool = s["state_out"].double()
    W = torch.zeros_like(pool[at]) if s["state"] is None else s["state"][at].double()
    o = torch.zeros(v.shape, dtype=torch.float64, device=v.device)
    order = sorted(range(len(lens)), key=lambda r: -lens[r])  # the longest first
    start = [sum(lens[:r]) for r in order]
    W = W[torch.tensor(order, device=W.device)]
    rows = torch.tensor(start, device=W.device)
    for t in range(max(lens)):
        n = sum(1 for x in lens if x > t)
        i, w = rows[:n] + t, W[:n]
        w = w * keep[i][..., None, None]
        u = beta[i][..., None] * (v[i] - (k[i][..., None] * w).sum(2))
        w = w + k[i][..., None] * u[:, :, None]
        o[i] = (q[i][..., None] * w).sum(2)
        W[:n] = w
    pool[at[torch.tensor(order, device=at.device)]] = W
    return o, pool


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["X"].double()
        total = []
        if s["R"] is not None:
            h = h + s["R"].double()
            total = [h]
        y = h / ((h * h).sum(-1, keepdim=True) / case["D"] + EPS).sqrt() * s["w"].double()
        if case["out"] != E4M3:
            return [y] + total
        parts = y.reshape(case["N"], -1, case["group"] or case["D"])
        scales = parts.abs().amax(-1) / 448
        return [(parts / scales[..., None]).reshape(y.shape), scales] + total
    if case["op"] == "paged":
        return _exact_paged(s, case, _lengths(case, seed))
    return _exact_delta(s, case, _lengths(case, seed) if case["op"] == "delta" else [1] * case["S"])
