"""A serving loop's operators as they are used together: prompts in pieces mixed with single tokens through a
block with attention and one with fast weights that forget, captured steps, streams, workspaces, offsets past 32 bits.
Tolerances as in the operators' own tests; the inputs of each stage are what the device made of the stage before, so
they do not add up."""
import numpy as np
import pytest

import chunked_weight_sequence_amd as ttt
import oracle.serving as osv
from helpers import dev, host_bits, host_f64, requires_gpu
from test_gpu_attention import _check, _draw, _f, _i32, _logit_size
from test_gpu_attention_block import _rotated
from test_gpu_add_norm import _check as _norm_check
from test_gpu_delta import EPS, _packed_check

pytestmark = [pytest.mark.gpu, requires_gpu]


def test_prompts_in_pieces_through_a_hybrid_block():
    """Three sequences, each step with other numbers of new tokens (none, one, many): the residual's norm, a product
    (plain torch), norm, rotation and cache write, attention over the pages; then the residual's norm again and the
    gated delta rule over the pool of states, by the packed call, and by the one-token call where every sequence has
    at most one. Each result against the oracle on what the device gave it."""
    import torch
    print("case: hybrid block", flush=True)
    rng = np.random.default_rng(21)
    D, Hq, Hkv, dh, page, Hk, Hv, dk, dv = 256, 4, 2, 64, 16, 2, 4, 64, 64
    S, steps = 3, [[70, 5, 0], [1, 40, 130], [1, 1, 1], [1, 0, 1], [66, 1, 1]]
    total = np.sum(steps, axis=0)
    most = int(-(-total.max() // page))
    table = rng.permutation(S * most).reshape(S, most).astype(np.int32)
    Kc = torch.full((S * most * page, Hkv, dh), float("nan"), dtype=torch.bfloat16, device="cuda")
    Vc = torch.full_like(Kc, float("nan"))
    pool = torch.zeros(S + 1, Hv, dk, dv, device="cuda")
    slots_of = [2, 0, 3]
    freq, rs = ttt.rope_frequencies(dh)
    w1, w2 = (dev(rng.uniform(0.5, 1.5, D).astype(np.float32), "f32") for _ in range(2))
    Wqkv = (torch.randn(D, (Hq + 2 * Hkv) * dh, device="cuda") / 16).bfloat16()
    Wo = (torch.randn(Hq * dh, D, device="cuda") / 16).bfloat16()
    Wd = (torch.randn(D, 2 * Hk * dk + Hv * dv, device="cuda") / 16).bfloat16()
    done = [0] * S
    for lens in steps:
        N = sum(lens)
        cu = _i32(np.concatenate([[0], np.cumsum(lens)]))
        x, r = (dev(_draw(rng, N, D), "bf16") for _ in range(2))
        before = [host_bits(t) for t in (x, r)]
        y, _, x = ttt.add_rms_norm(x, w1, residual=r, S=r)
        _norm_check((y, None, x), *before, host_f64(w1).astype(np.float32), 1e-6, "bf16")
        qkv = (y @ Wqkv).view(N, Hq + 2 * Hkv, dh)
        pos = [done[s] + i for s in range(S) for i in range(lens[s])]
        slots = [int(table[s, j // page]) * page + j % page for s in range(S) for j in range(done[s], done[s] + lens[s])]
        q, k = ttt.qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], _i32(pos), freq, rope_scale=rs, V=qkv[:, Hq + Hkv:],
                                K_cache=Kc, V_cache=Vc, slots=_i32(slots))
        want, bound = _rotated(host_bits(qkv[:, :Hq].contiguous()), None, pos, rs)
        assert (np.abs(host_f64(q) - want) <= 1.01 * bound).all()
        done = [a + b for a, b in zip(done, lens)]
        o, lse = ttt.attention_paged(q, Kc, Vc, cu, _i32(table), _i32(done), page, with_lse=True)
        torch.cuda.synchronize()
        kb, vb = host_bits(Kc), host_bits(Vc)
        want = osv.paged(_f(host_bits(q)), _f(kb), _f(vb), host_bits(cu), table, done, page, dh ** -0.5)
        _check(o, lse, want, _logit_size(_f(host_bits(q)), np.nan_to_num(_f(kb)), dh ** -0.5), dh, f"attention {lens}")
        h = o.reshape(N, Hq * dh) @ Wo
        before = [host_bits(t) for t in (h, x)]
        y, _, x = ttt.add_rms_norm(h, w2, residual=x)
        _norm_check((y, None, x), *before, host_f64(w2).astype(np.float32), 1e-6, "bf16")
        row = y @ Wd
        t = [row[:, :Hk * dk].view(N, Hk, dk), row[:, Hk * dk:2 * Hk * dk].view(N, Hk, dk), row[:, 2 * Hk * dk:].view(N, Hv, dv)]
        g = dev(-rng.uniform(0, 0.5, (N, Hv)).astype(np.float32), "f32")
        beta = dev(rng.uniform(0, 1, (N, Hv)).astype(np.float32), "f32")
        old = host_f64(pool)
        if max(lens) <= 1:
            at = [s for s in range(S) if lens[s]]
            o, st = ttt.gated_delta_decode(*t, g, beta, pool, slots=_i32([slots_of[s] for s in at]))
        else:
            o, st = ttt.gated_delta_packed(*t, g, beta, cu, state=pool, slots=_i32(slots_of))
        torch.cuda.synchronize()
        assert st is pool
        new = host_f64(pool)
        bits = [host_bits(a.contiguous()) for a in (*t, g, beta)]
        _packed_check(bits, o, lens, 0, [old[a] for a in slots_of], [new[a] for a in slots_of], dk ** -0.5, EPS)
        np.testing.assert_array_equal(new[1], old[1])  # no sequence's


def _step(rng, S, N):
    """The tensors of a step and a function that runs all operators on them."""
    import torch
    D, Hq, Hkv, dh, page, most, Hk, Hv, dk, dv = 384, 8, 2, 128, 16, 40, 2, 4, 128, 128
    table = _i32(rng.permutation(S * most).reshape(S, most))
    t = dict(x=dev(_draw(rng, N, D), "bf16"), r=dev(_draw(rng, N, D), "bf16"), w=torch.ones(D, device="cuda"),
             q=dev(_draw(rng, N, Hq, dh), "bf16"), Kc=dev(_draw(rng, S * most * page, Hkv, dh), "bf16"),
             Vc=dev(_draw(rng, S * most * page, Hkv, dh), "bf16"), cu=_i32([0] * (S + 1)), lens=_i32([0] * S),
             dq=dev(_draw(rng, N, Hk, dk), "bf16"), dk=dev(_draw(rng, N, Hk, dk), "bf16"), dv=dev(_draw(rng, N, Hv, dv), "bf16"),
             g=dev(-rng.uniform(0, 1, (N, Hv)).astype(np.float32), "f32"), b=dev(rng.uniform(0, 1, (N, Hv)).astype(np.float32), "f32"),
             state=dev(rng.standard_normal((S + 1, Hv, dk, dv)).astype(np.float32), "f32"), slots=_i32(range(S)))

    def run(**ws):
        y, sc, s = ttt.add_rms_norm(t["x"], t["w"], residual=t["r"], e4m3=True, group=128)
        z, _, _ = ttt.add_rms_norm(s, t["w"])
        o, lse = ttt.attention_paged(t["q"], t["Kc"], t["Vc"], t["cu"], table, t["lens"], page, with_lse=True,
                                     workspace=ws.get("paged"))
        d, st = ttt.gated_delta_packed(t["dq"], t["dk"], t["dv"], t["g"], t["b"], t["cu"], state=t["state"],
                                       state_out=torch.zeros_like(t["state"]), slots=t["slots"], workspace=ws.get("delta"))
        e, st2 = ttt.gated_delta_decode(t["dq"][:S], t["dk"][:S], t["dv"][:S], t["g"][:S], t["b"][:S], st,
                                        state_out=torch.zeros_like(st), slots=t["slots"])
        return y.view(torch.uint8), sc, s, z, o, lse, d, st, e, st2

    def set(new, lens, slots):
        for k in ("x", "r", "q", "dq", "dk", "dv"):
            t[k].copy_(dev(_draw(rng, *t[k].shape), "bf16"))
        t["cu"].copy_(_i32(np.concatenate([[0], np.cumsum(new)])))
        t["lens"].copy_(_i32(lens))
        t["slots"].copy_(_i32(slots))
    L = ttt.lib()
    need = dict(paged=L.ttt_attention_paged_workspace(S, N, most, page, Hq, Hkv, dh),
                delta=L.ttt_gated_delta_packed_workspace(S, N, Hk, Hv, dk, dv))
    assert all(n > 0 for n in need.values())
    return run, set, need


def _same(got, want, rows):
    """Bit for bit; of outputs by tokens the rows of sequences."""
    for i, (x, y) in enumerate(zip(got, want)):
        n = rows if i in (4, 5, 6) else len(y)
        np.testing.assert_array_equal(host_bits(x)[:n], y[:n], err_msg=f"output {i}")


def test_captured_steps_replay_with_other_batches():
    """Two graphs of all operators, replayed in turn and at once with other inputs, numbers of new tokens, lengths and
    slots, eager calls and synchronizations between; each replay has the eager call's bits."""
    import torch
    print("case: captured steps", flush=True)
    rng = np.random.default_rng(31)
    S, N = 3, 100
    two = [_step(rng, S, N) for _ in range(2)]
    graphs = []
    for run, set, _ in two:
        set([30, 1, 69], [600, 33, 69], [0, 1, 2])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            run()
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    for new, lens, slots in (([30, 1, 69], [600, 33, 69], [0, 1, 2]), ([1, 1, 1], [640, 2, 1], [3, 0, 2]),
                             ([0, 100, 0], [5, 300, 0], [1, 2, 3]), ([65, 0, 35], [65, 64, 500], [2, -1, 0])):
        want = []
        for run, set, _ in two:
            set(new, lens, slots)
            want.append([host_bits(x) for x in run()])
        torch.cuda.synchronize()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (_, out), w in zip(graphs, want):
            _same(out, w, sum(new))


def test_streams_and_given_workspaces():
    """The operators on two streams at once, each with its own workspaces whose contents are anything; workspaces that
    are too small, not aligned or of another device are refused."""
    import torch
    print("case: streams and workspaces", flush=True)
    rng = np.random.default_rng(32)
    run, set, need = _step(rng, 3, 100)
    set([30, 1, 69], [600, 33, 69], [0, 1, 2])
    want = [host_bits(x) for x in run()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [{k: torch.full((n,), 255, dtype=torch.uint8, device="cuda") for k, n in need.items()} for _ in streams]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s, w in zip(streams, ws):
            with torch.cuda.stream(s):
                got.append(run(**w))
    torch.cuda.synchronize()
    for g in got:
        _same(g, want, 100)
    for k, n in need.items():
        big = torch.empty(n + 16, dtype=torch.uint8, device="cuda")
        for bad, err in ((big[:n - 1], ttt.TTTError), (big[8:n + 8], ttt.TTTError), (torch.empty(n, dtype=torch.uint8), ValueError)):
            with pytest.raises(err):
                run(**{k: bad})


def test_the_same_bits_every_time():
    import torch
    print("case: the same call again", flush=True)
    run, set, _ = _step(np.random.default_rng(33), 3, 100)
    set([30, 1, 69], [600, 33, 69], [0, 1, 2])
    want = [host_bits(x) for x in run()]
    for _ in range(5):
        torch.cuda.synchronize()
        _same(run(), want, 100)


def test_offsets_past_32_bits():
    """Pages, states and rows that lie more than 4 GiB into their buffers."""
    import torch
    print("case: large offsets", flush=True)
    rng = np.random.default_rng(34)
    # a cache: the sequence's pages at its end
    Hq, Hkv, dh, page, n, new = 8, 8, 128, 256, 600, 70
    n_pages = (1 << 32) // (page * Hkv * dh * 2) + 9
    Kc = torch.empty(n_pages * page, Hkv, dh, dtype=torch.bfloat16, device="cuda")
    Vc = torch.empty_like(Kc)
    tb = [n_pages - 2, 0, n_pages - 1]
    k, v = _draw(rng, 3 * page, Hkv, dh), _draw(rng, 3 * page, Hkv, dh)
    for i, p in enumerate(tb):
        Kc[p * page:(p + 1) * page] = dev(k[i * page:(i + 1) * page], "bf16")
        Vc[p * page:(p + 1) * page] = dev(v[i * page:(i + 1) * page], "bf16")
    q = _draw(rng, new, Hq, dh)
    O, L = ttt.attention_paged(dev(q, "bf16"), Kc, Vc, _i32([0, new]), _i32([tb]), _i32([n]), page, with_lse=True)
    torch.cuda.synchronize()
    want = osv.paged(_f(q), _f(k), _f(v), [0, new], np.array([[0, 1, 2]]), [n], page, dh ** -0.5)
    _check(O, L, want, _logit_size(_f(q), _f(k), dh ** -0.5), dh, "pages")
    del Kc, Vc, O, L
    torch.cuda.empty_cache()
    # a pool of states, rows of queries, keys and values far apart, outputs too
    Hk, Hv, dk, dv, N, far = 1, 2, 128, 128, 70, 1 << 23
    slots = (1 << 32) // (Hv * dk * dv * 4) + 5
    pool = torch.zeros(slots, Hv, dk, dv, device="cuda")
    W = rng.standard_normal((2, Hv, dk, dv)).astype(np.float32)
    pool[slots - 1], pool[slots - 3] = dev(W[0], "f32"), dev(W[1], "f32")
    x = [_draw(rng, N, h, w) for h, w in ((Hk, dk), (Hk, dk), (Hv, dv))]
    x += [-rng.uniform(0, 0.1, (N, Hv)).astype(np.float32), rng.uniform(0, 1, (N, Hv)).astype(np.float32)]
    buf = [torch.empty((N - 1) * far + 1024, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    t = [buf[0].as_strided((N, h, w), (far, w, 1), o) for h, w, o in ((Hk, dk, 0), (Hk, dk, 128), (Hv, dv, 256))]
    for a, b in zip(t, x):
        a.copy_(dev(b, "bf16"))
    O = buf[1].as_strided((N, Hv, dv), (far, dv, 1), 0)
    gb = [dev(a, "f32") for a in x[3:]]
    ttt.gated_delta_packed(*t, *gb, _i32([0, 66, N]), state=pool, slots=_i32([slots - 1, slots - 3]), O=O)
    torch.cuda.synchronize()
    end = host_f64(pool[[slots - 1, slots - 3]])
    _packed_check(x, O.contiguous(), [66, 4], 0, [W[0], W[1]], [end[0], end[1]], dk ** -0.5, EPS)
    pool[slots - 1] = dev(W[0], "f32")
    ttt.gated_delta_decode(*[a[N - 1:] for a in t], *[a[N - 1:].clone() for a in gb], pool, slots=_i32([slots - 1]), O=O[N - 1:])
    torch.cuda.synchronize()
    _packed_check([a[N - 1:] for a in x], O[N - 1:].contiguous(), [1], 0, [W[0]], [host_f64(pool[slots - 1])], dk ** -0.5, EPS)
    del pool, buf, t, O
    torch.cuda.empty_cache()
    # rows of the residual stream
    N, D = 140000, 16384
    X = torch.empty(N, D, dtype=torch.bfloat16, device="cuda")
    x = _draw(rng, 3, D)
    X[-3:] = dev(x, "bf16")
    Y, sc, _ = ttt.add_rms_norm(X, e4m3=True)
    torch.cuda.synchronize()
    _norm_check((Y[-3:], sc[-3:], None), x, None, None, 1e-6, "bf16", 0)


def test_very_many_sequences():
    """Past 64, past a wave's search, with empty ones among them: pages and states."""
    import torch
    print("case: thousands of sequences", flush=True)
    rng = np.random.default_rng(35)
    n, page, Hq, Hkv, dh = 5000, 16, 2, 1, 64
    new = rng.integers(0, 4, n)
    lens = new + rng.integers(0, 5, n)
    held = -(-lens // page)
    table = np.where(held > 0, np.cumsum(held) - held, -1).astype(np.int32)[:, None]
    K, V = (_draw(rng, int(held.sum()) * page, Hkv, dh) for _ in range(2))
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    Q = _draw(rng, int(cu[-1]), Hq, dh)
    O, L = ttt.attention_paged(dev(Q, "bf16"), dev(K, "bf16"), dev(V, "bf16"), _i32(cu), _i32(table), _i32(lens), page,
                               with_lse=True)
    torch.cuda.synchronize()
    rows = np.unique(np.concatenate([rng.choice(cu[-1], 300, replace=False), [0, cu[-1] - 1]]))
    o, lse, a = osv.paged(_f(Q), _f(K), _f(V), cu, table, lens, page, dh ** -0.5, 0, set(rows.tolist()))
    _check(O[rows], L[rows], (o[rows], lse[rows], a[rows]), _logit_size(_f(Q)[rows], _f(K), dh ** -0.5), dh, "many")
    Hk, Hv, dk, dv = 1, 1, 64, 64
    x = [_draw(rng, int(cu[-1]), 1, 64) for _ in range(3)]
    x += [-rng.uniform(0, 1, (int(cu[-1]), 1)).astype(np.float32), rng.uniform(0, 1, (int(cu[-1]), 1)).astype(np.float32)]
    W = rng.standard_normal((n, Hv, dk, dv)).astype(np.float32)
    t = [dev(a, "bf16") for a in x[:3]] + [dev(a, "f32") for a in x[3:]]
    O, st = ttt.gated_delta_packed(*t, _i32(cu), state=dev(W, "f32"))
    torch.cuda.synchronize()
    st = host_f64(st)
    np.testing.assert_array_equal(st[new == 0], W[new == 0])
    for s in rng.choice(n, 60, replace=False):
        part = [a[cu[s]:cu[s + 1]] for a in x]
        _packed_check(part, O[cu[s]:cu[s + 1]], [int(new[s])], 0, [W[s]], [st[s]], dk ** -0.5, EPS)
    at = _i32(rng.permutation(n))
    O, st2 = ttt.gated_delta_decode(*[a[:n] for a in t], dev(W, "f32"), slots=at) if cu[-1] >= n else (None, None)
    if O is not None:
        torch.cuda.synchronize()
        st2, at = host_f64(st2), host_bits(at)
        for s in rng.choice(n, 60, replace=False):
            _packed_check([a[s:s + 1] for a in x], O[s:s + 1], [1], 0, [W[at[s]]], [st2[at[s]]], dk ** -0.5, EPS)
