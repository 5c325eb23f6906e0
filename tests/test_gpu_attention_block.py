"""GPU tests of norm and rotation, packed and one-token attention as they are used together: a
prompt in pieces through a paged cache and the tokens after it, streams, workspaces, captured graphs,
caches whose offsets pass 32 bits. Tolerances as in test_gpu_attention.py; the inputs of each stage are
what the device made of the stage before, so they do not add up."""
import numpy as np
import pytest

import chunked_weight_sequence_amd as ttt
import oracle.attention as oa
from helpers import dev, host_bits, host_f64, requires_gpu
from test_gpu_attention import _check, _draw, _f, _i32, _logit_size, _some_rows

pytestmark = [pytest.mark.gpu, requires_gpu]

THETA, EPS = 10000.0, 1e-6


def _rotated(x, w, pos, scale):
    """The oracle's norm and rotation of bf16 bits, and the bound of a bf16 result: half a step, and
    the fp32 arithmetic before it (40 half steps of the pair's size)."""
    freq, _ = oa.rope_frequencies(x.shape[-1], THETA)
    y = oa.norm_rope(_f(x), w, EPS, pos, freq, "half", scale)
    half = x.shape[-1] // 2
    size = np.hypot(y[..., :half], y[..., half:])
    return y, 2.0 ** -8 * np.abs(y) + 40 * 2.0 ** -24 * np.concatenate([size, size], -1) + 1e-38


@pytest.mark.parametrize("Hq,Hkv,dh,page,window", [(8, 2, 128, 16, 0), (4, 4, 64, 64, 0),
                                                   (6, 1, 64, 32, 100)])
def test_prompts_in_pieces_then_tokens(Hq, Hkv, dh, page, window):
    """Three sequences: prompts in two pieces (the second attends to what the first left in the cache,
    gathered by slot), then three single tokens; the rows of the fused projection go in as slices."""
    import torch
    print(f"case: block {Hq}/{Hkv}x{dh} page={page} window={window}", flush=True)
    rng = np.random.default_rng(Hq + dh)
    first, second = [130, 1, 64], [70, 40, 5]
    S, W = 3, (Hq + 2 * Hkv) * dh
    most = (max(first) + max(second) + 3 + page - 1) // page
    table = rng.permutation(S * most).reshape(S, most).astype(np.int32)
    freq, rs = ttt.rope_frequencies(dh, THETA)
    wq, wk = (rng.uniform(0.5, 1.5, dh).astype(np.float32) for _ in range(2))
    wqd, wkd = dev(wq, "f32"), dev(wk, "f32")
    Kc = torch.full((S * most * page, Hkv, dh), float("nan"), dtype=torch.bfloat16, device="cuda")
    Vc = torch.full_like(Kc, float("nan"))
    done = [0, 0, 0]
    seen = [[np.zeros((0, Hkv, dh), np.uint16)] * 2 for _ in range(S)]  # K, V of each sequence

    def slot(s, j):
        return int(table[s, j // page]) * page + j % page

    def step(lens):
        N = sum(lens)
        row = _draw(rng, N + 1, W)  # one padding token at the end
        R = dev(row, "bf16")
        q, k, v = (R[:, a * dh:b * dh].view(N + 1, b - a, dh) for a, b in
                   ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
        pos = [done[s] + i for s in range(S) for i in range(lens[s])] + [0]
        slots = [slot(s, done[s] + i) for s in range(S) for i in range(lens[s])] + [-1]
        ttt.qk_norm_rope(q, k, _i32(pos), freq, q_weight=wqd, k_weight=wkd, eps=EPS, rope_scale=rs,
                         V=v, K_cache=Kc, V_cache=Vc, slots=_i32(slots), Q_out=q, K_out=k)
        torch.cuda.synchronize()
        x = row.reshape(N + 1, -1, dh)
        for got, src, w in ((q, x[:, :Hq], wq), (k, x[:, Hq:Hq + Hkv], wk)):
            want, bound = _rotated(src, w, pos, rs)
            assert (np.abs(host_f64(got) - want) <= 1.01 * bound).all()
        kb, vb = host_bits(k.contiguous()), host_bits(v.contiguous())
        np.testing.assert_array_equal(host_bits(Kc)[slots[:-1]], kb[:-1])
        np.testing.assert_array_equal(host_bits(Vc)[slots[:-1]], vb[:-1])
        at = 0
        for s in range(S):
            seen[s] = [np.concatenate([seen[s][0], kb[at:at + lens[s]]]),
                       np.concatenate([seen[s][1], vb[at:at + lens[s]]])]
            done[s] += lens[s]
            at += lens[s]
        return q, host_bits(q.contiguous())

    def want(qb, cu):
        ks, vs = (np.concatenate([seen[s][i] for s in range(S)]) for i in range(2))
        return (oa.packed(_f(qb), _f(ks), _f(vs), cu, np.cumsum([0] + done), dh ** -0.5, window),
                _logit_size(_f(qb), _f(ks), dh ** -0.5))

    for lens in (first, second):
        q, qb = step(lens)
        cu = np.cumsum([0] + lens)
        rows = torch.tensor([slot(s, j) for s in range(S) for j in range(done[s])], device="cuda")
        O = torch.full((sum(lens) + 1, Hq, dh), 7.0, dtype=torch.bfloat16, device="cuda")
        _, L = ttt.attention_packed(q, Kc[rows], Vc[rows], _i32(cu), _i32(np.cumsum([0] + done)),
                                    window=window, O=O, with_lse=True)
        torch.cuda.synchronize()
        assert (O[-1] == 7).all()  # the padding token is of no sequence
        w, X = want(qb[:-1], cu)
        _check(O[:-1], L[:-1], w, X, dh, "prompt")
    for _ in range(3):
        q, qb = step([1, 1, 1])
        O, L = ttt.attention_decode(q[:3], Kc, Vc, _i32(table), _i32(done), page, window=window,
                                    with_lse=True)
        torch.cuda.synchronize()
        w, X = want(qb[:-1], np.arange(4))
        _check(O, L, w, X, dh, "token")


def test_a_captured_token_step_replays_with_other_lengths():
    """Norm, rotation, cache write and attention of one token per sequence in a graph, replayed with
    other inputs, positions, slots and lengths, with eager calls and synchronizations between; a second
    graph of the same step shares nothing with it."""
    import torch
    print("case: captured token step", flush=True)
    S, Hq, Hkv, dh, page, most = 3, 8, 2, 128, 16, 40
    rng = np.random.default_rng(1)
    freq, rs = ttt.rope_frequencies(dh, THETA)
    table = _i32(rng.permutation(S * most).reshape(S, most))

    class Step:
        def __init__(self):
            self.Kc = dev(_draw(rng, S * most * page, Hkv, dh), "bf16")
            self.Vc = dev(_draw(rng, S * most * page, Hkv, dh), "bf16")
            self.x = torch.empty(S, Hq + 2 * Hkv, dh, dtype=torch.bfloat16, device="cuda")
            self.pos, self.slots, self.lens = (_i32([0] * S) for _ in range(3))

        def run(self, Kc, Vc):
            q, k, v = self.x[:, :Hq], self.x[:, Hq:Hq + Hkv], self.x[:, Hq + Hkv:]
            q, _ = ttt.qk_norm_rope(q, k, self.pos, freq, rope_scale=rs, V=v, K_cache=Kc,
                                    V_cache=Vc, slots=self.slots)
            return ttt.attention_decode(q, Kc, Vc, table, self.lens, page, with_lse=True)

        def capture(self):
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                self.run(self.Kc, self.Vc)
            torch.cuda.current_stream().wait_stream(s)
            torch.cuda.synchronize()
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.out = self.run(self.Kc, self.Vc)

        def set(self, n):
            self.lens.copy_(_i32(n))
            self.pos.copy_(_i32(n) - 1)
            self.slots.copy_(torch.stack([table[s, (n[s] - 1) // page] * page + (n[s] - 1) % page
                                          for s in range(S)]))
            self.x.copy_(dev(_draw(rng, S, Hq + 2 * Hkv, dh), "bf16"))

    a, b = Step(), Step()
    for s in (a, b):
        s.set([1, 1, 1])
        s.capture()
    for n in ([1, 2, 3], [600, 1, 17], [601, 2, 18], [33, 640, 64]):
        for s in (a, b):
            s.set(n)
        want = [s.run(s.Kc.clone(), s.Vc.clone()) for s in (a, b)]
        torch.cuda.synchronize()
        a.graph.replay()
        b.graph.replay()
        torch.cuda.synchronize()
        for s, w in zip((a, b), want):
            for x, y in zip(s.out, w):
                np.testing.assert_array_equal(host_bits(x), host_bits(y))


def test_a_captured_prompt_replays_with_other_documents():
    """A packed call whose keys are split, in a graph: other inputs and offsets at each replay."""
    import torch
    print("case: captured prompt", flush=True)
    rng = np.random.default_rng(2)
    Nq, Nk, Hq, Hkv, dh = 48, 4000, 4, 1, 128
    assert ttt.lib().ttt_attention_packed_workspace(2, Nq, Nk, Hq, Hkv, dh) > 0
    Q = torch.empty(Nq, Hq, dh, dtype=torch.bfloat16, device="cuda")
    K, V = (torch.empty(Nk, Hkv, dh, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cq, ck = _i32([0, 0, 0]), _i32([0, 0, 0])

    def run():
        return ttt.attention_packed(Q, K, V, cq, ck, with_lse=True)

    def fill(i):
        for t in (Q, K, V):
            t.copy_(dev(_draw(rng, *t.shape), "bf16"))
        cq.copy_(_i32([[0, 20, 48], [0, 48, 48], [0, 1, 40]][i]))
        ck.copy_(_i32([[0, 3000, 4000], [0, 4000, 4000], [0, 64, 2000]][i]))
    fill(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for i in (0, 1, 2, 1, 0):
        fill(i)
        n = 40 if i == 2 else 48
        want = [host_bits(x)[:n] for x in run()]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, want):
            np.testing.assert_array_equal(host_bits(x)[:n], y)


def test_two_streams_and_given_workspaces():
    """The same calls on two streams at once, each with its own workspace, then with one workspace one
    after the other: the same bits. A workspace that is too small or not aligned is refused."""
    import torch
    print("case: streams and workspaces", flush=True)
    rng = np.random.default_rng(3)
    Nq, Nk, Hq, Hkv, dh, page = 32, 6000, 4, 2, 128, 16
    Q, K, V = dev(_draw(rng, Nq, Hq, dh), "bf16"), *(dev(_draw(rng, Nk, Hkv, dh), "bf16") for _ in "kv")
    cq, ck = _i32([0, Nq]), _i32([0, Nk])
    table, lens = _i32(np.arange(Nk // page)[None].repeat(4, 0)), _i32([5990, 17, 4000, 0])
    L = ttt.lib()
    n1 = L.ttt_attention_packed_workspace(1, Nq, Nk, Hq, Hkv, dh)
    n2 = L.ttt_attention_decode_workspace(4, Nk // page, page, Hq, Hkv, dh)
    assert n1 > 0 and n2 > 0

    def packed(**kw):
        return ttt.attention_packed(Q, K, V, cq, ck, with_lse=True, **kw)

    def token(**kw):
        return ttt.attention_decode(Q[:4], K, V, table, lens, page, with_lse=True, **kw)
    want = [host_bits(x) for x in (*packed(), *token())]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [(torch.full((n1,), 255, dtype=torch.uint8, device="cuda"),
           torch.full((n2,), 255, dtype=torch.uint8, device="cuda")) for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s, w in zip(streams, ws):
            with torch.cuda.stream(s):
                got.append((*packed(workspace=w[0]), *token(workspace=w[1])))
    torch.cuda.synchronize()
    one = torch.empty(max(n1, n2), dtype=torch.uint8, device="cuda")
    got.append((*packed(workspace=one), *token(workspace=one)))
    torch.cuda.synchronize()
    for g in got:
        for x, y in zip(g, want):
            np.testing.assert_array_equal(host_bits(x), y)
    for call, n in ((packed, n1), (token, n2)):
        for bad in (one[:n - 1], one[8:n + 4] if n + 4 <= one.numel() else one[8:], one[:0]):
            with pytest.raises(ttt.TTTError):
                call(workspace=bad)


def test_split_rows_of_no_sequence_are_left():
    import torch
    print("case: split keys, rows of no sequence", flush=True)
    rng = np.random.default_rng(7)
    Nq, Nk, Hq, Hkv, dh = 40, 5000, 4, 1, 128
    assert ttt.lib().ttt_attention_packed_workspace(2, Nq, Nk, Hq, Hkv, dh) > 0
    q, k, v = _draw(rng, Nq, Hq, dh), _draw(rng, Nk, Hkv, dh), _draw(rng, Nk, Hkv, dh)
    cq, ck = np.array([3, 20, 33]), np.array([40, 4000, 4990])
    O = torch.full((Nq, Hq, dh), 7.0, dtype=torch.bfloat16, device="cuda")
    L = torch.full((Nq, Hq), 7.0, device="cuda")
    ttt.attention_packed(dev(q, "bf16"), dev(k, "bf16"), dev(v, "bf16"), _i32(cq), _i32(ck), O=O, lse=L)
    torch.cuda.synchronize()
    for x in (O[:3], O[33:], L[:3], L[33:]):
        assert (x == 7).all()
    tokens = list(range(3, 33))
    want = _some_rows(_f(q), _f(k), _f(v), cq, ck, dh ** -0.5, 0, tokens, range(Hq))
    _check(O[3:33], L[3:33], want, _logit_size(_f(q), _f(k), dh ** -0.5)[3:33], dh, "split")


def test_offsets_past_32_bits():
    """A cache of more than 4 GiB: rows at its end are written and read; a packed call whose rows lie
    far apart."""
    import torch
    print("case: large offsets", flush=True)
    rng = np.random.default_rng(4)
    Hq, Hkv, dh, page = 8, 8, 128, 256
    n_pages = (1 << 32) // (page * Hkv * dh * 2) + 9
    Kc = torch.empty(n_pages * page, Hkv, dh, dtype=torch.bfloat16, device="cuda")
    Vc = torch.empty_like(Kc)
    n = 600
    table = _i32([[n_pages - 2, 0, n_pages - 1]])
    tb = [n_pages - 2, 0, n_pages - 1]
    slots = [tb[j // page] * page + j % page for j in range(n)]
    x = _draw(rng, n, Hq + 2 * Hkv, dh)
    X = dev(x, "bf16")
    q, _ = ttt.qk_norm_rope(X[:, :Hq], X[:, Hq:Hq + Hkv], _i32(range(n)),
                            torch.zeros(0, dtype=torch.float64, device="cuda"),
                            V=X[:, Hq + Hkv:], K_cache=Kc, V_cache=Vc, slots=_i32(slots))
    at = torch.tensor(slots, device="cuda")
    np.testing.assert_array_equal(host_bits(Kc[at]), x[:, Hq:Hq + Hkv])  # nothing to norm or rotate
    np.testing.assert_array_equal(host_bits(Vc[at]), x[:, Hq + Hkv:])
    O, L = ttt.attention_decode(q[-1:], Kc, Vc, table, _i32([n]), page, with_lse=True)
    torch.cuda.synchronize()
    qf, kf, vf = _f(x[:, :Hq]), _f(x[:, Hq:Hq + Hkv]), _f(x[:, Hq + Hkv:])
    cu = np.array([0, n])
    want = _some_rows(qf, kf, vf, cu, cu, dh ** -0.5, 0, [n - 1], range(Hq))
    _check(O, L, want, _logit_size(qf[-1:], kf, dh ** -0.5), dh, "token")
    # the cache as a buffer of tokens far apart: every 2^21 + 2^14 elements
    del Kc, Vc
    stride, H, N = (1 << 21) + (1 << 14), 1, 1100
    big = torch.empty(N * stride, dtype=torch.bfloat16, device="cuda").view(N, stride)
    y = _draw(rng, N, 4, dh)
    for i in range(3):  # query (later its result), key, value
        big[:, i * dh:(i + 1) * dh] = dev(y[:, i], "bf16")
    q, k, v = (big[:, i * dh:(i + 1) * dh].view(N, 1, dh) for i in range(3))
    out = big[:, 3 * dh:4 * dh].view(N, 1, dh)
    _, L = ttt.attention_packed(q, k, v, _i32([0, N]), O=out, with_lse=True)
    torch.cuda.synchronize()
    tokens = [0, 1, 500, 1023, 1024, N - 1]
    qf, kf, vf = (_f(y[:, i:i + 1]) for i in range(3))
    want = _some_rows(qf, kf, vf, [0, N], [0, N], dh ** -0.5, 0, tokens, [0])
    _check(out[tokens], L[tokens], want, _logit_size(qf[tokens], kf, dh ** -0.5), dh, "far apart")


def test_two_tokens_of_one_slot_leave_pieces_of_either():
    import torch
    print("case: the same slot twice", flush=True)
    rng = np.random.default_rng(5)
    k, v = _draw(rng, 2, 1, 64), _draw(rng, 2, 1, 64)
    Kc, Vc = (torch.zeros(4, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    K, V = dev(k, "bf16"), dev(v, "bf16")
    ttt.qk_norm_rope(K.clone(), K, _i32([0, 0]), torch.zeros(0, dtype=torch.float64, device="cuda"),
                     V=V, K_cache=Kc, V_cache=Vc, slots=_i32([2, 2]))
    torch.cuda.synchronize()
    for c, x in ((Kc, k), (Vc, v)):
        got = host_bits(c)
        assert ((got[2] == x[0]) | (got[2] == x[1])).all()
        assert (got[[0, 1, 3]] == 0).all()
