"""ttt_qk_norm_rope, ttt_attention_packed and ttt_attention_decode refuse bad arguments on the host,
before anything is enqueued (no GPU: every call below fails validation), and report their
workspaces."""
import pytest

import chunked_weight_sequence_amd as ttt

OK, E_NULL, E_SHAPE, E_DTYPE, E_ALIGN, E_WS, E_UNSUP, E_LAUNCH, E_ALIAS = range(9)
A = 0x7F0000000000          # fake, 16-byte aligned device addresses (never dereferenced)
MB = 1 << 20
F32, BF16 = 0, 1


def rope(**kw):
    a = dict(Q=A, qs=None, K=A + 64 * MB, ks=None, V=A + 96 * MB, vs=None, dt=BF16, qw=A + 128 * MB,
             kw=A + 129 * MB, eps=1e-6, pos=A + 130 * MB, inv=A + 131 * MB, rot=128, layout=0,
             rs=1.0, Qo=A + 192 * MB, qos=None, Ko=A + 256 * MB, kos=None, Kc=A + 320 * MB,
             Vc=A + 384 * MB, slots=A + 448 * MB, n_slots=2048, N=1000, Hq=32, Hkv=8, dh=128)
    a.update(kw)
    wq, wk = a["Hq"] * a["dh"], a["Hkv"] * a["dh"]
    for k, w in (("qs", wq), ("ks", wk), ("vs", wk), ("qos", wq), ("kos", wk)):
        a[k] = w if a[k] is None else a[k]
    return ttt.lib().ttt_qk_norm_rope(
        a["Q"], a["qs"], a["K"], a["ks"], a["V"], a["vs"], a["dt"], a["qw"], a["kw"], a["eps"],
        a["pos"], a["inv"], a["rot"], a["layout"], a["rs"], a["Qo"], a["qos"], a["Ko"], a["kos"],
        a["Kc"], a["Vc"], a["slots"], a["n_slots"], a["N"], a["Hq"], a["Hkv"], a["dh"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), E_DTYPE), (dict(Q=None), E_NULL), (dict(K=None), E_NULL), (dict(pos=None), E_NULL),
    (dict(Qo=None), E_NULL), (dict(inv=None), E_NULL), (dict(V=None), E_NULL),
    (dict(Kc=None), E_NULL), (dict(Vc=None), E_NULL),
    (dict(slots=None), E_NULL),                                 # a cache without slots
    (dict(slots=None, V=None, Kc=None, Vc=None, Ko=None), E_NULL),  # nowhere to put the keys
    (dict(N=0), E_SHAPE), (dict(N=(1 << 26) + 1), E_SHAPE), (dict(Hq=0), E_SHAPE),
    (dict(Hkv=0), E_SHAPE), (dict(dh=72, rot=64), E_SHAPE), (dict(dh=272), E_SHAPE),
    (dict(dh=0, rot=0), E_SHAPE), (dict(rot=8), E_SHAPE), (dict(rot=144), E_SHAPE),
    (dict(rot=-16), E_SHAPE), (dict(layout=2), E_SHAPE), (dict(eps=-1.0), E_SHAPE),
    (dict(eps=float("nan")), E_SHAPE), (dict(rs=float("inf")), E_SHAPE),
    (dict(Hq=8192, Hkv=8), E_SHAPE), (dict(n_slots=0), E_SHAPE), (dict(n_slots=1 << 31), E_SHAPE),
    (dict(qs=32 * 128 - 8), E_SHAPE), (dict(ks=8 * 128 + 4), E_SHAPE), (dict(vs=0), E_SHAPE),
    (dict(kos=-1024), E_SHAPE), (dict(qos=1 << 32), E_SHAPE),
    (dict(Q=A + 8), E_ALIGN), (dict(pos=A + 130 * MB + 4), E_ALIGN),
    (dict(Kc=A + 320 * MB + 2), E_ALIGN), (dict(qw=A + 128 * MB + 4), E_ALIGN),
    (dict(Qo=A, qos=32 * 128 + 8), E_ALIAS),                    # in place with another stride
    (dict(Qo=A + 256), E_ALIAS), (dict(Ko=A), E_ALIAS), (dict(Qo=A + 64 * MB), E_ALIAS),
    (dict(Ko=A + 192 * MB), E_ALIAS), (dict(Kc=A + 384 * MB + 16), E_ALIAS),
    (dict(Kc=A + 96 * MB), E_ALIAS), (dict(slots=A + 320 * MB), E_ALIAS),
    # slices of one buffer that do overlap: K's columns begin inside Q's
    (dict(Q=A, qs=48 * 128, K=A + 31 * 256, ks=48 * 128, Qo=A, qos=48 * 128), E_ALIAS),
    # a row that wraps into the next token's columns
    (dict(Q=A, qs=48 * 128, K=A + 32 * 256, ks=48 * 128, Ko=A + 41 * 256, kos=48 * 128), E_ALIAS),
])
def test_norm_rope_rejects_bad_arguments(kw, code):
    assert rope(**kw) == code


def packed(**kw):
    a = dict(Q=A, qs=None, K=A + 64 * MB, ks=None, V=A + 96 * MB, vs=None, dt=BF16, O=A + 128 * MB,
             os=None, lse=A + 192 * MB, cq=A + 200 * MB, ck=A + 201 * MB, n=4, Nq=1000, Nk=2000,
             Hq=32, Hkv=8, dh=128, scale=0.1, window=0, ws=A + 512 * MB, wsb=1 << 40)
    a.update(kw)
    wq, wk = a["Hq"] * a["dh"], a["Hkv"] * a["dh"]
    for k, w in (("qs", wq), ("ks", wk), ("vs", wk), ("os", wq)):
        a[k] = w if a[k] is None else a[k]
    return ttt.lib().ttt_attention_packed(
        a["Q"], a["qs"], a["K"], a["ks"], a["V"], a["vs"], a["dt"], a["O"], a["os"], a["lse"],
        a["cq"], a["ck"], a["n"], a["Nq"], a["Nk"], a["Hq"], a["Hkv"], a["dh"], a["scale"],
        a["window"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=7), E_DTYPE), (dict(dt=F32), E_UNSUP), (dict(dh=96), E_UNSUP), (dict(dh=256), E_UNSUP),
    (dict(Q=None), E_NULL), (dict(K=None), E_NULL), (dict(V=None), E_NULL), (dict(O=None), E_NULL),
    (dict(cq=None), E_NULL), (dict(ck=None), E_NULL),
    (dict(n=0), E_SHAPE), (dict(n=(1 << 20) + 1), E_SHAPE), (dict(Nq=0), E_SHAPE),
    (dict(Nk=0), E_SHAPE), (dict(Nk=(1 << 26) + 1), E_SHAPE), (dict(Hq=12), E_SHAPE),
    (dict(Hkv=0), E_SHAPE), (dict(Nq=1 << 26, Hq=32), E_SHAPE), (dict(scale=0.0), E_SHAPE),
    (dict(scale=-0.1), E_SHAPE), (dict(scale=float("nan")), E_SHAPE),
    (dict(scale=float("inf")), E_SHAPE), (dict(window=-1), E_SHAPE),
    (dict(window=(1 << 30) + 1), E_SHAPE), (dict(qs=32 * 128 - 8), E_SHAPE),
    (dict(ks=8 * 128 + 4), E_SHAPE), (dict(vs=(1 << 23) + 8), E_SHAPE), (dict(os=0), E_SHAPE),
    (dict(Q=A + 8), E_ALIGN), (dict(cq=A + 200 * MB + 4), E_ALIGN), (dict(ws=A + 8), E_ALIGN),
    (dict(lse=A + 192 * MB + 4), E_ALIGN),
    (dict(O=A), E_ALIAS), (dict(O=A + 64 * MB), E_ALIAS), (dict(lse=A + 128 * MB), E_ALIAS),
    (dict(lse=A + 96 * MB), E_ALIAS), (dict(O=A + 200 * MB - 4096), E_ALIAS),
])
def test_packed_rejects_bad_arguments(kw, code):
    assert packed(**kw) == code


def decode(**kw):
    a = dict(Q=A, qs=None, Kc=A + 64 * MB, Vc=A + 128 * MB, dt=BF16, O=A + 192 * MB, os=None,
             lse=A + 200 * MB, table=A + 208 * MB, mp=64, page=64, np=256, lens=A + 216 * MB, n=8,
             Hq=32, Hkv=8, dh=128, scale=0.1, window=0, ws=A + 512 * MB, wsb=1 << 40)
    a.update(kw)
    for k in ("qs", "os"):
        a[k] = a["Hq"] * a["dh"] if a[k] is None else a[k]
    return ttt.lib().ttt_attention_decode(
        a["Q"], a["qs"], a["Kc"], a["Vc"], a["dt"], a["O"], a["os"], a["lse"], a["table"], a["mp"],
        a["page"], a["np"], a["lens"], a["n"], a["Hq"], a["Hkv"], a["dh"], a["scale"], a["window"],
        a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=7), E_DTYPE), (dict(dt=F32), E_UNSUP), (dict(dh=80), E_UNSUP), (dict(page=8), E_UNSUP),
    (dict(page=48), E_UNSUP), (dict(page=1 << 17), E_UNSUP),
    (dict(Q=None), E_NULL), (dict(Kc=None), E_NULL), (dict(Vc=None), E_NULL), (dict(O=None), E_NULL),
    (dict(table=None), E_NULL), (dict(lens=None), E_NULL),
    (dict(n=0), E_SHAPE), (dict(mp=0), E_SHAPE), (dict(np=0), E_SHAPE), (dict(page=0), E_SHAPE),
    (dict(page=-16), E_SHAPE), (dict(mp=1 << 25), E_SHAPE), (dict(np=1 << 30, page=128), E_SHAPE),
    (dict(Hq=30), E_SHAPE), (dict(n=1 << 20, Hq=128), E_SHAPE), (dict(scale=0.0), E_SHAPE),
    (dict(window=-5), E_SHAPE), (dict(qs=8), E_SHAPE), (dict(os=32 * 128 + 4), E_SHAPE),
    (dict(Kc=A + 64 * MB + 8), E_ALIGN), (dict(table=A + 208 * MB + 4), E_ALIGN),
    (dict(ws=None), E_WS), (dict(wsb=100), E_WS),
    (dict(O=A), E_ALIAS), (dict(O=A + 128 * MB), E_ALIAS), (dict(lse=A + 208 * MB), E_ALIAS),
    (dict(ws=A + 64 * MB), E_ALIAS), (dict(ws=A + 192 * MB), E_ALIAS),
])
def test_decode_rejects_bad_arguments(kw, code):
    assert decode(**kw) == code


def test_launches_past_32_bits_of_threads_are_refused():
    """Empty sequences and one-head tokens reach them long before the tensors do."""
    assert rope(N=(1 << 25) + 1, Hq=1, Hkv=1, dh=16, rot=0) == E_SHAPE
    assert packed(n=1 << 20, Nq=1, Nk=1, Hq=16, Hkv=16) == E_SHAPE
    assert packed(n=1 << 17, Nq=1, Nk=1, Hq=128, Hkv=128, dh=64) == E_SHAPE
    assert packed(n=1, Nq=(1 << 26) - 4, Nk=1, Hq=32) == E_SHAPE   # the tokens alone would pass
    assert decode(n=1 << 20, Hq=16, Hkv=16) == E_SHAPE
    assert decode(n=1 << 18, Hq=64, Hkv=64, dh=64) == E_SHAPE


def test_workspace_queries():
    lib = ttt.lib()
    one = lib.ttt_attention_decode_workspace(1, 64, 64, 32, 8, 128)
    assert one > 0 and one % (32 * 130 * 4) == 0               # fp32 partial results, some pieces
    assert lib.ttt_attention_decode_workspace(4096, 64, 64, 32, 8, 128) == 0
    assert lib.ttt_attention_decode_workspace(1, 64, 48, 32, 8, 128) == 0    # refused
    assert lib.ttt_attention_decode_workspace(1, 64, 64, 30, 8, 128) == 0
    assert lib.ttt_attention_packed_workspace(0, 16, 16, 8, 8, 64) == 0
    assert lib.ttt_attention_packed_workspace(1, 16, 16, 8, 8, 96) == 0
    # a full prompt fills the chip with row tiles: nothing to join
    assert lib.ttt_attention_packed_workspace(1, 32768, 32768, 32, 8, 128) == 0


def test_binding_refuses_cpu_tensors_and_unknown_names():
    import torch
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        ttt.attention_packed(q, q, q, cu)
    with pytest.raises(ValueError):
        ttt.qk_norm_rope(q, q, cu, torch.zeros(8, dtype=torch.float64))
    with pytest.raises(ValueError):
        ttt.attention_decode(q, q, q, cu[None], cu, 16)
    with pytest.raises(ValueError):
        ttt.rope_frequencies(64, scaling="other")
    for bad in (0, 1, -64, 258, (1 << 40) + 64):
        with pytest.raises(ValueError):
            ttt.rope_frequencies(bad, device="cpu")
    with pytest.raises(ttt.TTTError):
        ttt.rope_frequencies(7, device="cpu")          # odd
    with pytest.raises(TypeError):
        ttt.rope_frequencies(64.0, device="cpu")
    with pytest.raises(ValueError):
        ttt.rope_frequencies(64, scaling="yarn", factor=4.0, original_length=(1 << 32) + 4096,
                             device="cpu")
