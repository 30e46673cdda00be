"""Pins of the paged KV-cache oracle (CPU), and the refusals of the paged calls
(host checks: nothing is launched)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle as O
from dequant_matmul_b200 import synth


def _pages(pool, H, P):
    return np.zeros((pool, H, P, 96), np.uint8), np.zeros((pool, H, P), np.float16)


def test_block_tables_by_hand():
    # P = 4, R = 2: request 0 goes from 5 to 9 tokens (3 -> 7 encoded, pages 1 -> 2), request 1 from 0 to 3
    # (0 -> 1 encoded, pages 0 -> 1), request 2 stays
    table = np.full((3, 3), -1)
    table[0, 0], table[2, 0] = 7, 8
    t, cu, slots, left = O.kv_block_tables([5, 0, 6], [4, 3, 0], [1, 2, 3, 4], table, 4, 2, 9)
    assert t.tolist() == [[7, 4, -1], [3, -1, -1], [8, -1, -1]]
    assert cu.tolist() == [0, 4, 7, 7]
    # tokens 3..6 of request 0 leave; of request 1 token 0 leaves when token 2 enters
    assert slots.tolist() == [31, 16, 17, 18, -1, -1, 12, -1, -1]
    assert left == 2


@pytest.mark.parametrize("R", [0, 1, 5, 128])
def test_paged_state_equals_the_one_head_cache(R):
    """Any batching of appends leaves each head in the state that quantizing all
    but the last R tokens and keeping those gives."""
    P, H, chunks = 16, 2, [3, 1, 40, 1, 7]
    N = sum(chunks)
    X = synth.activations(N * H, 256, seed=R + 1).reshape(N, H, 256)
    x = X.double().numpy()
    packed, norms = _pages(8, H, P)
    win = np.zeros((1, H, R, 256))
    table, free, n = np.full((1, 8), -1), [5, 2, 7, 0, 1], 0
    for c in chunks:
        table, cu, slots, left = O.kv_block_tables([n], [c], free, table, P, R, c)
        free = free[:left]
        packed, norms, win = O.kv_paged_append(X[n:n + c], slots, cu, [n], packed, norms, win, R)
        n += c
    e = max(0, N - R)
    for h in range(H):
        q = O.kv_quantize(x[:e, h]) if e else None
        for i in range(e):
            assert np.array_equal(packed[table[0, i // P], h, i % P], q["packed"][i])
            assert norms[table[0, i // P], h, i % P] == q["norms"][i]
        for i in range(e, N):
            assert np.array_equal(win[0, h, i % R], x[i, h])


def test_attention_agrees_with_scores_and_a_plain_softmax():
    P, H, G, R, N, n = 16, 2, 3, 6, 40, 4
    X, Y = (synth.activations(N * H, 256, seed=s).reshape(N, H, 256) for s in (1, 2))
    Q = synth.activations(n * H * G, 256, seed=3).reshape(n, H * G, 256)
    table, cu, slots, _ = O.kv_block_tables([0], [N], list(range(4)), np.full((1, 4), -1), P, R, N)
    k, v = (O.kv_paged_append(x, slots, cu, [0], *_pages(4, H, P), np.zeros((1, H, R, 256)), R) for x in (X, Y))
    out, tol = O.kv_paged_attention(Q, [0, n], [N - n], table, k, v, R, 0.0625)
    e = N - R
    for h in range(H):
        kq, vq = O.kv_quantize(X[:e, h]), O.kv_quantize(Y[:e, h])
        S = O.kv_scores_window(Q[:, h * G:(h + 1) * G].reshape(-1, 256), kq["packed"], kq["norms"],
                               X[e:, h].double().numpy()).reshape(n, G, N) * 0.0625
        V = np.concatenate([O.kv_dequantize(vq["packed"], vq["norms"]), Y[e:, h].double().numpy()])
        for j in range(n):
            w = torch.softmax(torch.from_numpy(S[j, :, :N - n + j + 1]), -1).numpy()
            assert np.allclose(out[j, h * G:(h + 1) * G], w @ V[:N - n + j + 1], rtol=1e-12, atol=1e-12)
    assert np.all(tol > 0) and np.all(tol < 0.1 * np.linalg.norm(out, axis=-1))


def test_planted_mistakes_fail_the_tolerance():
    """What a wrong kernel would give is outside the tolerance: a key too many,
    a window slot off by one, values un-normalised by 1 percent, a scale."""
    P, H, R, N = 16, 1, 8, 60
    X, Y = (synth.activations(N, 256, seed=s).reshape(N, H, 256) for s in (4, 5))
    Q = synth.activations(3, 256, seed=6).reshape(3, 1, 256)
    table, cu, slots, _ = O.kv_block_tables([0], [N], list(range(4)), np.full((1, 4), -1), P, R, N)
    k, v = (O.kv_paged_append(x, slots, cu, [0], *_pages(4, H, P), np.zeros((1, H, R, 256)), R) for x in (X, Y))
    out, tol = O.kv_paged_attention(Q, [0, 3], [N - 3], table, k, v, R, 0.0625)

    def off(got):
        return np.all(np.linalg.norm(got - out, axis=-1)[:2] > tol[:2])

    assert off(O.kv_paged_attention(Q, [0, 3], [N - 2], table, k, v, R, 0.0625)[0])
    assert off(O.kv_paged_attention(Q, [0, 3], [N - 3], table, k, (v[0], v[1], np.roll(v[2], 1, 2)), R, 0.0625)[0])
    assert off(O.kv_paged_attention(Q, [0, 3], [N - 3], table, k, v, R, 0.07)[0])
    assert off(1.02 * out)


# ------------------------------------------------------------------ refusals
@pytest.fixture(scope="module")
def hl():
    from dequant_matmul_b200 import build
    build.build()
    from dequant_matmul_b200 import hlwq
    return hlwq


P16 = ctypes.c_void_p(4096)   # fake, aligned, never dereferenced
P8 = ctypes.c_void_p(4104)
ODD = ctypes.c_void_p(4097)


def _refused(fn, good, cases):
    for i, (changes, want) in enumerate(cases):
        args = dict(good)
        assert all(k in args for k in changes)
        args.update(changes)
        assert fn(*args.values()) == want, (i, changes)


def test_block_tables_refusals(hl):
    good = dict(n_past=P16, n_new=P16, B=4, R=128, P=64, free=P16, cap=100, n_free=P16, n_free_out=P8, table=P16,
                max_pages=8, cu=P16, slots=P16, T=4, stream=None)
    EI, EU, EA = hl.HLWQ_EINVAL, hl.HLWQ_EUNSUPPORTED, hl.HLWQ_EALIGN
    _refused(hl.lib.hlwq_kv_block_tables, good, [
        (dict(n_past=None), EI), (dict(n_new=None), EI), (dict(free=None), EI), (dict(n_free=None), EI),
        (dict(n_free_out=None), EI), (dict(table=None), EI), (dict(cu=None), EI), (dict(slots=None), EI),
        (dict(n_free_out=P16), EI),                      # the same word as n_free
        (dict(B=0), EI), (dict(T=0), EI), (dict(T=(1 << 30) + 1), EI), (dict(R=-1), EI), (dict(R=(1 << 20) + 1), EI),
        (dict(cap=0), EI), (dict(max_pages=0), EI), (dict(P=0), EI), (dict(P=-16), EI),
        (dict(P=8), EU), (dict(P=24), EU), (dict(P=8192), EU), (dict(B=8193), EU),
        (dict(slots=ctypes.c_void_p(4100)), EA), (dict(n_past=ODD), EA), (dict(table=ctypes.c_void_p(4098)), EA)])


def test_append_refusals(hl):
    good = dict(K=P16, ldk=1024, V=P16, ldv=1024, T=4, H=4, slots=P16, cu=P16, n_past=P16, B=4, cb=P16, kp=P16, kn=P16,
                vp=P16, vn=P16, num_pages=10, P=64, kw=P16, vw=P16, R=128, stream=None)
    EI, EU, EA = hl.HLWQ_EINVAL, hl.HLWQ_EUNSUPPORTED, hl.HLWQ_EALIGN
    _refused(hl.lib.hlwq_kv_paged_append, good, [
        ({k: None}, EI) for k in ("K", "V", "slots", "cu", "n_past", "cb", "kp", "kn", "vp", "vn", "kw", "vw")])
    _refused(hl.lib.hlwq_kv_paged_append, good, [
        (dict(ldk=1016), EI), (dict(ldv=0), EI), (dict(H=0), EI), (dict(num_pages=0), EI), (dict(T=-1), EI),
        (dict(P=40), EU), (dict(H=1025, ldk=1 << 20, ldv=1 << 20), EU), (dict(B=9000), EU),
        (dict(ldk=1028), EA), (dict(K=P8), EA), (dict(kp=P8), EA), (dict(vn=P8), EA), (dict(kw=P8), EA),
        (dict(slots=ctypes.c_void_p(4100)), EA)])


def test_attention_refusals(hl):
    need = hl.workspace_bytes(hl.HLWQ_OP_KV_ATTENTION, 4, 1, 4, 24, 4)
    good = dict(Q=P16, ldq=6144, T=4, Hq=24, H=4, scale=0.0625, cu=P16, n_past=P16, B=4, max_new=1, table=P16,
                max_pages=8, cb=P16, kp=P16, kn=P16, vp=P16, vn=P16, num_pages=10, P=64, kw=P16, vw=P16, R=128, out=P16,
                ldo=6144, ws=P16, ws_bytes=need, stream=None)
    EI, EU, EA, EW = hl.HLWQ_EINVAL, hl.HLWQ_EUNSUPPORTED, hl.HLWQ_EALIGN, hl.HLWQ_EWORKSPACE
    _refused(hl.lib.hlwq_kv_paged_attention, good, [
        ({k: None}, EI) for k in ("Q", "cu", "n_past", "table", "cb", "kp", "kn", "vp", "vn", "kw", "vw", "out")])
    _refused(hl.lib.hlwq_kv_paged_attention, good, [
        (dict(Hq=23), EI), (dict(H=0), EI), (dict(ldq=6136), EI), (dict(ldo=6136), EI), (dict(max_new=0), EI),
        (dict(max_pages=0), EI), (dict(scale=float("nan")), EI), (dict(scale=float("inf")), EI),
        (dict(Hq=65, H=1, ldq=16640, ldo=16640), EU), (dict(P=17), EU),
        (dict(Q=P8), EA), (dict(out=P8), EA), (dict(ldq=6148), EA), (dict(vw=P8), EA), (dict(table=ODD), EA)])
    if need:
        _refused(hl.lib.hlwq_kv_paged_attention, good, [
            (dict(ws=None), EW), (dict(ws_bytes=need - 1), EW), (dict(ws=P8), EA)])


def test_binding_refuses_before_it_calls(hl):
    """Types and shapes are the binding's to check; CPU tensors are refused."""
    x = torch.zeros(4, 2, 256, dtype=torch.bfloat16)
    i = torch.zeros(5, dtype=torch.int32)
    with pytest.raises(hl.HLWQError, match="CUDA"):
        hl.kv_block_tables(i, i, i, i[:1], i.reshape(5, 1), 64, 128, T=4)
    with pytest.raises(hl.HLWQError, match="CUDA"):
        hl.kv_paged_append(x, x, i.long(), i, i[:4], None, None, None, None)
    with pytest.raises(hl.HLWQError, match="CUDA"):
        hl.kv_paged_attention(x, i, i[:4], None, None, None, None, None, 1)


def test_release_gives_back_the_pages_that_there_are(hl):
    """Row 0 has 5 pages' tokens, but the pool ran out behind the third page."""
    cache = hl.PagedKVCache(2, 1, 8, 6, page_size=16, R=4, device="cpu", cb8=torch.zeros(8))
    cache.block_table[0, :5] = torch.tensor([7, 2, 6, -1, -1], dtype=torch.int32)
    cache.block_table[1, :1] = 5
    cache.n_past[:] = torch.tensor([4 + 70, 4 + 3], dtype=torch.int32)
    cache.n_free[0] = 4                                      # pages 0, 1, 3, 4
    cache.free_pages[:4] = torch.tensor([0, 1, 3, 4], dtype=torch.int32)
    cache.release(0)
    assert int(cache.n_free) == 7 and cache.free_pages[:7].tolist() == [0, 1, 3, 4, 7, 2, 6]
    assert cache.block_table[0].tolist() == [-1] * 6 and cache.n_past.tolist() == [0, 7]
    cache.release(0)                                         # an empty row
    cache.release(1)
    assert int(cache.n_free) == 8 and sorted(cache.free_pages.tolist()) == list(range(8))


def test_attention_refuses_too_many_row_tiles(hl):
    """B times the row tiles of max_new tokens has to stay below 2^31, whatever the lengths are."""
    T, G, B = 1 << 24, 64, 8192
    ws = hl.workspace_bytes(hl.HLWQ_OP_KV_ATTENTION, T, T, B, G, 1)
    args = dict(Q=P16, ldq=G * 256, T=T, Hq=G, H=1, scale=0.0625, cu=P16, n_past=P16, B=B, max_new=T, table=P16, max_pages=8,
                cb=P16, kp=P16, kn=P16, vp=P16, vn=P16, num_pages=10, P=64, kw=P16, vw=P16, R=128, out=P16, ldo=G * 256,
                ws=P16, ws_bytes=ws, stream=None)
    assert B * (T * G // 128) >= 2 ** 31
    assert hl.lib.hlwq_kv_paged_attention(*args.values()) == hl.HLWQ_EUNSUPPORTED
