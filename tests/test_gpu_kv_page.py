"""GPU tests of the paged Q3 KV cache against the oracle: tables, slots, codes,
norms and window bit-exact, attention within the oracle's derived tolerance."""
import numpy as np
import pytest
import torch

import oracle as O
from dequant_matmul_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hl():
    from dequant_matmul_b200 import hlwq
    return hlwq


@pytest.fixture(scope="module")
def cb8(hl):
    return hl.kv_codebook("cuda")


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _rows(n, H, seed, spikes=True):
    X = synth.activations(n * H, 256, seed=seed).float().reshape(n, H, 256)
    if spikes:
        X[..., :3] *= 30.0   # a few large channels, as keys have
    return X.to(torch.bfloat16)


# ------------------------------------------------------------------ tables
@pytest.mark.parametrize("B,past,new,P,R,pad", [
    (1, 0, 1, 16, 0, 0), (1, 127, 2, 16, 128, 1), (3, 500, 1, 64, 128, 0), (33, 300, 1, 48, 31, 7),
    (5, 700, 900, 16, 1, 3), (1030, 40, 3, 16, 5, 2), (4, 0, 4000, 256, 128, 0)])
def test_block_tables(hl, B, past, new, P, R, pad):
    rng = np.random.default_rng(B + past + new)
    n_past, n_new = rng.integers(0, past + 1, B), rng.integers(0, new + 1, B)
    n_past[0], n_new[0] = past, new
    held = [O.kv_pages(int(p), P, R) for p in n_past]
    need = sum(O.kv_pages(int(p + n), P, R) for p, n in zip(n_past, n_new))
    order = rng.permutation(need + 9)
    width = max(1, max(O.kv_pages(int(p + n), P, R) for p, n in zip(n_past, n_new)))
    table = np.full((B, width), -1)
    at = 0
    for b, k in enumerate(held):
        table[b, :k] = order[at:at + k]
        at += k
    free, T = order[at:], int(n_new.sum()) + pad
    want = O.kv_block_tables(n_past, n_new, free, table, P, R, T)
    t, out, cu = _ints(table), torch.full((1,), -7, dtype=torch.int32, device="cuda"), None
    for _ in range(2):   # a repeated call repeats its result
        cu, slots, left = hl.kv_block_tables(_ints(n_past), _ints(n_new), _ints(free), _ints([len(free)]), t, P, R, T,
                                             n_free_out=out)
        torch.cuda.synchronize()
        assert np.array_equal(t.cpu().numpy(), want[0])
        assert np.array_equal(cu.cpu().numpy(), want[1])
        assert np.array_equal(slots.cpu().numpy(), want[2])
        assert int(left) == want[3]
    assert hl.device_error() == 0


def test_block_tables_without_enough_pages(hl):
    """The pool gives out its last page and then -1; a full table row likewise."""
    hl.device_error()
    past, new, free = [0, 0, 100], [40, 40, 1], [3, 1, 2]
    table = np.full((3, 7), -1)
    table[2, :7] = range(10, 17)
    want = O.kv_block_tables(past, new, free, table, 16, 0, 81)
    t = _ints(table)
    cu, slots, left = hl.kv_block_tables(_ints(past), _ints(new), _ints(free), _ints([3]), t, 16, 0, 81)
    assert hl.device_error() == hl.DEVERR_KV_PAGES
    assert np.array_equal(t.cpu().numpy(), want[0]) and np.array_equal(slots.cpu().numpy(), want[2])
    assert (want[2] == -1).sum() == 40 and int(left) == 0
    t = _ints(table[:, :2])   # rows of two pages: tokens from 32 on have no place
    cu, slots, left = hl.kv_block_tables(_ints(past), _ints(new), _ints(range(20, 40)), _ints([20]), t, 16, 0, 81)
    assert hl.device_error() == hl.DEVERR_KV_PAGES
    want = O.kv_block_tables(past, new, range(20, 40), table[:, :2], 16, 0, 81)
    assert np.array_equal(t.cpu().numpy(), want[0]) and np.array_equal(slots.cpu().numpy(), want[2])
    assert int(left) == 16


def test_block_tables_with_lengths_out_of_range(hl):
    hl.device_error()
    t = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    cu, slots, left = hl.kv_block_tables(_ints([-5, 3]), _ints([2, -1]), _ints([0, 1]), _ints([2]), t, 16, 0, 4)
    assert hl.device_error() == hl.DEVERR_KV_RANGE
    assert cu.tolist() == [0, 2, 2] and slots.tolist() == [16, 17, -1, -1] and int(left) == 1
    # more new tokens than rows
    hl.kv_block_tables(_ints([0, 0]), _ints([3, 3]), _ints([0, 1]), _ints([2]), t, 16, 0, 4)
    assert hl.device_error() == hl.DEVERR_KV_RANGE


# ------------------------------------------------------------------ a batch for append and attention
def _batch(past, new, H, P, R, seed, spikes=True):
    """Host state of a batch with its pages interleaved in a pool."""
    rng = np.random.default_rng(seed)
    B = len(past)
    need = sum(O.kv_pages(p + n, P, R) for p, n in zip(past, new))
    order = rng.permutation(need + 3)
    width = max(1, max(O.kv_pages(p + n, P, R) for p, n in zip(past, new))) + 1
    table, at = np.full((B, width), -1), 0
    for b, p in enumerate(past):
        k = O.kv_pages(p, P, R)
        table[b, :k] = order[at:at + k]
        at += k
    T = sum(new)
    table, cu, slots, _ = O.kv_block_tables(past, new, order[at:], table, P, R, T)
    kv = []
    for which in range(2):
        X = _rows(T, H, seed + 10 + which, spikes and which == 0)
        if T > 2:
            X[1] = 0    # a zero vector
        win = _rows(B * max(R, 1), H, seed + 20 + which).reshape(B, max(R, 1), H, 256).transpose(1, 2)[:, :, :R]
        old = O.kv_quantize(_rows(order.size * P, H, seed + 30 + which, spikes and which == 0).reshape(-1, 256))
        kv.append((X, win.contiguous(), old["packed"].reshape(order.size, P, H, 96).swapaxes(1, 2).copy(),
                   old["norms"].reshape(order.size, P, H).swapaxes(1, 2).copy()))
    return table, cu, slots, kv


def _dev_pages(packed, norms):
    return torch.from_numpy(packed.copy()).cuda(), torch.from_numpy(norms.copy().view(np.uint16)).cuda()


APPENDS = [([0], [1], 1, 16, 0), ([5], [1], 2, 16, 1), ([130, 0, 127, 64], [1, 1, 1, 1], 3, 64, 128),
           ([10, 0, 3], [7, 0, 300], 2, 48, 31), ([200, 1], [65, 128], 4, 16, 64), ([100], [17], 5, 256, 0),
           ([40, 40, 0, 0, 9], [3, 0, 0, 40, 0], 1, 16, 7)]


@pytest.mark.parametrize("past,new,H,P,R", APPENDS)
def test_append(hl, cb8, past, new, H, P, R):
    table, cu, slots, kv = _batch(past, new, H, P, R, seed=sum(past) + R)
    T = sum(new)
    dev, want = [], []
    for X, win, packed, norms in kv:
        want.append(O.kv_paged_append(X, slots, cu, past, packed, norms, win.double().numpy(), R))
        wide = torch.full((T + 2, H * 256 + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:T, :H * 256] = X.reshape(T, -1).cuda()     # rows behind the last request are not read
        dev.append((wide[:, :H * 256].unflatten(1, (H, 256)), win.cuda() if R else None, _dev_pages(packed, norms)))
    (K, kw, kp), (V, vw, vp) = dev
    hl.kv_paged_append(K, V, _ints(list(slots) + [-1, -1], torch.int64), _ints(cu), _ints(past), kp, vp,
                       (kw, vw) if R else None, cb8)
    torch.cuda.synchronize()
    for (_, w, (p, n)), (wp, wn, ww) in zip(dev, want):
        assert np.array_equal(p.cpu().numpy(), wp)
        assert np.array_equal(n.cpu().numpy(), wn.view(np.uint16))
        if R:
            assert np.array_equal(w.double().cpu().numpy(), ww)
    assert hl.device_error() == 0


def test_append_near_the_borders(hl, cb8):
    """Vectors whose rotated values lie on, or a few units of fp32 beside, a
    decision border, and norms next to a binary16 rounding border: the codes and
    norms are still those of the fp64 definition."""
    rng = np.random.default_rng(1)
    n = 4096
    X = np.zeros((n, 256))
    # few distinct integers: rotated values are integers and repeat, norms are roots of integers
    X[:, :] = rng.integers(-2, 3, (n, 256)) * 2.0 ** rng.integers(-60, 60, (n, 1))
    X[: n // 2, 4:] = 0
    X[5] = 0
    X = torch.from_numpy(X).to(torch.bfloat16)
    want = O.kv_quantize(X)
    H, P = 4, 64
    T = n // H
    pages = [(torch.zeros(T // P, H, P, 96, dtype=torch.uint8, device="cuda"),
              torch.zeros(T // P, H, P, dtype=torch.uint16, device="cuda")) for _ in range(2)]
    x = X.reshape(T, H, 256).cuda()
    hl.kv_paged_append(x, x, torch.arange(T, device="cuda"), _ints([0, T]), _ints([0]), *pages, None, cb8)
    torch.cuda.synchronize()
    for p, nr in pages:
        got = p.transpose(1, 2).reshape(n, 96).cpu().numpy()
        bad = O.unpack_codes(got, bits=3) != want["codes"]
        if bad.any():   # two fp64 evaluations may differ only where they cannot tell
            _, mid, _ = O.codebook_fp32(8)
            assert np.all(np.min(np.abs(want["y"][bad][:, None] - mid[None, :]), axis=1) < 1e-12)
        assert np.array_equal(nr.transpose(1, 2).reshape(n).cpu().numpy(), want["norms"].view(np.uint16))


@pytest.mark.parametrize("levels", [[-2.1, -1.2, -0.7, -0.2, 0.3, 0.7, 1.3, 2.2], [-1.0, -0.6, -0.3, -0.1, 0.1, 0.3, 0.6, 1.0],
                                    [-4.5, -2.5, -1.5, -0.5, 0.5, 1.5, 2.5, 4.5]])
def test_append_with_another_codebook(hl, levels):
    """Not symmetric, narrower, with borders beyond 3; and chunks of several requests."""
    H, P, T = 3, 16, 700
    X = _rows(T, H, 31)
    cb = np.array(levels, np.float32)
    x = X.double().reshape(-1, 256).numpy()
    had = np.array([[1.0]])
    while had.shape[0] < 256:
        had = np.block([[had, had], [had, -had]])
    norm = np.sqrt((x * x).sum(-1))
    y = x @ had / np.where(norm > 0, norm, 1.0)[:, None]
    mid = (cb[1:].astype(np.float64) + cb[:-1].astype(np.float64)) / 2
    want = (y[:, :, None] > mid).sum(-1)
    tell = np.min(np.abs(y[:, :, None] - mid), axis=-1) > 1e-12   # two fp64 evaluations agree here
    n = -(-T // P)
    pages = [(torch.zeros(n, H, P, 96, dtype=torch.uint8, device="cuda"),
              torch.zeros(n, H, P, dtype=torch.uint16, device="cuda")) for _ in range(2)]
    hl.kv_paged_append(X.cuda(), X.cuda(), torch.arange(T, device="cuda"), _ints([0, 1, 1, 300, T]), _ints([0, 0, 5, 9]), *pages,
                       None, torch.from_numpy(cb).cuda())
    torch.cuda.synchronize()
    for p, nr in pages:
        got = p.transpose(1, 2).reshape(n * P * H, 96)[:T * H].cpu().numpy()
        assert np.array_equal(O.unpack_codes(got, bits=3)[tell], want[tell])
        assert np.array_equal(nr.transpose(1, 2).reshape(-1)[:T * H].cpu().numpy(), norm.astype(np.float16).view(np.uint16))
    assert hl.device_error() == 0


def test_append_with_slots_out_of_range(hl, cb8):
    """A slot that is not one of the pool is not written, and is reported."""
    hl.device_error()
    pages = [(torch.zeros(2, 1, 16, 96, dtype=torch.uint8, device="cuda"),
              torch.zeros(2, 1, 16, dtype=torch.uint16, device="cuda")) for _ in range(2)]
    x = _rows(3, 1, 5).cuda()
    hl.kv_paged_append(x, x, _ints([3, 32, -1], torch.int64), _ints([0, 3]), _ints([0]), *pages, None, cb8)
    assert hl.device_error() == hl.DEVERR_KV_RANGE
    for p, n in pages:
        assert n.view(torch.int16).reshape(-1).nonzero().tolist() == [[3]]
    # offsets past the rows, and negative lengths
    for cu, past in (([0, 9], [0]), ([2, 1], [0]), ([0, 3], [-1])):
        hl.kv_paged_append(x, x, _ints([4, 5, 6], torch.int64), _ints(cu), _ints(past), *pages, None, cb8)
        assert hl.device_error() & ~hl.DEVERR_KV_RANGE == 0
    for p, n in pages:
        assert n.view(torch.int16).reshape(-1).nonzero().tolist() == [[3]]


# ------------------------------------------------------------------ attention
ATTENTIONS = [
    # past, new, H, G, P, R
    ([0], [1], 1, 1, 16, 0), ([0], [1], 2, 6, 64, 128), ([1], [1], 1, 8, 16, 1), ([15], [1], 1, 4, 16, 0),
    ([16], [1], 1, 4, 16, 0), ([63, 64, 65], [1, 1, 1], 2, 6, 64, 0), ([299], [1], 4, 6, 64, 128),
    ([128], [1], 2, 6, 64, 128), ([1000, 3, 0, 517], [1, 1, 1, 1], 2, 6, 64, 128), ([700, 60], [1, 0], 1, 16, 48, 31),
    ([513], [1], 3, 3, 256, 64), ([400, 33], [1, 1], 1, 64, 16, 7), ([250], [1], 2, 17, 16, 128),
    # a few tokens each
    ([100, 0, 255], [3, 4, 2], 2, 4, 16, 0), ([300, 77], [2, 2], 1, 8, 64, 128), ([90], [5], 1, 3, 16, 3),
    # chunks
    ([0], [40], 2, 6, 16, 0), ([0], [200], 1, 6, 64, 128), ([300], [70], 2, 6, 64, 128),
    ([0, 130, 50], [33, 1, 129], 1, 8, 128, 64), ([37], [257], 1, 1, 16, 31), ([500], [90], 1, 16, 48, 1),
    ([0, 20], [17, 300], 1, 5, 16, 128)]


def _attend(hl, cb8, past, new, H, G, P, R, seed=0, scale=None, behind=2, max_new=None, spikes=True):
    table, cu, slots, kv = _batch(past, new, H, P, R, seed, spikes)
    T = sum(new)
    Q = _rows(T, H * G, seed + 40, spikes=False)
    state = [O.kv_paged_append(X, slots, cu, past, packed, norms, win.double().numpy(), R) for X, win, packed, norms in kv]
    want, tol = O.kv_paged_attention(Q, cu, past, table, *state, R, 0.0625 if scale is None else scale)
    # what attention must not read: pages of no request, places behind the last token, unused ring slots
    used = np.zeros(kv[0][2].shape[0] * P, bool)
    ring = np.zeros((len(past), max(R, 1)), bool)
    for b, (p, n) in enumerate(zip(past, new)):
        i = np.arange(O.kv_encoded(p + n, R))
        used[table[b, i // P] * P + i % P] = True
        if R:
            ring[b, np.arange(O.kv_encoded(p + n, R), p + n) % R] = True
    dev = []
    for packed, norms, win in state:
        norms = np.where(used.reshape(-1, 1, P), norms, np.float16(np.nan))
        packed = np.where(used.reshape(-1, 1, P, 1), packed, np.uint8(255))
        w = torch.from_numpy(win).to(torch.bfloat16).cuda() if R else None
        if R:
            w.transpose(1, 2)[torch.from_numpy(~ring[:, :R]).cuda()] = float("nan")
        dev.append((_dev_pages(packed, norms), w))
    Qd = torch.full((T + behind, H * G, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
    Qd[:T] = Q.cuda()
    out = torch.full_like(Qd, 7.0)
    args = (Qd, _ints(cu), _ints(past), _ints(table), dev[0][0], dev[1][0], (dev[0][1], dev[1][1]) if R else None, cb8,
            max_new or max(new))
    return args, dict(scale=scale, out=out), want, tol


def _check(out, want, tol, T):
    got = out[:T].double().cpu().numpy()
    err = np.linalg.norm(got - want, axis=-1)
    assert np.all(np.isfinite(got))
    assert np.all(err <= tol), (np.max(err / tol), np.unravel_index(np.argmax(err / tol), err.shape))
    assert torch.all(out[T:] == 7.0)   # rows behind the last request stay as they were


@pytest.mark.parametrize("past,new,H,G,P,R", ATTENTIONS)
def test_attention(hl, cb8, past, new, H, G, P, R):
    args, kw, want, tol = _attend(hl, cb8, past, new, H, G, P, R, seed=sum(past) + R + G)
    out = hl.kv_paged_attention(*args, **kw)
    torch.cuda.synchronize()
    _check(out, want, tol, sum(new))
    # the same inputs give the same bits, whatever the workspace held
    ws = torch.full((hl.kv_attention_workspace(args[0], H, len(past), max(new)),), 255, dtype=torch.uint8, device="cuda")
    again = hl.kv_paged_attention(*args, scale=kw["scale"], out=torch.full_like(out, 7.0), workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(out, again)
    assert hl.device_error() == 0


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.25, 1e-6])
def test_attention_scales(hl, cb8, scale):
    """A flat softmax, a sharp one (scores of some tens), a negative scale."""
    for past, new in (([200], [1]), ([150], [40])):
        args, kw, want, tol = _attend(hl, cb8, past, new, 2, 4, 16, 32, seed=9, scale=scale, spikes=False)
        out = hl.kv_paged_attention(*args, **kw)
        torch.cuda.synchronize()
        _check(out, want, tol, sum(new))


def test_attention_bound_on_new_tokens_may_be_loose(hl, cb8):
    for max_new in (3, 8, 100, 1000):
        args, kw, want, tol = _attend(hl, cb8, [60, 5], [1, 3], 1, 6, 16, 16, seed=4, max_new=max_new)
        out = hl.kv_paged_attention(*args, **kw)
        torch.cuda.synchronize()
        _check(out, want, tol, 4)


def test_attention_norms_of_very_different_size(hl, cb8):
    """Value norms from 2^-20 to 2^14: small ones next to large ones neither
    overflow nor vanish; each request has one magnitude in its output."""
    args, kw, _, _ = _attend(hl, cb8, [100, 100, 100], [1, 1, 1], 1, 6, 16, 0, seed=3, spikes=False)
    table = args[3].cpu().numpy()
    for which, norms in ((0, args[4][1]), (1, args[5][1])):
        n = norms.cpu().view(torch.float16).clone()
        for b, e in enumerate((-18, 10, 0)):
            for k in range(7):
                n[int(table[b, k])] *= 2.0 ** e if which else 1.0
        if which:
            n[int(table[2, 0])] *= 2.0 ** -18
            n[int(table[2, 5])] *= 2.0 ** 9
        norms.copy_(n.view(torch.uint16).cuda())
    state = [(p[0].cpu().numpy(), p[1].cpu().numpy().view(np.float16), np.zeros((3, 1, 0, 256))) for p in (args[4], args[5])]
    for p, n, _ in state:   # the unused places: any finite value for the oracle, which does not read them
        n[np.isnan(n)] = 0
    want, tol = O.kv_paged_attention(args[0][:3].cpu(), args[1].tolist(), [100, 100, 100], table, *state, 0, 0.0625)
    out = hl.kv_paged_attention(*args, **kw)
    torch.cuda.synchronize()
    # norms below 2^-14 are subnormal binary16: exact as stored, the oracle reads the same
    _check(out, want, tol, 3)


def test_attention_with_strided_rows(hl, cb8):
    """Q and out inside wider rows (a fused projection's output)."""
    args, kw, want, tol = _attend(hl, cb8, [90, 10], [1, 20], 2, 3, 16, 16, seed=6)
    T, Hq = args[0].shape[:2]
    wide = torch.zeros(T, Hq + 4, 256, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:2 + Hq] = args[0]
    res = torch.full((T, Hq + 1, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    hl.kv_paged_attention(wide[:, 2:2 + Hq], *args[1:], out=res[:, :Hq])
    torch.cuda.synchronize()
    _check(res[:, :Hq], want, tol, 21)
    assert torch.all(res[:, Hq] == 7.0)


def test_attention_leaves_out_pages_that_are_not_there(hl, cb8):
    """Table entries outside the pool are reported and their keys left out."""
    hl.device_error()
    for new in (1, 40):
        args, kw, _, _ = _attend(hl, cb8, [64], [new], 1, 6, 16, 0, seed=8)
        table = args[3].clone()
        table[0, 1], table[0, 3] = -1, args[4][0].shape[0]
        out = hl.kv_paged_attention(*args[:3], table, *args[4:], **kw)
        assert hl.device_error() == hl.DEVERR_KV_RANGE
        # the same as without these pages' keys: the queries see the other ones
        k, v = ((p[0].cpu().numpy(), p[1].cpu().numpy().view(np.float16)) for p in (args[4], args[5]))
        t = args[3].cpu().numpy()[0]
        i = np.array([i for i in range(64 + new) if i // 16 not in (1, 3)])
        K, V = (O.kv_dequantize(p[t[i // 16], 0, i % 16], n[t[i // 16], 0, i % 16]) for p, n in (k, v))
        for j in range(new):
            for g in range(6):
                seen = i <= 64 + j
                s = K[seen] @ args[0][j, g].double().cpu().numpy() / 16
                w = np.exp(s - s.max())
                want = w / w.sum() @ V[seen]
                got = out[j, g].double().cpu().numpy()
                assert np.linalg.norm(got - want) <= 2.0 ** -6 * np.linalg.norm(want) + 2.0 ** -6


def test_attention_rows_whose_every_page_is_gone(hl, cb8):
    """No key left: the row is zero, and nothing is NaN."""
    hl.device_error()
    for new in (1, 30):
        args, kw, _, _ = _attend(hl, cb8, [20], [new], 1, 4, 16, 0, seed=8)
        out = hl.kv_paged_attention(*args[:3], torch.full_like(args[3], -1), *args[4:], **kw)
        assert hl.device_error() == hl.DEVERR_KV_RANGE
        assert torch.all(out[:new] == 0) and torch.all(out[new:] == 7.0)


def test_attention_with_offsets_out_of_range(hl, cb8):
    hl.device_error()
    args, kw, want, tol = _attend(hl, cb8, [20, 30], [1, 1], 1, 4, 16, 0, seed=8)
    T = args[0].shape[0]
    for cu in ([0, 1, T + 1], [0, 5, 2], [-1, 1, 2]):
        hl.kv_paged_attention(args[0], _ints(cu), *args[2:], **kw)
        assert hl.device_error() & ~hl.DEVERR_KV_RANGE == 0
    hl.kv_paged_attention(args[0], args[1], _ints([-1, 30]), *args[3:], **kw)
    assert hl.device_error() == hl.DEVERR_KV_RANGE
    out = hl.kv_paged_attention(*args, **kw)
    torch.cuda.synchronize()
    _check(out, want, tol, 2)


def test_attention_nan_stays_in_its_row(hl, cb8):
    for past, new in (([40], [3]), ([40], [60])):
        args, kw, want, tol = _attend(hl, cb8, past, new, 1, 4, 16, 8, seed=2)
        args[0][1, 2, 7] = float("nan")
        out = hl.kv_paged_attention(*args, **kw)
        torch.cuda.synchronize()
        assert torch.all(torch.isnan(out[1, 2]))
        out[1, 2] = torch.from_numpy(want[1, 2]).to(out.dtype).cuda()
        _check(out, want, tol, new[0])


@pytest.mark.parametrize("new", [3, 40])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_attention_tokens_ahead_have_no_say(hl, cb8, new, value):
    """Norms that are not finite, of tokens that a query does not see."""
    args, kw, want, tol = _attend(hl, cb8, [70], [new], 1, 4, 16, 0, seed=12)
    page, at = int(args[3][0, (70 + new - 1) // 16]), (70 + new - 1) % 16
    for norms in (args[4][1], args[5][1]):
        norms.view(torch.float16)[page, 0, at] = value
    out = hl.kv_paged_attention(*args, **kw)
    torch.cuda.synchronize()
    if value != value:   # the last token itself sees it (an infinite norm may give a score of -inf, which has no weight)
        assert not torch.any(torch.isfinite(out[new - 1]))
    out[new - 1] = torch.from_numpy(want[new - 1]).to(out.dtype).cuda()
    _check(out, want, tol, new)


@pytest.mark.parametrize("new,R", [(3, 16), (2, 1), (40, 8), (60, 64)])
@pytest.mark.parametrize("which,value", [(0, float("nan")), (1, float("nan")), (1, float("inf")), (1, float("-inf"))])
def test_attention_window_tokens_ahead_have_no_say(hl, cb8, new, R, which, value):
    """One value of the last token's key or value that is not finite, in the window."""
    args, kw, want, tol = _attend(hl, cb8, [70], [new], 2, 4, 16, R, seed=21)
    args[6][which][0, 1, (70 + new - 1) % R, 130] = value
    out = hl.kv_paged_attention(*args, **kw)
    torch.cuda.synchronize()
    assert not torch.any(torch.all(torch.isfinite(out[new - 1, 4:]), -1))   # the last token itself, kv head 1
    out[new - 1, 4:] = torch.from_numpy(want[new - 1, 4:]).to(out.dtype).cuda()
    _check(out, want, tol, new)


@pytest.mark.parametrize("past,new,R", [([5000, 40], [1, 1], 128), ([5000], [3], 0), ([3000, 10], [60, 5], 128)])
def test_attention_into_the_queries(hl, cb8, past, new, R):
    args, kw, want, tol = _attend(hl, cb8, past, new, 2, 4, 16, R, seed=22)
    T = sum(new)
    hl.kv_paged_attention(*args, **kw)
    rows = args[0].clone()
    hl.kv_paged_attention(rows, *args[1:], out=rows)
    torch.cuda.synchronize()
    _check(kw["out"], want, tol, T)
    assert torch.equal(rows[:T], kw["out"][:T])
    assert torch.all(torch.isnan(rows[T:]))


@pytest.mark.parametrize("new", [1, 2, 60])
def test_attention_long_items_are_cut_and_joined(hl, cb8, new):
    """One request, one kv head: every CTA gets a part of the same rows."""
    args, kw, want, tol = _attend(hl, cb8, [5000], [new], 1, 8, 64, 100, seed=5)
    out = hl.kv_paged_attention(*args, **kw)
    torch.cuda.synchronize()
    _check(out, want, tol, new)


def test_attention_many_requests(hl, cb8):
    """More requests than CTAs, most of them without tokens."""
    rng = np.random.default_rng(0)
    past, new = [int(x) for x in rng.integers(0, 60, 700)], [0] * 700
    for b in rng.choice(700, 90, replace=False):
        new[b] = 1
    args, kw, want, tol = _attend(hl, cb8, past, new, 1, 2, 16, 8, seed=1)
    out = hl.kv_paged_attention(*args, **kw)
    torch.cuda.synchronize()
    _check(out, want, tol, 90)


def test_attention_wait_runs_out(hl, cb8):
    """The tile kernel whose code copies never come (failure-detection build, waits of
    5 ms): the status says so, the tensor memory is given back, the next call is right."""
    args, kw, want, tol = _attend(hl, cb8, [100, 30], [40, 50], 2, 4, 16, 8, seed=7)
    prod = hl.lib
    hl.lib = hl.load_library(hl.FAULT_LIB_PATH)
    try:
        hl.device_error()
        assert hl.lib.hlwq_fault_inject(1, 5_000_000) == hl.HLWQ_OK
        hl.kv_paged_attention(*args, **kw)
        assert hl.device_error() & hl.DEVERR_TIMEOUT
        assert hl.lib.hlwq_fault_inject(0, 2_000_000_000) == hl.HLWQ_OK
        out = hl.kv_paged_attention(*args, scale=None, out=torch.full_like(kw["out"], 7.0))
        torch.cuda.synchronize()
        assert hl.device_error() == 0
    finally:
        hl.lib.hlwq_fault_inject(0, 2_000_000_000)
        hl.lib = prod
    _check(out, want, tol, 90)


def test_two_streams_at_once(hl, cb8):
    """Two batches on two streams, each with its own workspace."""
    runs = [_attend(hl, cb8, p, n, 2, 6, 64, 128, seed=s) for s, (p, n) in enumerate([([900, 300], [1, 1]), ([200], [150])])]
    side = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        outs = []
        for (args, kw, _, _), st in zip(runs, side):
            with torch.cuda.stream(st):
                outs.append(hl.kv_paged_attention(*args, scale=None, out=torch.full_like(kw["out"], 7.0)))
    torch.cuda.synchronize()
    for out, (args, kw, want, tol) in zip(outs, runs):
        _check(out, want, tol, want.shape[0])


def test_a_step_on_a_given_stream(hl, cb8):
    """stream=...: the step waits for nothing of the current stream, and what it
    allocates itself is not handed to the current stream's work meanwhile."""
    H, G, T = 2, 4, 60
    K, V, Q = _rows(T, H, 1).cuda(), _rows(T, H, 2).cuda(), _rows(T, H * G, 3, False).cuda()
    cache = hl.PagedKVCache(1, H, num_pages=8, max_pages=8, page_size=16, R=16, cb8=cb8)
    n_new, side = _ints([T]), torch.cuda.Stream()
    torch.cuda.synchronize()
    cache.begin(n_new, T, stream=side)
    cache.append(K, V, stream=side)
    out = cache.attention(Q, T, stream=side)
    cache.end(stream=side)
    noise = [torch.full((1 << 18,), 255, dtype=torch.uint8, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    want, tol = _reference(K.cpu(), V.cpu(), Q.cpu(), T, T, 16, G)
    _check(out, want, tol, T)
    assert len(noise) == 64 and cache.n_past.tolist() == [T]


# ------------------------------------------------------------------ together
def _reference(X, Y, Q, N, n, R, G):
    """The last n queries of one request's N tokens, heads [N][H][256]."""
    H = X.shape[1]
    P = 16
    pages = -(-N // P)
    table, cu, slots, _ = O.kv_block_tables([0], [N], list(range(pages)), np.full((1, pages), -1), P, R, N)
    st = [O.kv_paged_append(x, slots, cu, [0], np.zeros((pages, H, P, 96), np.uint8), np.zeros((pages, H, P), np.float16),
                            np.zeros((1, H, R, 256)), R) for x in (X, Y)]
    return O.kv_paged_attention(Q, [0, n], [N - n], table, *st, R, 0.0625)


@pytest.mark.parametrize("R,P", [(16, 16), (0, 48), (128, 64)])
def test_serving_run(hl, cb8, R, P):
    """Requests that arrive, decode, verify drafts, leave and come back in rows
    that had others before, all through the cache's public calls."""
    H, G, B = 2, 3, 3
    cache = hl.PagedKVCache(B, H, num_pages=40, max_pages=24, page_size=P, R=R, cb8=cb8)
    story = [[30, 0, 0], [1, 50, 0], [1, 1, 7], [4, 1, 130], [0, 1, 1], "free 1", [1, 0, 1], [2, 33, 1], [1, 1, 1]]
    seen = [[], [], []]
    for k, new in enumerate(story):
        if isinstance(new, str):
            cache.release(1)
            seen[1] = []
            continue
        T = sum(new)
        K, V, Q = _rows(T + 3, H, 100 * k + 1), _rows(T + 3, H, 100 * k + 2), _rows(T + 3, H * G, 100 * k + 3, False)
        cache.begin(_ints(new), T + 3)
        cache.append(K.cuda(), V.cuda())
        out = cache.attention(Q.cuda(), max(new), out=torch.full((T + 3, H * G, 256), 7.0, dtype=torch.bfloat16, device="cuda"))
        cache.end()
        torch.cuda.synchronize()
        at = 0
        for b, n in enumerate(new):
            seen[b] += [(K[at + j], V[at + j]) for j in range(n)]
            if n:
                X, Y = (torch.stack([s[w] for s in seen[b]]) for w in (0, 1))
                want, tol = _reference(X, Y, Q[at:at + n], len(seen[b]), n, R, G)
                _check(torch.cat([out[at:at + n], out[T:]]), want, tol, n)
            at += n
    held = sum(O.kv_pages(len(s), P, R) for s in seen)
    assert int(cache.n_free) == 40 - held
    rest = cache.free_pages[:40 - held].tolist()
    table = cache.block_table.cpu().numpy()
    mine = [int(table[b, k]) for b in range(B) for k in range(O.kv_pages(len(seen[b]), P, R))]
    assert sorted(rest + mine) == list(range(40))   # no page twice, none lost
    assert hl.device_error() == 0


@pytest.mark.parametrize("T,max_new", [(4, 1), (24, 20)])
def test_step_in_a_graph(hl, cb8, T, max_new):
    """One captured step, replayed with other lengths and inputs on another
    stream, does what the eager calls do."""
    H, G, B, R, P = 2, 6, 4, 8, 16

    def cache():
        return hl.PagedKVCache(B, H, num_pages=60, max_pages=20, page_size=P, R=R, cb8=cb8)

    K, V, Q = (torch.zeros(T, n, 256, dtype=torch.bfloat16, device="cuda") for n in (H, H, H * G))
    n_new, out = _ints([0] * B), torch.zeros(T, H * G, 256, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(T, dtype=torch.int64, device="cuda")
    a, b = cache(), cache()
    ws = torch.empty(max(16, hl.kv_attention_workspace(Q, H, B, max_new)), dtype=torch.uint8, device="cuda")

    def step(c, out):
        c.begin(n_new, T, slot_map=slots)
        c.append(K, V)
        c.attention(Q, max_new, out=out, workspace=ws)
        c.end()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(a, out)    # nothing yet: all lengths are 0
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step(a, out)
    torch.cuda.current_stream().wait_stream(side)
    step(b, out)
    rng = np.random.default_rng(T)
    for k in range(6):
        new = rng.integers(0, max_new + 1, B)
        new[3] = 0 if k == 2 else new[3]
        while new.sum() > T:
            new[int(np.argmax(new))] //= 2
        n_new.copy_(_ints(new))
        for x, h, s in ((K, H, 1), (V, H, 2), (Q, H * G, 3)):
            x.copy_(_rows(T, h, 50 * k + s).cuda())
        want = torch.full_like(out, 3.0)
        out.fill_(3.0)
        g.replay()
        step(b, want)
        torch.cuda.synchronize()
        assert torch.equal(out, want), k
        for x, y in ((a.n_past, b.n_past), (a.n_free, b.n_free), (a.block_table, b.block_table),
                     (a.k_pages[0], b.k_pages[0]), (a.v_pages[1], b.v_pages[1]), (a.window[0], b.window[0])):
            assert torch.equal(x, y), k
    assert hl.device_error() == 0


def test_long_cache_offsets(hl, cb8):
    """Page offsets past 2^31 bytes: a pool of 2.6 GB whose last pages are used."""
    H, P, G = 4, 4096, 6
    n = 2 ** 31 // (H * P * 96) + 300
    packed, norms = torch.zeros(n, H, P, 96, dtype=torch.uint8, device="cuda"), torch.zeros(n, H, P, dtype=torch.uint16, device="cuda")
    T = 40
    K, V = _rows(T, H, 1), _rows(T, H, 2)
    Q = _rows(T, H * G, 3, False)
    table = _ints([[n - 1]])
    slots = _ints([(n - 1) * P + i for i in range(T)], torch.int64)
    pages = (packed, norms)
    vpages = (packed.clone(), norms.clone())
    hl.kv_paged_append(K.cuda(), V.cuda(), slots, _ints([0, T]), _ints([0]), pages, vpages, None, cb8)
    want, tol = _reference(K, V, Q, T, T, 0, G)
    out = hl.kv_paged_attention(Q.cuda(), _ints([0, T]), _ints([0]), table, pages, vpages, None, cb8, T)
    one = hl.kv_paged_attention(Q[-1:].cuda(), _ints([0, 1]), _ints([T - 1]), table, pages, vpages, None, cb8, 1)
    torch.cuda.synchronize()
    _check(out, want, tol, T)
    _check(one, want[-1:], tol[-1:], 1)


# ------------------------------------------------------------------ values of very different size in one row
def _attend_on(hl, cb8, X, Y, Q, n, R, G, P=16):
    """Call, reference and tolerance of the last n queries Q over one request's keys X
    and values Y [N][H][256], all from the oracle's state."""
    N, H, _ = X.shape
    pages = -(-N // P)
    table, cu, slots, _ = O.kv_block_tables([0], [N], list(range(pages)), np.full((1, pages), -1), P, R, N)
    st = [O.kv_paged_append(x, slots, cu, [0], np.zeros((pages, H, P, 96), np.uint8), np.zeros((pages, H, P), np.float16),
                            np.zeros((1, H, R, 256)), R) for x in (X, Y)]
    want, tol = O.kv_paged_attention(Q, [0, n], [N - n], table, *st, R, 0.0625)
    dev = [(_dev_pages(p, nr), torch.from_numpy(w).to(torch.bfloat16).cuda() if R else None) for p, nr, w in st]
    out = torch.full(Q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    args = (Q.cuda(), _ints([0, n]), _ints([N - n]), _ints(table), dev[0][0], dev[1][0],
            (dev[0][1], dev[1][1]) if R else None, cb8, n)
    return args, dict(out=out), want, tol


def _small_values(N, n, Hq, seed):
    """Keys, values of norm 2^-12 and queries near a common direction, which is returned."""
    base = _rows(1, 1, seed, False)[0, 0]
    Q = (base + 0.2 * _rows(n, Hq, seed + 1, False).float()).to(torch.bfloat16)
    return _rows(N, 1, seed + 2, False), (_rows(N, 1, seed + 3, False).float() * 2.0 ** -16).to(torch.bfloat16), Q, base.float()


ROWS = [(1, 6), (3, 4), (20, 6), (40, 4)]   # few rows per kv head, and tiles of 128


@pytest.mark.parametrize("new,G", ROWS)
def test_attention_large_value_without_weight(hl, cb8, new, G):
    """A value of norm 60000 whose key is far from every query (weight e^-48), among
    values of norm 2^-12: these are the row's terms and keep their accuracy."""
    N = 150 + new
    for heavy in (3, 40, 149):
        X, Y, Q, base = _small_values(N, new, G, 50)
        X[heavy, 0] = (-3 * base).to(torch.bfloat16)
        Y[heavy, 0] = 3750.0 * torch.sign(Y[heavy, 0].float()).to(torch.bfloat16)
        args, kw, want, tol = _attend_on(hl, cb8, X, Y, Q, new, 0, G)
        out = hl.kv_paged_attention(*args, **kw)
        torch.cuda.synchronize()
        assert np.all(np.linalg.norm(want, axis=-1) < 2.0 ** -12)
        _check(out, want, tol, new)


@pytest.mark.parametrize("new,G", [c for c in ROWS if c[0] > 1])
@pytest.mark.parametrize("value", [60000.0, float("inf")])
def test_attention_large_value_ahead(hl, cb8, new, G, value):
    """The last token's value is large or infinite: rows that do not see it keep the
    accuracy that their own values of norm 2^-12 have."""
    N = 60 + new
    X, Y, Q, _ = _small_values(N, new, G, 60)
    args, kw, want, tol = _attend_on(hl, cb8, X, Y, Q, new, 0, G)
    args[5][1].view(torch.float16)[int(args[3][0, (N - 1) // 16]), 0, (N - 1) % 16] = value
    out = hl.kv_paged_attention(*args, **kw)
    torch.cuda.synchronize()
    _check(out[:new - 1], want[:new - 1], tol[:new - 1], new - 1)


@pytest.mark.parametrize("new,G", ROWS)
def test_attention_value_norms_that_grow(hl, cb8, new, G):
    """The largest term comes late, by its score, by its norm, or by both: what came
    before is rescaled, and zero norms and the smallest ones do not disturb it."""
    N = 300 + new
    for grow_key, grow_value in ((0.0, 2.0), (3.0, 0.0), (3.0, -2.0), (-1.0, 2.0)):
        X, Y, Q, base = _small_values(N, new, G, 70)
        Y = Y.float() * 2.0 ** 6
        at = torch.arange(N)[:, None, None] / N
        X = (X.float() + grow_key * at * base).to(torch.bfloat16)
        Y = (Y * torch.exp2(6 * grow_value * at)).to(torch.bfloat16)
        Y[7], Y[8] = 0, 2.0 ** -28   # a zero vector, a norm of 2^-24
        args, kw, want, tol = _attend_on(hl, cb8, X, Y, Q, new, 0, G)
        out = hl.kv_paged_attention(*args, **kw)
        torch.cuda.synchronize()
        _check(out, want, tol, new)


# ------------------------------------------------------------------ operands of fewer bits
def _centroid_spread(c):
    """How far binary16 roundings of a times the levels c can agree with one common
    factor: the best of 256 factors a between two powers of two."""
    a = (1.0 + np.arange(256) / 256)[:, None] * np.asarray(c, np.float64)
    r = a.astype(np.float16).astype(np.float64) / np.asarray(c, np.float64)
    return np.min((r.max(1) - r.min(1)) / (r.max(1) + r.min(1)))


@pytest.mark.parametrize("unit", [1.0, 2.0 ** -30, 2.0 ** 40])
@pytest.mark.parametrize("new,G", ROWS)
def test_attention_sharp_scores_of_exact_queries(hl, cb8, new, G, unit):
    """Two keys with scores near 200 through different centroids, the others near
    -200.  The queries have one rotated coordinate and are exact in any binary type, so
    scores differ only by the centroids' roundings; a codebook of another unit changes
    nothing (the norms take it back) as long as its levels are finite.

    Bound: half a bf16 step of the output, 2^-8 |o|; the scores' errors e_j move o by
    at most sum_j p_j |e_j| |v_j - o|, |e_j| <= (d + 2^-20) |s_j| with d the centroids'
    half spread; a term of the sum has p n rounded (2^-11) and its centroids (d)."""
    c = cb8.double().cpu().numpy()
    d = _centroid_spread(c)
    assert d < 0.15 * 2.0 ** -12
    rng = np.random.default_rng(new)
    N, P, coord = 50 + new, 16, 77
    i = np.arange(N)
    codes = rng.integers(0, 8, (2, N, 256))
    codes[0, :, coord] = rng.integers(0, 4, N)
    pair = [3, 45]
    codes[0, pair, coord] = [5, 7]
    s = np.full(N, 200.0)
    s[pair] += [0.2, -0.3]
    norms = np.stack([(s * 16 / (4 * np.abs(c[codes[0, :, coord]]))), np.full(N, 20.0)]).astype(np.float16)
    s = 4 * norms[0].astype(np.float64) * c[codes[0, :, coord]] / 16          # the query is 4 (H256)_coord
    w = np.exp(s - s.max())
    w /= w.sum()
    had = np.array([[1.0]])
    while had.shape[0] < 256:
        had = np.block([[had, had], [had, -had]])
    V = c[codes[1]] @ had * norms[1].astype(np.float64)[:, None] / 256
    want = w @ V
    size = np.linalg.norm(V, axis=1)
    tol = 2.0 ** -8 * np.linalg.norm(want) + (w * ((d + 2.0 ** -20) * np.abs(s) * np.linalg.norm(V - want, axis=1)
                                                   + (2.0 ** -11 + d) * size)).sum()
    pages = -(-N // P)
    dev = []
    for which in range(2):
        packed, nr = np.zeros((pages, 1, P, 96), np.uint8), np.zeros((pages, 1, P), np.float16)
        packed[i // P, 0, i % P] = O.pack_codes(codes[which], bits=3)
        nr[i // P, 0, i % P] = norms[which]
        dev.append(_dev_pages(packed, nr))
    Q = torch.from_numpy(np.broadcast_to(4 * had[coord], (new, G, 256)).copy()).to(torch.bfloat16)
    out = hl.kv_paged_attention((Q.double() / unit).to(torch.bfloat16).cuda(), _ints([0, new]), _ints([N - new]),
                                _ints(np.arange(pages)[None]), *dev, None, (cb8.double() * unit).float(), new)
    torch.cuda.synchronize()
    err = np.linalg.norm(out.double().cpu().numpy() / unit - want, axis=-1)
    assert np.all(err <= tol), (err.max() / tol)


@pytest.mark.parametrize("e", [-110, -70, 50, 70, 100, 122])
@pytest.mark.parametrize("new,G", ROWS)
def test_attention_query_magnitudes(hl, cb8, new, G, e):
    """Queries 2^e times as large under a scale 2^-e times as large give the same scores:
    powers of two, so the same tolerance holds."""
    X, Y, Q = _rows(90, 1, 80, False), _rows(90, 1, 81, False), _rows(new, G, 82, False)
    for R in (0, 30):
        args, kw, want, tol = _attend_on(hl, cb8, X, Y, Q, new, R, G)
        out = hl.kv_paged_attention((Q.double() * 2.0 ** e).to(torch.bfloat16).cuda(), *args[1:], scale=2.0 ** (-4 - e), **kw)
        torch.cuda.synchronize()
        _check(out, want, tol, new)


@pytest.mark.parametrize("R,P", [(0, 16), (3, 64), (128, 4096)])
def test_block_tables_with_lengths_whose_sum_is_near_2_32(hl, R, P):
    """Such a request is reported and gets no page; the others' pages are what they are without it."""
    hl.device_error()
    top = 2 ** 31 - 1
    past, new, width = [5, top, 40], [2 * P, top, R + 3 * P], 6
    table = np.full((3, width), -1)
    table[1] = range(20, 26)
    for b in (0, 2):
        k = O.kv_pages(past[b], P, R)
        table[b, :k] = range(30 + b * 6, 30 + b * 6 + k)
    free, T = list(range(12)), 2 * P + 3
    want = O.kv_block_tables(past, [new[0], 0, new[2]], free, table, P, R, T)
    t = _ints(table)
    cu, slots, left = hl.kv_block_tables(_ints(past), _ints(new), _ints(free), _ints([12]), t, P, R, T)
    torch.cuda.synchronize()
    assert hl.device_error() & hl.DEVERR_KV_RANGE
    assert np.array_equal(t.cpu().numpy(), want[0]) and int(left) == want[3]
    assert np.array_equal(slots[:2 * P].cpu().numpy(), want[2][:2 * P])
    # just below the limit: nothing to report about the length itself
    hl.kv_block_tables(_ints([top - 3]), _ints([3]), _ints(free), _ints([12]), torch.full((1, width), -1, dtype=torch.int32, device="cuda"),
                       P, R, 3)
    assert hl.device_error() == hl.DEVERR_KV_PAGES


def test_release_on_the_stream_of_the_steps(hl, cb8):
    """Steps and a release between them on a side stream that is far behind the host, without
    a synchronisation of the device: no page is lost or given out twice."""
    H, P, B = 1, 16, 3
    cache = hl.PagedKVCache(B, H, num_pages=12, max_pages=12, page_size=P, R=0, cb8=cb8)
    x = _rows(120, H, 9).cuda()
    news = [_ints(v) for v in ([70, 40, 0], [0, 1, 60])]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    for k, n_new in enumerate(news):
        T = int(sum(([70, 40, 0], [0, 1, 60])[k]))
        cache.begin(n_new, T, stream=side)
        cache.append(x[:T], x[:T], stream=side)
        cache.end(stream=side)
        if k == 0:
            cache.release(0, stream=side)
    side.synchronize()
    assert cache.n_past.tolist() == [0, 41, 60] and int(cache.n_free) == 12 - 3 - 4
    held = [p for row in cache.block_table.tolist() for p in row if p >= 0]
    assert sorted(held + cache.free_pages[:5].tolist()) == list(range(12))
    assert hl.device_error() == 0


@pytest.mark.parametrize("R", [0, 8])
def test_the_step_ends_with_the_lengths_it_began_with(hl, cb8, R):
    """n_new lowered after the append (as if drafts were rejected) does not make appended tokens
    older ones, and a negative length counts as 0 to the end."""
    hl.device_error()
    H, G, N = 1, 4, 26
    X, Y, Q = _rows(N, H, 1), _rows(N, H, 2), _rows(N, G, 3, False)
    cache = hl.PagedKVCache(2, H, num_pages=8, max_pages=8, page_size=16, R=R, cb8=cb8)
    for lo, n in ((0, 20), (20, 5), (25, 1)):
        n_new = _ints([n, -3])
        cache.begin(n_new, n)
        cache.append(X[lo:lo + n].cuda(), Y[lo:lo + n].cuda())
        out = torch.full((n, G, 256), 7.0, dtype=torch.bfloat16, device="cuda")
        cache.attention(Q[lo:lo + n].cuda(), n, out=out)
        n_new[0] = 2
        cache.end()
        assert cache.n_past.tolist() == [lo + n, 0]
        assert hl.device_error() == hl.DEVERR_KV_RANGE   # the negative length
        want, tol = _reference(X[:lo + n], Y[:lo + n], Q[lo:lo + n], lo + n, n, R, G)
        _check(out, want, tol, n)
    assert int(cache.n_free) == 8 - O.kv_pages(N, 16, R)


@pytest.mark.parametrize("max_new,new,G", [(2, 3, 2), (1, 2, 8), (7, 8, 2), (100, 120, 1), (100, 101, 6), (20, 300, 6)])
def test_attention_more_tokens_than_max_new(hl, cb8, max_new, new, G):
    """Reported whether or not the rows still fit the last row tile; the other request's
    rows are right, and so are the rows that were written."""
    hl.device_error()
    args, kw, want, tol = _attend(hl, cb8, [30, 50], [1, new], 1, G, 16, 8, seed=13, max_new=max_new)
    out = hl.kv_paged_attention(*args, **kw)
    assert hl.device_error() == hl.DEVERR_KV_RANGE
    written = 1 + max_new
    err = np.linalg.norm(out[:written].double().cpu().numpy() - want[:written], axis=-1)
    assert np.all(err <= tol[:written])
    hl.kv_paged_attention(*args[:-1], new, **kw)
    assert hl.device_error() == 0


# Offsets that are not those of requests in [0, T), and negative lengths (T = 3 rows).
BAD_STEPS = [([0, 4], [0]), ([0, 9], [0]), ([2, 1], [0]), ([2, 0], [0]), ([-1, 2], [0]), ([0, 3], [-1]), ([0, 0], [-5]),
             ([0, 2, 1], [0, 0]), ([0, 3, 2], [0, 0]), ([0, 1, 3], [0, -2]), ([0, 0, 3], [-1, 0])]


@pytest.mark.parametrize("cu,past", BAD_STEPS)
def test_append_reports_rows_out_of_range(hl, cb8, cu, past):
    """Always, whether or not the request has a token; places of no slot stay as they are."""
    hl.device_error()
    pages = [(torch.zeros(2, 1, 16, 96, dtype=torch.uint8, device="cuda"),
              torch.zeros(2, 1, 16, dtype=torch.uint16, device="cuda")) for _ in range(2)]
    x = _rows(3, 1, 5).cuda()
    hl.kv_paged_append(x, x, _ints([4, 5, 6], torch.int64), _ints(cu), _ints(past), *pages, None, cb8)
    assert hl.device_error() == hl.DEVERR_KV_RANGE
    for p, n in pages:
        assert set(n.view(torch.int16).reshape(-1).nonzero().flatten().tolist()) <= {4, 5, 6}
    hl.kv_paged_append(x, x, _ints([4, 5, 6], torch.int64), _ints([0, 3]), _ints([0]), *pages, None, cb8)
    assert hl.device_error() == 0


@pytest.mark.parametrize("cu,past", BAD_STEPS)
@pytest.mark.parametrize("max_new", [1, 40])
def test_attention_reports_rows_out_of_range(hl, cb8, cu, past, max_new):
    hl.device_error()
    T, G = 3, 4
    args, kw, want, tol = _attend(hl, cb8, [20, 30], [2, 1], 1, G, 16, 0, seed=8, behind=0)
    if len(past) == 1:
        args = (args[0], args[1], args[2], args[3][:1], *args[4:])
    hl.kv_paged_attention(args[0], _ints(cu), _ints(past), *args[3:-1], max(3, max_new), **kw)
    assert hl.device_error() == hl.DEVERR_KV_RANGE


def test_attention_of_parts_of_a_step(hl, cb8):
    """The decoding requests of a step and the one with a chunk in calls of their own, each
    with the kernel for its lengths: together what one call gives."""
    past, new = [100, 0, 37, 60, 300], [1, 1, 1, 50, 1]
    args, kw, want, tol = _attend(hl, cb8, past, new, 2, 4, 16, 32, seed=17)
    out = kw["out"]
    Q, cu, n_past, table, kp, vp, (kw_, vw), cb, _ = args
    for b0, b1, max_new in ((0, 3, 1), (3, 4, 50), (4, 5, 1)):
        hl.kv_paged_attention(Q, cu[b0:b1 + 1], n_past[b0:b1], table[b0:b1], kp, vp, (kw_[b0:b1], vw[b0:b1]), cb, max_new, out=out)
    torch.cuda.synchronize()
    _check(out, want, tol, sum(new))
    assert hl.device_error() == 0


@pytest.mark.parametrize("e", [-90, 60, 110, 121])
@pytest.mark.parametrize("new,G", ROWS)
def test_attention_window_key_magnitudes(hl, cb8, new, G, e):
    """Exact keys 2^e times as large under a scale 2^-e times as large (all tokens in the window)."""
    N, R = 60 + new, 128
    X, Y, Q = _rows(N, 1, 83, False), _rows(N, 1, 84, False), _rows(new, G, 85, False)
    args, kw, want, tol = _attend_on(hl, cb8, X, Y, Q, new, R, G)
    window = ((args[6][0].double() * 2.0 ** e).to(torch.bfloat16), args[6][1])
    out = hl.kv_paged_attention(*args[:6], window, *args[7:], scale=2.0 ** (-4 - e), **kw)
    torch.cuda.synchronize()
    _check(out, want, tol, new)


@pytest.mark.parametrize("e", [-100, 60, 110, 122])
@pytest.mark.parametrize("flat", [False, True])
@pytest.mark.parametrize("new,G", ROWS)
def test_attention_window_value_magnitudes(hl, cb8, new, G, flat, e):
    """Exact values 2^e times as large give outputs 2^e times as large; with flat weights
    and one sign their plain sum would overflow."""
    N, R = 90 + new, 160
    X, Y, Q = _rows(N, 1, 86, False), _rows(N, 1, 87, False), _rows(new, G, 88, False)
    if flat:
        Y, Q = Y.abs(), (Q.double() * 2.0 ** -20).to(torch.bfloat16)
    args, kw, want, tol = _attend_on(hl, cb8, X, Y, Q, new, R, G)
    window = (args[6][0], (args[6][1].double() * 2.0 ** e).to(torch.bfloat16))
    out = hl.kv_paged_attention(*args[:6], window, *args[7:], **kw)
    torch.cuda.synchronize()
    _check(out.double() * 2.0 ** -e, want, tol, new)


def test_attention_of_few_tokens_under_the_largest_max_new(hl, cb8):
    """B times max_new's row tiles just below its limit of 2^31: two requests of thousands have
    tokens, and the bound costs nothing that grows with it."""
    B, T, G, R, P = 8191, 262176 * 2, 64, 4, 16
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("Q of 17 GB")
    X, Y, q = _rows(50, 1, 90, False), _rows(50, 1, 91, False), _rows(3, G, 92, False)
    args, kw, want, tol = _attend_on(hl, cb8, X, Y, q, 3, R, G)
    past, new = torch.zeros(B, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    past[[40, 8190]], new[[40, 8190]] = 47, 3
    cu = torch.cat([torch.zeros(1, dtype=torch.int32), new.cumsum(0).int()])
    table = torch.full((B, args[3].shape[1]), -1, dtype=torch.int32, device="cuda")
    table[[40, 8190]] = args[3]
    window = []
    for w in args[6]:
        window.append(torch.zeros(B, 1, R, 256, dtype=torch.bfloat16, device="cuda"))
        window[-1][[40, 8190]] = w
    Q = torch.empty(T, G, 256, dtype=torch.bfloat16, device="cuda")
    Q[:6] = torch.cat([q, q]).cuda()
    Q[6] = 7.0
    call = (Q, cu.cuda(), past.cuda(), table, *args[4:6], tuple(window), cb8, T)
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    ends[0].record()
    hl.kv_paged_attention(*call, out=Q)
    ends[1].record()
    torch.cuda.synchronize()
    assert hl.device_error() == 0
    _check(Q[:7].cpu(), np.concatenate([want, want]), np.concatenate([tol, tol]), 6)
    assert ends[0].elapsed_time(ends[1]) < 100


@pytest.mark.parametrize("e", [16, 24, 30, 100])
@pytest.mark.parametrize("R", [0, 60, 400])
@pytest.mark.parametrize("new,G", ROWS)
def test_attention_scores_of_any_size(hl, cb8, new, G, R, e):
    """One key's score is far above the others' (all of them below 0 or not), at sizes of
    2^18 to 2^106, where neighbouring fp32 numbers are up to 2^82 apart: its value is the
    output, with the tolerance of a single term."""
    N = 160 + new
    for hot in (3, N - new - 1):
        for sign in (1, -1):
            X, Y, Q, base = _small_values(N, new, G, 95)
            if sign < 0:
                X = ((0.1 * X.float() - base) * (1 + torch.arange(N)[:, None, None] / N)).to(torch.bfloat16)
            X[hot, 0] = ((3 if sign > 0 else -0.25) * base).to(torch.bfloat16)
            Y[80, 0] = 3750.0 * torch.sign(Y[80, 0].float()).to(torch.bfloat16)
            args, kw, want, tol = _attend_on(hl, cb8, X, Y, (Q.double() * 2.0 ** e).to(torch.bfloat16), new, R, G)
            assert np.ptp(want.reshape(-1, 256), axis=0).max() == 0 and tol.max() < 0.02 * np.linalg.norm(want[0, 0])
            out = hl.kv_paged_attention(*args, **kw)
            torch.cuda.synchronize()
            _check(out, want, tol, new)


@pytest.mark.parametrize("e", [16, 24, 60])
@pytest.mark.parametrize("R", [0, 400])
@pytest.mark.parametrize("new,G", ROWS)
def test_attention_equal_keys_at_scores_of_any_size(hl, cb8, new, G, R, e):
    """Two keys that are the same and far above the others have half the weight each,
    whichever tiles and parts they are in: equal scores are rounded alike."""
    N = 200 + new
    for pair in ((3, 5), (3, 70), (20, N - new - 1)):
        X, Y, Q, base = _small_values(N, new, G, 99)
        X[list(pair), 0] = (3 * base).to(torch.bfloat16)
        args, kw, want, _ = _attend_on(hl, cb8, X, Y, (Q.double() * 2.0 ** e).to(torch.bfloat16), new, R, G)
        # half a bf16 step of the output; p n rounded (2^-11) and centroids (2^-13) of two terms
        # no larger than twice the output's norm together
        tol = (2.0 ** -8 + 2 * (2.0 ** -11 + 2.0 ** -13)) * np.linalg.norm(want, axis=-1)
        sizes = [np.linalg.norm(Y[i, 0].double().numpy()) for i in pair]
        assert sum(sizes) / 2 < 2 * np.linalg.norm(want[0, 0])
        out = hl.kv_paged_attention(*args, **kw)
        torch.cuda.synchronize()
        _check(out, want, tol, new)


@pytest.mark.parametrize("e", [118, 122, 124])
@pytest.mark.parametrize("new,G", ROWS)
def test_attention_largest_queries_with_a_window(hl, cb8, new, G, e):
    """Queries near the top of bf16's range whose scores fp32 holds: the key with the
    largest score wins, and no row comes out NaN."""
    N, R = 60 + new, 128
    X, Y, Q, base = _small_values(N, new, G, 97)
    X[5, 0] = 3 * base
    X = (X.float() * 2.0 ** -6).to(torch.bfloat16)
    args, kw, want, tol = _attend_on(hl, cb8, X, Y, (Q.double() * 2.0 ** e).to(torch.bfloat16), new, R, G)
    assert np.ptp(want.reshape(-1, 256), axis=0).max() == 0 and tol.max() < 0.02 * np.linalg.norm(want[0, 0])
    out = hl.kv_paged_attention(*args, **kw)
    torch.cuda.synchronize()
    _check(out, want, tol, new)
