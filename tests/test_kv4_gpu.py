"""The 4-bit cache on a GPU against its fp64 oracle: the number format bit for bit, attention within derived bounds.

Bounds of the decode step (out in fp32; u = 2^-24):
* A score is a sum of products of fp16 numbers that are exact, accumulated in fp32 over 128 terms in 8 matrix
  instructions and 8 fused steps, times constants.  With A = scale * sum_d |q_d| (s n_d + |z|) every partial sum is at
  most A, each instruction adds up 16 terms with at most 2^-22 of A lost (alignment, truncation and the carry of the
  running sum), so a score is within 2^-18 A; the cap's tanh adds 2^-22 cap, the bias one rounding of its size.
* p = exp(t - lse): a relative error of 2 * (score bound) + 2^-18 for exp2, the sums and the division.
* p s is rounded to fp16 once: 2^-11 relative (half a step of fp16), so out is within 2^-11 sum p s n plus the error of
  p times sum p (s n + |z|), plus fp32 accumulation.
"""
import numpy as np
import pytest
import torch

from _harness import Guards
from oracle import h2o, kv4

import attention_guided_kv_gb300 as K

pytestmark = pytest.mark.gpu
D = 128


class Cache:
    """A 4-bit cache in permuted pages, its rows random codes and scales, with a host copy by logical row."""

    def __init__(self, rng, B, Hkv, Hq, page, cap, spare=3):
        self.B, self.Hkv, self.Hq, self.page, self.cap = B, Hkv, Hq, page, cap
        self.pages = (cap + page - 1) // page
        n = B * self.pages + spare
        self.table_np = rng.permutation(n)[:B * self.pages].astype(np.int32).reshape(B, self.pages)
        self.g = Guards()
        self.codes = [self.g.like(torch.from_numpy(rng.integers(0, 256, (n, Hkv, page, 64), dtype=np.uint8)).cuda())
                      for _ in range(2)]
        self.scales = []
        for _ in range(2):
            s = np.abs(rng.standard_normal((n, Hkv, page, 4, 1))) * 0.3
            z = rng.standard_normal((n, Hkv, page, 4, 1)) * 0.5 - 2.2
            self.scales.append(self.g.like(torch.from_numpy(np.concatenate([s, z], -1)).bfloat16().cuda()))
        self.table = self.g.like(torch.from_numpy(self.table_np).cuda())
        self.kv = K.paged_kv4(self.codes[0], self.codes[1], self.scales[0], self.scales[1], Hq)

    def rows(self, b, h, n, side):
        """codes [n, 128], s and z [n, 4] fp64 of the first n slots, as they are now."""
        t = torch.from_numpy(self.table_np[b, :(n + self.page - 1) // self.page].astype(np.int64)).cuda()
        c = self.codes[side][t, h].reshape(-1, 64)[:n].cpu().numpy()
        s = self.scales[side][t, h].reshape(-1, 4, 2)[:n].double().cpu().numpy()
        return kv4.unpack(c), s[..., 0], s[..., 1]


def bf(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float64)).bfloat16()


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


# ----------------------------------------------------------------------------------------------------------------------
# append, read
# ----------------------------------------------------------------------------------------------------------------------
def _inputs(rng, kind, rows):
    x = rng.standard_normal((rows, D))
    if kind == "grid":                      # few distinct values: ties at every other border
        x = rng.integers(-8, 9, (rows, D)) * 0.25
    elif kind == "wide":                    # magnitudes over 70 binades: differences round in fp32
        x = x * 2.0 ** rng.integers(-40, 30, (rows, D))
    elif kind == "corners":
        x = x * 0
        x[0, :] = -3.25                     # constant
        x[1 % rows, ::3] = -0.0
        x[2 % rows, 5] = 2.0 ** 126         # the largest the format holds
        x[3 % rows, 5] = -2.0 ** 126
        x[3 % rows, 6] = 2.0 ** 126
        x[4 % rows, 40] = 2.0 ** 127        # past it: NaN, in its group only
        x[5 % rows, 70] = np.nan
        x[6 % rows, 100] = np.inf
        x[7 % rows, 3] = 2.0 ** -98         # scale below 2^-100
        x[8 % rows, 3] = 2.0 ** -95
        x[9 % rows] = rng.standard_normal(D) * 2.0 ** -126
        x[10 % rows, :32] = 1.0             # range / 15 on a border of bf16
        x[10 % rows, 0] = 1.0 + 15 * 2.0 ** -7 * (1 + 2.0 ** -8)
    return bf(x)


@pytest.mark.parametrize("kind", ["normal", "grid", "wide", "corners"])
@pytest.mark.parametrize("page,Hkv,start,new", [(16, 2, [0, 15, 7], [1, 33, 0]), (64, 3, [60, 0], [0, 71]),
                                                (256, 1, [255], [2]), (32, 5, [5, 31, 32, 0], [1, 1, 1, 1])])
def test_append_is_the_format(kind, page, Hkv, start, new):
    rng = np.random.default_rng(7)
    B, total = len(new), sum(new)
    c = Cache(rng, B, Hkv, Hkv, page, max(a + b for a, b in zip(start, new)) + 1)
    before = [t.clone() for t in c.codes + c.scales]
    pad = 3                                   # packed rows behind the last sequence
    k, v = _inputs(rng, kind, (total + pad) * Hkv), _inputs(rng, kind, (total + pad) * Hkv)
    seq, off = c.g.like(ints(start)), ints(np.concatenate([[0], np.cumsum(new)]))
    cap = c.cap
    pos, nxt = c.g.new((B, Hkv, cap), torch.int32, -9), c.g.like(ints([100 * (b + 1) for b in range(B)]))
    cum = c.g.new((B, Hkv, cap), torch.float32, 5.0)
    ws = K.workspace(K.kvsel_kv4_append_workspace(c.kv, B))
    kd, vd = k.view(-1, Hkv, D).cuda(), v.view(-1, Hkv, D).cuda()
    K.kvsel_kv4_append(c.kv, c.table, seq, off, kd, vd, ws, pos_map=pos, next_pos=nxt, h2o_cum=cum)
    assert K.read_status(ws) == 0
    assert seq.tolist() == [a + b for a, b in zip(start, new)]
    assert nxt.tolist() == [100 * (b + 1) + new[b] for b in range(B)]
    back = [c.g.new((total + pad, Hkv, D), torch.bfloat16, 9.0) for _ in range(2)]
    K.kvsel_kv4_read(c.kv, c.table, seq, off, back[0], back[1], ws, start=ints(start))
    assert K.read_status(ws) == 0
    touched = [torch.zeros_like(t, dtype=torch.bool) for t in before]
    for side, x in ((0, k), (1, v)):
        want = kv4.quantise_rows(x.double().numpy())
        at = 0
        for b in range(B):
            for i in range(new[b]):
                slot = start[b] + i
                p = int(c.table_np[b, slot // page])
                for h in range(Hkv):
                    r = at * Hkv + h
                    codes = kv4.unpack(c.codes[side][p, h, slot % page].cpu().numpy())
                    sz = c.scales[side][p, h, slot % page].double().cpu().numpy()
                    assert np.array_equal(codes, want[0][r]), (kind, b, i, h)
                    assert np.array_equal(sz[:, 0], want[1][r], equal_nan=True)
                    assert np.array_equal(sz[:, 1], want[2][r], equal_nan=True)
                    value = kv4.values(want[0][r], want[1][r], want[2][r])
                    # fp64 to fp32 to bf16: s n + z has one fp32 rounding in the kernel as well
                    got = back[side][at, h].double().cpu().numpy()
                    ref = torch.from_numpy(value).float().bfloat16().double().numpy()
                    assert np.array_equal(got, ref, equal_nan=True)
                    touched[side][p, h, slot % page] = True
                    touched[2 + side][p, h, slot % page] = True
                    if side == 0:
                        assert int(pos[b, h, slot]) == 100 * (b + 1) + i and float(cum[b, h, slot]) == 0.0
                at += 1
    for now, old, t in zip(c.codes + c.scales, before, touched):   # nothing else was written
        assert torch.equal(torch.where(t, 0, now), torch.where(t, 0, old))
    assert bool((back[0][total:] == 9.0).all()) and bool((back[1][total:] == 9.0).all())
    assert int((pos == -9).sum()) == B * Hkv * cap - total * Hkv and int((cum == 5.0).sum()) == B * Hkv * cap - total * Hkv
    c.g.check()


def test_append_many_ctas_and_again_on_the_same_workspace():
    """More rows than the grid takes at once, and a second call on the counters the first left."""
    rng = np.random.default_rng(8)
    Hkv, page, n = 8, 64, 5001
    c = Cache(rng, 2, Hkv, Hkv, page, 2 * n)
    x = bf(rng.standard_normal((2 * n, Hkv, D))).cuda()
    seq, off = ints([0, 3]), ints([0, n - 1, 2 * n - 4])
    ws = K.workspace(K.kvsel_kv4_append_workspace(c.kv, 2))
    K.kvsel_kv4_append(c.kv, c.table, seq, off, x, x, ws)
    K.kvsel_kv4_append(c.kv, c.table, seq, ints([0, 2, 2]), x, x, ws)
    assert K.read_status(ws) == 0 and seq.tolist() == [n + 1, n]
    out = [torch.zeros(n + 1, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    K.kvsel_kv4_read(c.kv, c.table, seq, ints([0, n + 1, n + 1]), out[0], out[1], ws)
    assert K.read_status(ws) == 0
    assert torch.equal(out[0], out[1]) and torch.equal(out[0][n - 1:], out[0][:2])
    g = x[:n - 1].float().unflatten(-1, (4, 32))
    step = (g.amax(-1) - g.amin(-1)) / 15
    # half a step of the scale, the scale's rounding at the top code and the output's rounding
    err = (out[0][:n - 1].float().unflatten(-1, (4, 32)) - g).abs()
    assert bool((err <= step[..., None] * (0.5 + 15 * 2.0 ** -9) + g.abs().amax(-1, keepdim=True) * 2.0 ** -8).all())
    c.g.check()


def test_append_and_read_report_what_does_not_fit():
    rng = np.random.default_rng(9)
    c = Cache(rng, 3, 2, 2, 16, 40)
    ws = K.workspace(512)
    x = bf(rng.standard_normal((9, 2, D))).cuda()
    before = [t.clone() for t in c.codes + c.scales]
    full = c.pages * 16

    def unchanged(b):
        t = torch.from_numpy(c.table_np[b].astype(np.int64)).cuda()
        return all(torch.equal(now[t], old[t]) for now, old in zip(c.codes + c.scales, before))

    seq = ints([5, full - 2, 7])                       # sequence 1 has room for two, gets three
    K.kvsel_kv4_append(c.kv, c.table, seq, ints([0, 3, 6, 9]), x, x, ws)
    assert K.read_status(ws) == K.KVSEL_ERR_BAD_INDEX
    assert seq.tolist() == [8, full - 2, 10] and unchanged(1) and not unchanged(0) and not unchanged(2)
    for off in ([0, 5, 3, 9], [0, 3, 6, 10], [-1, 3, 6, 9]):   # bad runs
        before = [t.clone() for t in c.codes + c.scales]
        seq = ints([5, 6, 7])
        K.kvsel_kv4_append(c.kv, c.table, seq, ints(off), x, x, ws)
        assert K.read_status(ws) == K.KVSEL_ERR_BAD_INDEX
    bad = c.table.clone()
    bad[0, 0], bad[2, 0] = 10 ** 6, -1
    before = [t.clone() for t in c.codes + c.scales]
    seq = ints([5, 6, 7])
    K.kvsel_kv4_append(c.kv, bad, seq, ints([0, 3, 6, 9]), x, x, ws)
    assert K.read_status(ws) == K.KVSEL_ERR_BAD_INDEX
    # rows for bad pages go nowhere; sequence 1 gets the rows that an earlier call put there
    assert seq.tolist() == [8, 9, 10] and unchanged(0) and unchanged(1) and unchanged(2)
    out = [torch.full((4, 2, D), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    K.kvsel_kv4_read(c.kv, c.table, ints([5, 6, 7]), ints([0, 2, 4, 4]), out[0], out[1], ws, start=ints([4, 2, 0]))
    assert K.read_status(ws) == K.KVSEL_ERR_BAD_INDEX    # slot 5 of sequence 0 is not live
    assert bool((out[0][1] == 3.0).all()) and not bool((out[0][0] == 3.0).any())
    c.g.check()


def test_empty_append_is_a_no_op():
    c = Cache(np.random.default_rng(1), 2, 1, 1, 16, 20)
    ws = K.workspace(512)
    x = torch.zeros(0, 1, D, dtype=torch.bfloat16, device="cuda")
    seq = ints([3, 4])
    K.kvsel_kv4_append(c.kv, c.table, seq, ints([0, 0, 0]), x, x, ws)
    assert K.read_status(ws) == 0 and seq.tolist() == [3, 4]


# ----------------------------------------------------------------------------------------------------------------------
# decode
# ----------------------------------------------------------------------------------------------------------------------
def _bounds(q, k, v, s_n, z_abs, vs_n, vz_abs, p, scale, softcap, bias):
    """(relative bound of p [G], absolute bound of out [G, 128]) from the module's derivation; s_n = s * n of the keys."""
    A = np.max(np.abs(q) @ (s_n + z_abs).T, axis=1) * abs(scale) if k.shape[0] else np.zeros(q.shape[0])
    t = 2.0 ** -18 * A + 2.0 ** -22 * softcap + 2.0 ** -22 * bias
    rel = 2 * t + 2.0 ** -18
    out = 2.0 ** -11 * (p @ vs_n) + (rel[:, None] + 2.0 ** -18) * (p @ (vs_n + vz_abs)) + 2.0 ** -38 * np.max(vs_n, initial=0.0)
    return rel, out


def _check_decode(c, st, S, pos, pos_q, scale, softcap, slopes, window, n_sink, out, probs, cum, cum0, new_slot):
    G = c.Hq // c.Hkv
    for b in range(c.B):
        n = S[b]
        for h in range(c.Hkv):
            kc, ks, kz = c.rows(b, h, n, 0)
            vc, vs, vz = c.rows(b, h, n, 1)
            k, v = kv4.values(kc, ks, kz), kv4.values(vc, vs, vz)
            q = st["q"][b, h * G:(h + 1) * G].double().cpu().numpy()
            sl = None if slopes is None else slopes[h * G:(h + 1) * G].astype(np.float64)
            if n == 0:
                assert np.all(out[b, h * G:(h + 1) * G] == 0)
                continue
            o, p = kv4.decode(q, k, v, scale, pos[b, h, :n], pos_q[b][h], softcap, sl, window, n_sink)
            seen = p.sum(0) > 0
            rep = lambda a: np.repeat(a, 32, -1)  # noqa: E731
            bias = 0.0 if sl is None else float(np.max(sl) * np.max(np.abs(pos_q[b][h] - pos[b, h, :n])))
            fin = np.isfinite(kz).all(1) & np.isfinite(vz).all(1)
            assert fin[seen].all()
            m = seen
            rel, bound = _bounds(q, k[m], v[m], kc[m] * rep(ks[m]), rep(np.abs(kz[m])), vc[m] * rep(vs[m]),
                                 rep(np.abs(vz[m])), p[:, m], scale, softcap, bias)
            got = out[b, h * G:(h + 1) * G]
            assert np.all(np.abs(got - o) <= bound), (b, h, float(np.max(np.abs(got - o) / bound)))
            if probs is not None:
                gp = probs[b, h * G:(h + 1) * G, :n]
                assert np.all(np.abs(gp - p) <= rel[:, None] * p + 1e-37), (b, h)
            if cum is not None:
                want = cum0[b, h, :n].astype(np.float64).copy()
                if new_slot is not None:
                    want[new_slot[b]] = 0.0
                want += p.sum(0)
                assert np.all(np.abs(cum[b, h, :n] - want) <= rel.max() * p.sum(0) + 2.0 ** -20 * want + 1e-37), (b, h)


def _decode_case(G, Hkv, page, S, *, append=True, softcap=0.0, alibi=False, window=0, n_sink=0, mapped=False, probs=True,
                 cum=True, out_f32=True, cap_extra=0, seed=0, spoil=False, scale=None, big_v=False):
    rng = np.random.default_rng(seed)
    B, Hq = len(S), G * Hkv
    cap = max(max(S), 1) + cap_extra
    c = Cache(rng, B, Hkv, Hq, page, cap)
    if big_v:          # value scales over 30 binades
        c.scales[1].mul_(torch.from_numpy(2.0 ** rng.integers(-15, 15, c.scales[1].shape[:-1] + (1,))).cuda().to(c.scales[1].dtype))
    live = [s - 1 for s in S] if append else list(S)
    st = dict(q=bf(rng.standard_normal((B, Hq, D)) * 1.3).cuda())
    kn, vn = bf(rng.standard_normal((B, Hkv, D))).cuda(), bf(rng.standard_normal((B, Hkv, D))).cuda()
    pos_np = np.tile(np.arange(cap), (B, Hkv, 1))
    nxt = None
    pm = None
    if mapped:
        pos_np = np.cumsum(rng.integers(1, 5, (B, Hkv, cap)), -1) - 1
        nxt_np = pos_np.max((1, 2)) + 3
        pm = c.g.like(ints(pos_np))
        nxt = c.g.like(ints(nxt_np)) if append else None
    pos_q = [[(int(nxt_np[b]) if append else int(pos_np[b, h, S[b] - 1])) if mapped else S[b] - 1 for h in range(Hkv)]
             for b in range(B)]
    if mapped and append:
        for b in range(B):
            pos_np[b, :, S[b] - 1] = nxt_np[b]
    seen_np = (np.asarray(pos_q)[:, :, None] - pos_np < window) | (pos_np < n_sink) if window else None
    if spoil:          # NaN in every dead slot and in every live one that the window hides
        for b in range(B):
            for s in range(c.pages * page):
                p = int(c.table_np[b, s // page])
                for h in range(Hkv):
                    if s >= S[b] or (window and not seen_np[b, h, s]):
                        if append and s == S[b] - 1:
                            continue
                        c.scales[0][p, h, s % page] = float("nan")
                        c.scales[1][p, h, s % page] = float("inf")
    slopes = (2.0 ** (-8.0 * (np.arange(Hq) + 1) / Hq)).astype(np.float32) if alibi else None
    cum0 = rng.random((B, Hkv, cap)).astype(np.float32)
    seq = c.g.like(ints(live))
    out = c.g.new((B, Hq, D), torch.float32 if out_f32 else torch.bfloat16, 7.0)
    pr = c.g.new((B, Hq, cap), torch.float32, -4.0) if probs else None
    cm = c.g.like(torch.from_numpy(cum0).cuda()) if cum else None
    need = K.kvsel_kv4_decode_attn_workspace(c.kv, B, cap, probs, cum)
    ws = c.g.new((need,), torch.uint8)
    sc = D ** -0.5 if scale is None else scale
    K.kvsel_kv4_decode_attn(c.kv, c.table, seq, st["q"], out, ws, k_new=kn if append else None, v_new=vn if append else None,
                            pos_map=pm, next_pos=nxt, scale=sc, softcap=softcap,
                            slopes=None if slopes is None else torch.from_numpy(slopes).cuda(), window=window,
                            n_sink=n_sink, probs=pr, h2o_cum=cm, max_len=cap)
    assert K.read_status(ws) == 0
    assert seq.tolist() == list(S)
    if append:   # the appended rows are the format's
        for b in range(B):
            for side, x in ((0, kn), (1, vn)):
                want = kv4.quantise_rows(x[b].double().cpu().numpy())
                for h in range(Hkv):
                    got = [a[-1] for a in c.rows(b, h, S[b], side)]
                    assert all(np.array_equal(w[h], y) for w, y in zip(want, got))
        if mapped:
            assert nxt.tolist() == (nxt_np + 1).tolist()
            for b in range(B):
                assert pm[b, :, S[b] - 1].tolist() == [int(nxt_np[b])] * Hkv
    c.g.check()
    o = out.double().cpu().numpy()
    if not out_f32:
        return c, o
    pn = pr.double().cpu().numpy() if probs else None
    _check_decode(c, st, S, pos_np, pos_q, sc, softcap, slopes, window, n_sink, o, pn, cm.double().cpu().numpy() if cum else None,
                  cum0, [s - 1 for s in S] if append else None)
    for b in range(B):   # nothing behind the live slots is written
        if probs:
            assert np.all(pn[b, :, S[b]:] == -4.0)
        if cum:
            assert np.array_equal(cm[b, :, S[b]:].cpu().numpy(), cum0[b, :, S[b]:])
    return c, o


@pytest.mark.parametrize("G,Hkv", [(1, 4), (2, 2), (4, 1), (5, 2), (7, 3), (8, 2), (9, 1), (12, 2), (16, 1)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_decode_heads_and_pages(G, Hkv, page):
    _decode_case(G, Hkv, page, [1, 31, 32, 33, 300], seed=G * 31 + page)


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("S", [[1], [2], [16, 17], [64], [65, 1], [1999]])
def test_decode_lengths(S, append):
    _decode_case(4, 2, 32, S, append=append, seed=S[0], cap_extra=5)


def test_decode_without_keys():
    _decode_case(2, 2, 16, [0, 5, 0], append=False)
    _decode_case(2, 2, 16, [0], append=False, probs=False, cum=False)


@pytest.mark.parametrize("kw", [dict(softcap=30.0), dict(softcap=2.0), dict(alibi=True), dict(window=1), dict(window=40),
                                dict(window=40, n_sink=4), dict(window=33, n_sink=70), dict(window=500, n_sink=1),
                                dict(softcap=50.0, alibi=True, window=100, n_sink=3),
                                dict(alibi=True, mapped=True), dict(window=90, n_sink=5, mapped=True),
                                dict(window=90, mapped=True, append=False, alibi=True)])
@pytest.mark.parametrize("G", [3, 16])
def test_decode_modified_scores(kw, G):
    _decode_case(G, 2, 16, [400, 77, 33, 1], spoil=True, seed=5, cap_extra=3, **kw)


def test_append_is_the_format_on_many_rows():
    """Scales and codes next to their borders: quarter steps, a wide spread of magnitudes, plain normals."""
    rng = np.random.default_rng(77)
    rows, Hkv = 96, 2
    for kind in ("grid", "wide", "normal"):
        c = Cache(rng, 1, Hkv, Hkv, 32, rows)
        x = _inputs(rng, kind, rows * Hkv)
        if kind == "normal":      # maxima that are 15 bf16 borders above the minimum
            x = x.view(rows, Hkv, 4, 32).clone()
            lo = x.amin(-1).float()
            step = torch.from_numpy(2.0 ** rng.integers(-6, 3, lo.shape) * (1 + (2 * rng.integers(0, 128, lo.shape) + 1) / 256.0))
            x[..., 0] = (lo + 15 * step.float()).bfloat16()
            x = x.view(rows * Hkv, D)
        xd = x.view(rows, Hkv, D).cuda()
        seq, ws = ints([0]), K.workspace(512)
        K.kvsel_kv4_append(c.kv, c.table, seq, ints([0, rows]), xd, xd, ws)
        assert K.read_status(ws) == 0
        want = kv4.quantise_rows(x.double().numpy())
        for h in range(Hkv):
            for side in range(2):
                codes, s, z = c.rows(0, h, rows, side)
                assert np.array_equal(s, want[1][h::Hkv]) and np.array_equal(z, want[2][h::Hkv]), kind
                assert np.array_equal(codes, want[0][h::Hkv]), kind


@pytest.mark.parametrize("probs,cum", [(True, False), (False, True), (False, False)])
def test_decode_outputs_are_optional(probs, cum):
    _decode_case(8, 2, 16, [130, 64], probs=probs, cum=cum, seed=3)


def test_decode_no_nan_from_dead_slots_and_extreme_scales():
    _decode_case(8, 2, 64, [100, 3], spoil=True, seed=6)
    _decode_case(4, 2, 16, [300], big_v=True, seed=7)
    _decode_case(4, 1, 16, [40], scale=0.0, seed=8)
    _decode_case(4, 1, 16, [40], scale=-0.3, seed=9)


def test_decode_nan_in_a_seen_key_reaches_its_heads_only():
    rng = np.random.default_rng(4)
    c = Cache(rng, 1, 2, 4, 16, 50)
    c.scales[0][int(c.table_np[0, 1]), 0, 3, 2] = float("nan")      # slot 19, kv head 0
    out = torch.zeros(1, 4, D, device="cuda")
    ws = K.workspace(K.kvsel_kv4_decode_attn_workspace(c.kv, 1, 50, False, False))
    q = bf(rng.standard_normal((1, 4, D))).cuda()
    K.kvsel_kv4_decode_attn(c.kv, c.table, ints([50]), q, out, ws, max_len=50)
    assert bool(torch.isnan(out[0, :2]).all()) and bool(torch.isfinite(out[0, 2:]).all())


def test_decode_large_q_and_bf16_out():
    """q far outside fp16's range: its power-of-two scale keeps the product exact."""
    rng = np.random.default_rng(11)
    c = Cache(rng, 1, 1, 2, 16, 70)
    ws = K.workspace(K.kvsel_kv4_decode_attn_workspace(c.kv, 1, 70, False, False))
    q = rng.standard_normal((1, 2, D))
    outs = []
    for e in (0, 90, -90):
        out = torch.zeros(1, 2, D, device="cuda")
        K.kvsel_kv4_decode_attn(c.kv, c.table, ints([70]), bf(q * 2.0 ** e).cuda(), out, ws, scale=0.05 * 2.0 ** -e, max_len=70)
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    out16 = torch.zeros(1, 2, D, dtype=torch.bfloat16, device="cuda")
    K.kvsel_kv4_decode_attn(c.kv, c.table, ints([70]), bf(q).cuda(), out16, ws, scale=0.05, max_len=70)
    assert torch.equal(out16, outs[0].bfloat16())


def test_decode_many_warps_share_a_row():
    """One long row over every warp of the GPU, and many short rows: partials are joined."""
    _decode_case(2, 1, 256, [9000], seed=12, append=False)
    _decode_case(1, 8, 16, [40] * 100, seed=13)


@pytest.mark.parametrize("S", [2048, 2080, 3100, 3600, 9000])
@pytest.mark.parametrize("G,window", [(1, 0), (8, 0), (3, 40), (16, 1)])
def test_decode_joins_few_and_many_partials(S, G, window):
    """Around 64 and 96 partials, with windows that leave most of them empty."""
    _decode_case(G, 1, 64, [S], seed=S + G, append=False, window=window, n_sink=2 if window else 0)


def test_decode_reports_lengths_and_pages_that_do_not_fit():
    rng = np.random.default_rng(14)
    c = Cache(rng, 3, 2, 4, 16, 64)
    ws = K.workspace(K.kvsel_kv4_decode_attn_workspace(c.kv, 3, 64, True, True))
    q, kn = bf(rng.standard_normal((3, 4, D))).cuda(), bf(rng.standard_normal((3, 2, D))).cuda()
    probs, cum = torch.full((3, 4, 64), -1.0, device="cuda"), torch.zeros(3, 2, 64, device="cuda")
    out = torch.full((3, 4, D), 7.0, device="cuda")
    seq = ints([10, 64, -1])                                        # 64 + 1 does not fit, -1 is no length
    K.kvsel_kv4_decode_attn(c.kv, c.table, seq, q, out, ws, k_new=kn, v_new=kn, probs=probs, h2o_cum=cum)
    assert K.read_status(ws) == K.KVSEL_ERR_BAD_INDEX
    assert seq.tolist() == [11, 64, -1]
    assert bool((out[1:] == 7.0).all()) and bool((probs[1:] == -1.0).all()) and bool(torch.isfinite(out[0]).all())
    good = torch.zeros(3, 4, D, device="cuda")
    K.kvsel_kv4_decode_attn(c.kv, c.table, ints([32, 32, 32]), q, good, ws, max_len=64)
    bad = c.table.clone()
    bad[1, 2:] = -1                                                 # pages behind the length do not matter
    K.kvsel_kv4_decode_attn(c.kv, bad, ints([32, 32, 32]), q, out, ws, max_len=64)
    assert K.read_status(ws) == 0 and torch.equal(out, good)
    bad[1, 1] = 10 ** 6
    K.kvsel_kv4_decode_attn(c.kv, bad, ints([32, 32, 32]), q, out, ws, max_len=64)
    assert K.read_status(ws) == K.KVSEL_ERR_BAD_INDEX
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    K.kvsel_kv4_decode_attn(c.kv, c.table, ints([16, 16, 16]), q, good, ws, max_len=64)
    assert torch.equal(out[1], good[1])                             # keys on the bad page are not seen


# ----------------------------------------------------------------------------------------------------------------------
# evict
# ----------------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("S,budget,sink,window,page", [([40], 20, 4, 8, 16), ([300, 20, 299], 100, 4, 32, 16),
                                                       ([1000, 999], 999, 1, 0, 64), ([9100], 8000, 4, 100, 256),
                                                       ([5000, 70], 64, 0, 64, 32), ([500], 33, 33, 0, 16)])
@pytest.mark.parametrize("mapped", [False, True])
def test_evict_keeps_what_the_oracle_keeps(S, budget, sink, window, page, mapped):
    rng = np.random.default_rng(S[0] + budget)
    B, Hkv, cap = len(S), 2, max(S) + 3
    c = Cache(rng, B, Hkv, 2 * Hkv, page, cap)
    cum_np = np.round(np.exp(2 * rng.standard_normal((B, Hkv, cap))) * 4) / 4          # ties
    cum_np = cum_np.astype(np.float32)
    pos_np = (np.cumsum(rng.integers(1, 4, (B, Hkv, cap)), -1) if mapped else np.tile(np.arange(cap), (B, Hkv, 1))).astype(np.int32)
    seq, cum, pos = c.g.like(ints(S)), c.g.like(torch.from_numpy(cum_np).cuda()), c.g.like(ints(pos_np))
    keep, freed = c.g.new((B, Hkv, budget), torch.int32, -5), c.g.new((B, c.pages), torch.int32, -5)
    ws = c.g.new((K.kvsel_kv4_evict_workspace(c.kv, B, budget),), torch.uint8)
    rows = {(b, h, side): c.rows(b, h, S[b], side) for b in range(B) for h in range(Hkv) for side in range(2)}
    K.kvsel_kv4_evict(c.kv, c.table, seq, cum, ws, budget=budget, n_sink=sink, window=window, pos_map=pos if mapped else None,
                      keep_out=keep)                              # select only: nothing moves
    assert seq.tolist() == S and torch.equal(cum, torch.from_numpy(cum_np).cuda())
    first = keep.clone()
    K.kvsel_kv4_evict(c.kv, c.table, seq, cum, ws, budget=budget, n_sink=sink, window=window, compact=True,
                      pos_map=pos if mapped else None, keep_out=keep, freed_pages=freed)
    assert K.read_status(ws) == 0
    assert torch.equal(keep, first)
    assert seq.tolist() == [min(s, budget) for s in S]
    for b in range(B):
        n = min(S[b], budget)
        old, new = (S[b] + page - 1) // page, (n + page - 1) // page
        tb = c.table[b].tolist()
        assert tb[:new] == c.table_np[b, :new].tolist() and tb[new:old] == [-1] * (old - new)
        assert tb[old:] == c.table_np[b, old:].tolist()
        assert freed[b].tolist() == c.table_np[b, new:old].tolist() + [-1] * (c.pages - (old - new))
        for h in range(Hkv):
            slots = h2o.h2o_keep(cum_np[b, h], S[b], budget, sink, window)
            want = pos_np[b, h, slots] if mapped else slots
            assert keep[b, h].tolist() == want.tolist() + [-1] * (budget - n)
            assert np.array_equal(cum[b, h, :n].cpu().numpy(), cum_np[b, h, slots])
            if mapped:
                assert pos[b, h, :n].tolist() == want.tolist()
            for side in range(2):
                for was, now in zip(rows[b, h, side], c.rows(b, h, n, side)):
                    assert np.array_equal(was[slots], now)
            assert np.array_equal(cum[b, h, n:].cpu().numpy(), cum_np[b, h, n:])   # behind the kept slots: as it was
    c.g.check()


def test_evict_of_one_long_row_and_of_many_rows():
    """More chunks than the grid holds at once, of one row and of many; every kept row arrives whole."""
    for B, Hkv, S, budget, page in ((1, 1, 160001, 150017, 256), (5, 7, 9000, 6000, 64)):
        rng = np.random.default_rng(B)
        pages = (S + page - 1) // page
        table_np = rng.permutation(B * pages).astype(np.int32).reshape(B, pages)
        gen = torch.Generator(device="cuda").manual_seed(B)
        codes = [torch.randint(0, 256, (B * pages, Hkv, page, 64), generator=gen, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.randn(B * pages, Hkv, page, 4, 2, generator=gen, device="cuda").bfloat16() for _ in range(2)]
        table, seq = ints(table_np), ints([S] * B)
        cum = torch.rand(B, Hkv, S, generator=gen, device="cuda")
        pos = torch.arange(S, dtype=torch.int32, device="cuda").expand(B, Hkv, S).contiguous()

        def rows(pool, t, n):
            return pool[t.long()].transpose(1, 2).flatten(2, 3)[:, :, :n].clone()
        before, cum0 = [rows(p, table, S) for p in codes + scales], cum.clone()
        keep = torch.zeros(B, Hkv, budget, dtype=torch.int32, device="cuda")
        kv = K.paged_kv4(*codes, *scales, Hkv)
        ws = K.workspace(K.kvsel_kv4_evict_workspace(kv, B, budget))
        t0 = table.clone()
        K.kvsel_kv4_evict(kv, table, seq, cum, ws, budget=budget, n_sink=4, window=100, compact=True, pos_map=pos, keep_out=keep)
        assert K.read_status(ws) == 0 and seq.tolist() == [budget] * B
        for b in range(B):
            for h in range(Hkv):
                want = h2o.h2o_keep(cum0[b, h].cpu().numpy(), S, budget, 4, 100)
                assert np.array_equal(keep[b, h].cpu().numpy(), want)
        at = keep.long()
        for was, pool in zip(before, codes + scales):
            now = rows(pool, t0, budget)
            idx = at.view(B, Hkv, budget, *[1] * (was.dim() - 3)).expand(B, Hkv, budget, *was.shape[3:])
            assert torch.equal(now, was.gather(2, idx))
        assert torch.equal(cum[:, :, :budget], cum0.gather(2, at)) and torch.equal(pos[:, :, :budget], keep)


@pytest.mark.parametrize("S,budget,sink,window", [([70000, 500, 66001, 20, 69999], 4000, 4, 300), ([70000], 69999, 0, 0),
                                                  ([65537, 70000], 1, 0, 0), ([70000, 3000], 3000, 1000, 2000),
                                                  ([70000], 30000, 7, 29993), ([69000], 50000, 0, 5)])
def test_evict_of_rows_in_long_buffers(S, budget, sink, window):
    """Rows that may exceed 64K slots are selected by many CTAs each: ties, short rows, every budget's edges."""
    rng = np.random.default_rng(budget)
    B, Hkv, cap, page = len(S), 2, 70000, 256
    pages = (cap + page - 1) // page
    table = ints(rng.permutation(B * pages).reshape(B, pages))
    codes = [torch.from_numpy(rng.integers(0, 256, (B * pages, Hkv, page, 64), dtype=np.uint8)).cuda() for _ in range(2)]
    scales = [torch.zeros(B * pages, Hkv, page, 4, 2, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cum_np = np.exp(2 * rng.standard_normal((B, Hkv, cap))).astype(np.float32)
    cum_np = np.where(rng.random(cum_np.shape) < 0.5, np.floor(cum_np * 2) / 2, cum_np).astype(np.float32)   # many ties
    cum_np[0, 0] = 1.0                                                                                       # and only ties
    kv = K.paged_kv4(*codes, *scales, Hkv)
    g = Guards()
    ws = g.new((K.kvsel_kv4_evict_workspace(kv, B, budget),), torch.uint8)
    keep, freed = g.new((B, Hkv, budget), torch.int32, -5), g.new((B, pages), torch.int32, -5)
    seq, cum = g.like(ints(S)), g.like(torch.from_numpy(cum_np).cuda())
    rows = codes[0][table.long()].transpose(1, 2).flatten(2, 3).clone()
    t0 = table.clone()
    K.kvsel_kv4_evict(kv, table, seq, cum, ws, budget=budget, n_sink=sink, window=window, compact=True, keep_out=keep,
                      freed_pages=freed)
    assert K.read_status(ws) == 0 and seq.tolist() == [min(s, budget) for s in S]
    g.check()
    now = codes[0][t0.long()].transpose(1, 2).flatten(2, 3)
    for b in range(B):
        n = min(S[b], budget)
        for h in range(Hkv):
            want = h2o.h2o_keep(cum_np[b, h], S[b], budget, sink, window)
            assert keep[b, h].tolist() == want.tolist() + [-1] * (budget - n), (b, h)
            at = torch.from_numpy(want).cuda()
            assert torch.equal(now[b, h, :n], rows[b, h, at]) and torch.equal(cum[b, h, :n], torch.from_numpy(cum_np[b, h, want]).cuda())


@pytest.mark.parametrize("B,Hkv,cap", [(1, 2, 33000), (1, 3, 99000), (1, 3, 101000), (4, 8, 101000), (3, 11, 101000)])
def test_evict_selects_the_same_however_a_row_is_spread(B, Hkv, cap):
    """Rows on both sides of the rule that spreads a row over many CTAs, full ones and short ones."""
    rng = np.random.default_rng(cap + B)
    budget, sink, window, page = 500, 4, 60, 16
    kv = K.paged_kv4(*[torch.zeros(B, Hkv, page, 64, dtype=torch.uint8, device="cuda") for _ in range(2)],
                     *[torch.zeros(B, Hkv, page, 4, 2, dtype=torch.bfloat16, device="cuda") for _ in range(2)], Hkv)
    pages = (cap + page - 1) // page
    cum_np = rng.random((B, Hkv, cap)).astype(np.float32)
    cum_np[..., ::7] = 0.9975                                  # ties, which the long rows' last kept scores are among
    S = [cap if b % 2 == 0 else 900 + b for b in range(B)]
    g = Guards()
    ws = g.new((K.kvsel_kv4_evict_workspace(kv, B, budget),), torch.uint8)
    keep, seq, cum = g.new((B, Hkv, budget), torch.int32, -5), g.like(ints(S)), g.like(torch.from_numpy(cum_np).cuda())
    K.kvsel_kv4_evict(kv, torch.zeros(B, pages, dtype=torch.int32, device="cuda"), seq, cum, ws, budget=budget, n_sink=sink,
                      window=window, compact=False, keep_out=keep)
    assert K.read_status(ws) == 0 and seq.tolist() == S
    g.check()
    for b in range(B):
        for h in range(Hkv):
            assert keep[b, h].tolist() == h2o.h2o_keep(cum_np[b, h], S[b], budget, sink, window).tolist(), (b, h)


def test_evict_in_chunks_whose_wait_may_run_out_ends():
    """As below, with more kept rows than the clusters move."""
    for limit in (1, 0):
        c = Cache(np.random.default_rng(2), 2, 2, 2, 16, 9000)
        ws = K.workspace(K.kvsel_kv4_evict_workspace(c.kv, 2, 8000))
        seq = ints([9000, 9000])
        K.set_wait_limit(ws, limit)
        K.kvsel_kv4_evict(c.kv, c.table, seq, torch.rand(2, 2, 9000, device="cuda"), ws, budget=8000, n_sink=4, window=50, compact=True)
        assert K.read_status(ws) in ((0, K.KVSEL_ERR_TIMEOUT) if limit else (0,))
        if not limit:
            assert seq.tolist() == [8000, 8000]
        c.g.check()


def test_evict_whose_wait_may_run_out_ends():
    """With a wait of one poll the move ends at once, with KVSEL_ERR_TIMEOUT where a chunk was not ready."""
    rng = np.random.default_rng(2)
    c = Cache(rng, 2, 2, 2, 16, 4000)
    ws = K.workspace(K.kvsel_kv4_evict_workspace(c.kv, 2, 3500))
    cum = torch.rand(2, 2, 4000, device="cuda")
    K.set_wait_limit(ws, 1)
    K.kvsel_kv4_evict(c.kv, c.table, ints([4000, 4000]), cum, ws, budget=3500, n_sink=4, window=50, compact=True)
    assert K.read_status(ws) in (0, K.KVSEL_ERR_TIMEOUT)
    K.set_wait_limit(ws, 0)
    c2 = Cache(np.random.default_rng(2), 2, 2, 2, 16, 4000)
    seq = ints([4000, 4000])
    K.kvsel_kv4_evict(c2.kv, c2.table, seq, torch.rand(2, 2, 4000, device="cuda"), ws, budget=3500, n_sink=4, window=50, compact=True)
    assert K.read_status(ws) == 0 and seq.tolist() == [3500, 3500]
    c.g.check()
    c2.g.check()


def test_evict_reports_what_does_not_fit():
    rng = np.random.default_rng(3)
    c = Cache(rng, 2, 1, 1, 16, 64)
    ws = K.workspace(K.kvsel_kv4_evict_workspace(c.kv, 2, 20))
    cum = torch.rand(2, 1, 60, device="cuda")
    before = [t.clone() for t in c.codes + c.scales]
    K.kvsel_kv4_evict(c.kv, c.table, ints([61, -3]), cum, ws, budget=20, n_sink=2, window=4, compact=True)
    assert K.read_status(ws) == K.KVSEL_ERR_BAD_INDEX
    assert all(torch.equal(a, b) for a, b in zip(before, c.codes + c.scales))


# ----------------------------------------------------------------------------------------------------------------------
# together
# ----------------------------------------------------------------------------------------------------------------------
class _Run:
    """Prompts into the cache, decode steps that gather H2O scores, eviction, further steps at mapped positions."""

    def __init__(self, seed=0):
        rng = np.random.default_rng(seed)
        self.B, self.Hkv, self.G, self.page, self.cap, self.budget = 3, 2, 4, 16, 160, 60
        self.lens = [101, 48, 130]
        Hq = self.Hkv * self.G
        self.c = Cache(rng, self.B, self.Hkv, Hq, self.page, self.cap)
        total = sum(self.lens)
        self.k, self.v = (bf(rng.standard_normal((total, self.Hkv, D))).cuda() for _ in range(2))
        self.off = ints(np.concatenate([[0], np.cumsum(self.lens)]))
        self.n = 6
        self.q = bf(rng.standard_normal((self.n, self.B, Hq, D)) * 1.3).cuda()
        self.kn, self.vn = (bf(rng.standard_normal((self.n, self.B, self.Hkv, D))).cuda() for _ in range(2))
        self.seq, self.nxt = ints([0] * self.B), ints([0] * self.B)
        self.cum = torch.full((self.B, self.Hkv, self.cap), 3.0, device="cuda")
        self.pos = torch.full((self.B, self.Hkv, self.cap), -1, dtype=torch.int32, device="cuda")
        self.out = torch.zeros(self.n, self.B, Hq, D, device="cuda")
        self.keep = torch.zeros(self.B, self.Hkv, self.budget, dtype=torch.int32, device="cuda")
        self.slopes = torch.tensor([2.0 ** -(h + 1) for h in range(Hq)], device="cuda")
        self.ws = K.workspace(K.kvsel_kv4_decode_attn_workspace(self.c.kv, self.B, self.cap, False, True))
        self.ws_ap = K.workspace(K.kvsel_kv4_append_workspace(self.c.kv, self.B))
        self.ws_ev = K.workspace(K.kvsel_kv4_evict_workspace(self.c.kv, self.B, self.budget))

    def go(self):
        c = self.c
        K.kvsel_kv4_append(c.kv, c.table, self.seq, self.off, self.k, self.v, self.ws_ap, pos_map=self.pos,
                           next_pos=self.nxt, h2o_cum=self.cum)
        for i in range(self.n):
            if i == 3:
                K.kvsel_kv4_evict(c.kv, c.table, self.seq, self.cum, self.ws_ev, budget=self.budget, n_sink=4, window=10,
                                  compact=True, pos_map=self.pos, keep_out=self.keep)
            K.kvsel_kv4_decode_attn(c.kv, c.table, self.seq, self.q[i], self.out[i], self.ws, k_new=self.kn[i],
                                    v_new=self.vn[i], pos_map=self.pos, next_pos=self.nxt, softcap=20.0,
                                    slopes=self.slopes, h2o_cum=self.cum)

    def state(self):
        torch.cuda.synchronize()
        assert [K.read_status(w) for w in (self.ws, self.ws_ap, self.ws_ev)] == [0, 0, 0]
        return [t.clone() for t in (self.out, self.cum, self.pos, self.seq, self.nxt, self.keep, *self.c.codes, *self.c.scales)]


def test_a_run_of_the_operators_together():
    r = _Run()
    r.go()
    out, cum, pos, seq, nxt, keep = r.state()[:6]
    assert nxt.tolist() == [n + r.n for n in r.lens]
    table = r.c.table_np
    held = {}
    for side, (x, new) in enumerate(((r.k, r.kn), (r.v, r.vn))):
        held[side] = kv4.values(*kv4.quantise_rows(x.double().cpu().numpy().reshape(-1, D))).reshape(-1, r.Hkv, D)
        held[side, "new"] = kv4.values(*kv4.quantise_rows(new.double().cpu().numpy().reshape(-1, D))).reshape(r.n, r.B, r.Hkv, D)
    assert table is not None
    at = 0
    for b in range(r.B):
        n0 = r.lens[b]
        for h in range(r.Hkv):
            k, v = list(held[0][at:at + n0, h]), list(held[1][at:at + n0, h])
            p, c = list(range(n0)), [0.0] * n0
            for i in range(r.n):
                if i == 3 and len(p) > r.budget:
                    # select by the GPU's own scores would hide an error in them: the oracle's must agree but for near ties
                    sel = h2o.h2o_keep(np.array(c), len(p), r.budget, 4, 10)
                    got = keep[b, h].tolist()
                    assert got == [p[j] for j in sel]
                    k, v, p, c = [[a[j] for j in sel] for a in (k, v, p, c)]
                k.append(held[0, "new"][i, b, h])
                v.append(held[1, "new"][i, b, h])
                p.append(n0 + i)
                c.append(0.0)
                q = r.q[i, b, h * r.G:(h + 1) * r.G].double().cpu().numpy()
                sl = r.slopes[h * r.G:(h + 1) * r.G].double().cpu().numpy()
                o, pr = kv4.decode(q, np.array(k), np.array(v), D ** -0.5, np.array(p), n0 + i, 20.0, sl)
                c = (np.array(c) + pr.sum(0)).tolist()
                got = out[i, b, h * r.G:(h + 1) * r.G].double().cpu().numpy()
                # p s rounds to fp16 (2^-11); s n <= |v| + |z| is at most 3 times the largest |v| here
                assert np.all(np.abs(got - o) <= 2.0 ** -11 * 3 * np.max(np.abs(v))), (b, h, i)
            assert pos[b, h, :len(p)].tolist() == p
            assert np.allclose(cum[b, h, :len(p)].cpu().numpy(), c, rtol=1e-4, atol=1e-6)
        assert int(seq[b]) == len(p)
        at += n0


def test_the_run_replayed_from_a_graph_and_on_another_stream():
    eager = _Run(5)
    eager.go()
    want = eager.state()
    other = _Run(5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other.go()
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(other.state(), want):
        assert torch.equal(a, b)
    replayed = _Run(5)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        replayed.go()
    g.replay()
    for a, b in zip(replayed.state(), want):
        assert torch.equal(a, b)


def test_two_runs_interleaved_on_two_streams_with_workspaces_of_their_own():
    want = []
    for seed in (21, 22):
        r = _Run(seed)
        r.go()
        want.append(r.state())
    runs = [_Run(21), _Run(22)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for r, s in zip(runs, streams):
        with torch.cuda.stream(s):
            r.go()
    torch.cuda.synchronize()
    for r, w in zip(runs, want):
        for a, b in zip(r.state(), w):
            assert torch.equal(a, b)


def test_binding_checks_shapes_and_devices():
    rng = np.random.default_rng(0)
    c = Cache(rng, 2, 2, 4, 16, 32)
    ws = K.workspace(K.kvsel_kv4_decode_attn_workspace(c.kv, 2, 32, True, True))
    q, out, seq = torch.zeros(2, 4, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 4, D, device="cuda"), ints([3, 4])
    ok = dict(max_len=32)
    K.kvsel_kv4_decode_attn(c.kv, c.table, seq, q, out, ws, **ok)
    for bad in (dict(q=q[:, :3]), dict(q=q.float()), dict(out=out[:1]), dict(out=out.half()), dict(seq=seq[:1]),
                dict(q=q.cpu()), dict(seq=seq.cpu()), dict(q=q.transpose(0, 1).contiguous().transpose(0, 1))):
        a = dict(q=q, out=out, seq=seq)
        a.update(bad)
        with pytest.raises(ValueError):
            K.kvsel_kv4_decode_attn(c.kv, c.table, a["seq"], a["q"], a["out"], ws, **ok)
    for bad in (dict(probs=torch.zeros(2, 4, 31, device="cuda"), max_len=32), dict(h2o_cum=torch.zeros(2, 4, 32, device="cuda")),
                dict(slopes=torch.zeros(2, device="cuda")), dict(next_pos=ints([1])), dict(k_new=q[:, :2].contiguous()[:1])):
        with pytest.raises(ValueError):
            K.kvsel_kv4_decode_attn(c.kv, c.table, seq, q, out, ws, **bad)
    with pytest.raises(ValueError):
        K.kvsel_kv4_decode_attn(c.kv, c.table, seq, q, out, None, **ok)
    with pytest.raises(ValueError):
        K.paged_kv4(c.codes[0], c.codes[1][:1], c.scales[0], c.scales[1], 4)
    with pytest.raises(ValueError):
        K.paged_kv4(c.codes[0], c.codes[1], c.scales[0], c.scales[1].float(), 4)
    x = torch.zeros(3, 2, D, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        K.kvsel_kv4_append(c.kv, c.table, seq, ints([0, 1]), x, x, ws)
    with pytest.raises(ValueError):
        K.kvsel_kv4_read(c.kv, c.table, seq, ints([0, 1, 2]), x, x[:2], ws)
    with pytest.raises(ValueError):
        K.kvsel_kv4_evict(c.kv, c.table, seq, torch.zeros(2, 2, 32, device="cuda"), ws, budget=8, n_sink=1, window=2,
                          keep_out=torch.zeros(2, 2, 7, dtype=torch.int32, device="cuda"))
