"""Attention of prompt tokens over the paged bf16 cache against its fp64 oracle.

Bounds (out in fp32; every product of bf16 numbers is exact):
* a score is accumulated in fp32 over 8 matrix instructions of 16 terms; with A = scale * sum_d |q_d k_d| it is within
  2^-18 A, the cap adds 2^-20 cap (an approximate reciprocal and exponential), the bias 2^-22 of its size;
* exp(t - m) and the sums: a relative error of twice that and 2^-18;
* p is rounded to bf16 for the second product: half a step is 2^-8 of p (bf16 has eps 2^-7).
So out is within (2^-8 + rel) sum p |v|, and lse within the score's bound and 2^-18 of 1 + |lse|.
"""
import numpy as np
import pytest
import torch

from _harness import Guards
from oracle import kv4

import attention_guided_kv_gb300 as K

pytestmark = pytest.mark.gpu
D = 128


def bf(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float64)).bfloat16()


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def _case(G, Hkv, page, S, new, *, softcap=0.0, alibi=False, window=0, prefix=None, doc_start=None, out_f32=True, pad=0,
          seed=0, scale=None, spoil=True, with_lse=True, spare_table=0, stream=None):
    """Run one call and check it.  doc_start: per sequence, a list of the first position each query sees."""
    rng = np.random.default_rng(seed)
    B, Hq = len(S), G * Hkv
    pages = (max(max(S), 1) + page - 1) // page + spare_table
    n_pages = B * pages + 2
    table_np = rng.permutation(n_pages)[:B * pages].astype(np.int32).reshape(B, pages)
    g = Guards()
    pools = [g.like(bf(rng.standard_normal((n_pages, Hkv, page, D))).cuda()) for _ in range(2)]
    if spoil:            # what is no live key holds NaN
        live = torch.zeros(n_pages, page, dtype=torch.bool)
        for b in range(B):
            for s in range(S[b]):
                live[int(table_np[b, s // page]), s % page] = True
        dead = ~live.cuda()
        for p in pools:
            p.masked_fill_(dead[:, None, :, None], float("nan"))
    for b in range(B):   # entries behind the length are not looked at
        table_np[b, (S[b] + page - 1) // page:] = -1
    total = sum(new)
    q = bf(rng.standard_normal((total + pad, Hq, D)) * 1.3).cuda()
    off = np.concatenate([[0], np.cumsum(new)])
    slopes = (2.0 ** (-8.0 * (np.arange(Hq) + 1) / Hq)).astype(np.float32) if alibi else None
    ds = None
    if doc_start is not None:
        ds = np.concatenate([np.asarray(d) for d in doc_start] + [np.zeros(pad)]).astype(np.int64)
    out = g.new((total + pad, Hq, D), torch.float32 if out_f32 else torch.bfloat16, 7.0)
    lse = g.new((total + pad, Hq), torch.float32, 7.0) if with_lse else None
    kv = K.paged_kv(pools[0], pools[1], Hq)
    ws = g.new((max(256, K.kvsel_prefill_attn_workspace(kv, B, total + pad)),), torch.uint8)
    sc = D ** -0.5 if scale is None else scale
    seq = g.like(ints(S))
    K.kvsel_prefill_attn(kv, g.like(ints(table_np)), seq, q, ints(off), out, ws, scale=sc, softcap=softcap,
                         slopes=None if slopes is None else torch.from_numpy(slopes).cuda(), window=window,
                         prefix=None if prefix is None else ints(prefix), doc_start=None if ds is None else ints(ds), lse=lse,
                         stream=stream)
    assert K.read_status(ws) == 0
    g.check()
    assert bool((out[total:] == 7.0).all())
    got = out.double().cpu().numpy()
    gl = lse.double().cpu().numpy() if with_lse else None
    qn = q.double().cpu().numpy()
    for b in range(B):
        t = torch.from_numpy(table_np[b, :(S[b] + page - 1) // page].astype(np.int64)).cuda()
        rows = slice(off[b], off[b + 1])
        for h in range(Hkv):
            k, v = [p[t, h].reshape(-1, D)[:S[b]].double().cpu().numpy() for p in pools]
            for i in range(G):
                hq = h * G + i
                slope = 0.0 if slopes is None else float(slopes[hq])
                o, l = kv4.prefill(qn[rows, hq], k, v, sc, softcap, slope, window, 0 if prefix is None else prefix[b],
                                   None if ds is None else ds[rows])
                A = np.max(np.abs(qn[rows, hq]) @ np.abs(k).T, axis=1, initial=0.0) * sc
                err = 2.0 ** -18 * A + 2.0 ** -20 * softcap + 2.0 ** -22 * slope * max(S[b], 1)
                rel = 2 * err + 2.0 ** -18
                # sum p |v| <= max |v|; tighter: the same average over |v|
                oa, _ = kv4.prefill(qn[rows, hq], k, np.abs(v), sc, softcap, slope, window,
                                    0 if prefix is None else prefix[b], None if ds is None else ds[rows])
                bound = (2.0 ** -8 + rel[:, None] + (0 if out_f32 else 2.0 ** -8 * 1.02)) * oa + 1e-30
                bad = np.abs(got[rows, hq] - o) > bound
                assert not bad.any(), (b, hq, np.argwhere(bad)[:5], np.max(np.abs(got[rows, hq] - o) / bound))
                if with_lse:
                    x = gl[rows, hq]
                    assert np.array_equal(np.isneginf(x), np.isneginf(l))
                    f = np.isfinite(l)
                    assert np.all(np.abs(x[f] - l[f]) <= err[f] + 2.0 ** -18 * (1 + np.abs(l[f])))
    return out, lse


@pytest.mark.parametrize("G,Hkv", [(1, 3), (2, 1), (4, 2), (5, 1), (7, 2), (8, 1), (12, 1), (16, 1)])
def test_heads(G, Hkv):
    _case(G, Hkv, 16, [77, 200], [77, 40], seed=G)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_pages(page):
    _case(4, 2, page, [300, 1, 129], [300, 1, 65], seed=page, spare_table=1)


@pytest.mark.parametrize("S,new", [([1], [1]), ([128], [128]), ([127, 129], [127, 129]), ([256, 255, 257], [3, 255, 1]),
                                   ([640], [1]), ([500, 0, 30], [129, 0, 0]), ([5], [9]), ([0], [3])])
def test_lengths(S, new):
    """Whole prompts, chunks, single tokens, empty sequences, and more queries than keys (the first see nothing)."""
    _case(2, 2, 16, S, new, seed=S[0])


def test_padded_batch():
    _case(4, 1, 16, [60, 33], [60, 20], pad=5)


def test_many_rows_without_splits():
    """Enough query tiles that the keys are not split, tiles of both halves, odd ends."""
    _case(8, 2, 64, [700], [700], seed=3, softcap=30.0)


@pytest.mark.parametrize("kw", [dict(softcap=50.0), dict(softcap=1.5), dict(alibi=True), dict(window=1), dict(window=50),
                                dict(window=200, alibi=True), dict(prefix=[100, 7]), dict(prefix=[900, 0]),
                                dict(window=33, prefix=[90, 40], softcap=20.0), dict(window=20, prefix=[4, 4], alibi=True)])
@pytest.mark.parametrize("new", [[450, 300], [37, 5]])
def test_modified_scores(kw, new):
    _case(3, 2, 32, [450, 300], new, seed=9, **kw)


def test_documents_and_rows_that_see_nothing():
    S, new = [400, 260], [400, 200]
    docs = []
    for s, n in zip(S, new):
        edges = np.array([0, 3, 130, 131, 250])
        pos = np.arange(s - n, s)
        d = edges[np.searchsorted(edges, pos, side="right") - 1]
        d[-4:] = s + 10                          # left out
        d[1::50] = pos[1::50]                    # alone with themselves
        docs.append(d)
    out, lse = _case(4, 1, 16, S, new, doc_start=docs, seed=2)
    assert bool((out[396:400] == 0).all()) and bool(torch.isneginf(lse[396:400]).all())
    _case(4, 1, 16, S, new, doc_start=docs, prefix=[140, 20], window=64, alibi=True, softcap=9.0, seed=2)
    _case(4, 1, 16, S, new, doc_start=[np.full(400, 10 ** 6), np.full(200, 10 ** 6)], seed=2)   # nobody sees anything


def test_out_types_and_optional_lse():
    _case(4, 2, 16, [150], [150], out_f32=False)
    _case(4, 2, 16, [150], [20], out_f32=False, with_lse=False)


def test_scores_that_grow_along_the_keys():
    """Each key tile's scores exceed the last one's: the running maximum and O are rescaled tile by tile."""
    rng = np.random.default_rng(5)
    S, page = 1024, 16
    ramp = np.linspace(0.02, 3.0, S)[:, None]
    base = rng.standard_normal(D)
    for sign in (1.0, -1.0):
        k = bf(ramp * base * sign + 0.05 * rng.standard_normal((S, D))).cuda()
        v = bf(rng.standard_normal((S, D))).cuda()
        q = bf(np.tile(base, (300, 1)) + 0.05 * rng.standard_normal((300, D))).cuda()
        kv = K.paged_kv(k.view(-1, 1, page, D), v.view(-1, 1, page, D), 1)
        out, lse = torch.zeros(300, 1, D, device="cuda"), torch.zeros(300, 1, device="cuda")
        ws = K.workspace(K.kvsel_prefill_attn_workspace(kv, 1, 300))
        K.kvsel_prefill_attn(kv, ints([list(range(S // page))]), ints([S]), q.view(300, 1, D), ints([0, 300]), out, ws, scale=0.5,
                             lse=lse)
        assert K.read_status(ws) == 0
        qn, kn, vn = (x.double().cpu().numpy() for x in (q, k, v))
        o, l = kv4.prefill(qn, kn, vn, 0.5)
        oa, _ = kv4.prefill(qn, kn, np.abs(vn), 0.5)
        err = 2.0 ** -18 * 0.5 * np.max(np.abs(qn) @ np.abs(kn).T, axis=1)
        assert np.all(np.abs(out[:, 0].double().cpu().numpy() - o) <= (2.0 ** -8 + 2 * err[:, None] + 2.0 ** -18) * oa)
        assert np.all(np.abs(lse[:, 0].double().cpu().numpy() - l) <= err + 2.0 ** -18 * (1 + np.abs(l)))


def test_reports_what_does_not_fit():
    rng = np.random.default_rng(1)
    pool = bf(rng.standard_normal((8, 1, 16, D))).cuda()
    kv = K.paged_kv(pool, pool, 2)
    q = bf(rng.standard_normal((9, 2, D))).cuda()
    ws = K.workspace(K.kvsel_prefill_attn_workspace(kv, 3, 9))
    table = ints([[0, 1], [2, 3], [4, 5]])

    def run(S, off, t=table):
        out = torch.full((9, 2, D), 7.0, device="cuda")
        K.kvsel_prefill_attn(kv, t, ints(S), q, ints(off), out, ws)
        return K.read_status(ws), out
    st, good = run([20, 20, 20], [0, 3, 6, 9])
    assert st == 0 and not bool((good == 7.0).any())
    for S in ([20, 33, 20], [20, -1, 20]):
        st, out = run(S, [0, 3, 6, 9])
        assert st == K.KVSEL_ERR_BAD_INDEX
        assert bool((out[3:6] == 7.0).all()) and torch.equal(out[:3], good[:3]) and torch.equal(out[6:], good[6:])
    assert run([20, 20, 20], [0, 3, 6, 10])[0] == K.KVSEL_ERR_BAD_INDEX
    assert run([20, 20, 20], [-1, 3, 6, 9])[0] == K.KVSEL_ERR_BAD_INDEX
    many = torch.full((18, 2, D), 7.0, device="cuda")    # a bad length far behind the first CTA's sequence
    lens = [20] * 36
    lens[35] = 40
    ws2 = K.workspace(1 << 20)
    K.kvsel_prefill_attn(kv, table[:1].expand(36, 2).contiguous(), ints(lens), q.repeat(2, 1, 1), ints([0] * 2 + list(range(1, 18)) + [18] * 18),
                         many, ws2)
    assert K.read_status(ws2) == K.KVSEL_ERR_BAD_INDEX
    bad = table.clone()
    bad[1, 0] = 10 ** 6
    st, out = run([20, 20, 20], [0, 3, 6, 9], bad)
    assert st == K.KVSEL_ERR_BAD_INDEX and torch.equal(out[:3], good[:3]) and torch.equal(out[6:], good[6:])


class _Prompt:
    """A prompt in bf16 pages: prompt attention, then the same tokens into the 4-bit cache and a decode step there."""

    def __init__(self, seed):
        rng = np.random.default_rng(seed)
        self.S, page, Hkv, Hq, pages = [150, 70], 16, 2, 8, 11
        n = 2 * pages
        self.table = ints(rng.permutation(n).reshape(2, pages))
        self.pools = [bf(rng.standard_normal((n, Hkv, page, D))).cuda() for _ in range(2)]
        self.kv = K.paged_kv(*self.pools, Hq)
        total = sum(self.S)
        self.q, self.off, self.seq = bf(rng.standard_normal((total, Hq, D))).cuda(), ints([0, 150, total]), ints(self.S)
        self.out, self.lse = torch.zeros(total, Hq, D, device="cuda"), torch.zeros(total, Hq, device="cuda")
        self.ws = K.workspace(K.kvsel_prefill_attn_workspace(self.kv, 2, total))
        self.k, self.v = (self._packed(p) for p in self.pools)
        codes = [torch.zeros(n, Hkv, page, 64, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.zeros(n, Hkv, page, 4, 2, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        self.codes, self.scales = codes, scales
        self.kv4 = K.paged_kv4(*codes, *scales, Hq)
        self.seq4 = ints([0, 0])
        self.ws4 = K.workspace(K.kvsel_kv4_decode_attn_workspace(self.kv4, 2, 176, False, False))
        self.ws_ap = K.workspace(K.kvsel_kv4_append_workspace(self.kv4, 2))
        self.out4 = torch.zeros(2, Hq, D, device="cuda")
        self.last = torch.tensor([149, total - 1], device="cuda")
        self.q_last = self.q[self.last].contiguous()

    def _packed(self, pool):
        rows = []
        for b, s in enumerate(self.S):
            r = pool[self.table[b].long()].transpose(1, 2).flatten(0, 1)[:s]
            rows.append(r)
        return torch.cat(rows).contiguous()

    def go(self):
        K.kvsel_prefill_attn(self.kv, self.table, self.seq, self.q, self.off, self.out, self.ws, softcap=15.0, lse=self.lse)
        K.kvsel_kv4_append(self.kv4, self.table, self.seq4, self.off, self.k, self.v, self.ws_ap)
        K.kvsel_kv4_decode_attn(self.kv4, self.table, self.seq4, self.q_last, self.out4, self.ws4, softcap=15.0, max_len=176)

    def state(self):
        torch.cuda.synchronize()
        assert K.read_status(self.ws) == 0 and K.read_status(self.ws4) == 0 and K.read_status(self.ws_ap) == 0
        return [t.clone() for t in (self.out, self.lse, self.out4, self.seq4)]


def test_prompt_then_4_bit_cache_then_decode():
    r = _Prompt(3)
    r.go()
    out, lse, out4, seq4 = r.state()
    assert seq4.tolist() == r.S
    # the prompt's last row is a decode step: the same as over the cached values but for their quantisation
    last = out[r.last]
    # 4 bits of a normal's range: an error of a few percent of the output's size
    assert float((out4 - last).norm() / last.norm()) < 0.35
    # exactly: the decode over the values that the 4-bit cache stands for
    back = [torch.zeros_like(r.k) for _ in range(2)]
    K.kvsel_kv4_read(r.kv4, r.table, r.seq4, r.off, *back, r.ws4)
    at = 0
    for b, s in enumerate(r.S):
        for h in range(8):
            k, v = (x[at:at + s, h // 4].double().cpu().numpy() for x in back)
            o, _ = kv4.decode(r.q_last[b, h:h + 1].double().cpu().numpy(), k, v, D ** -0.5, np.arange(s), s - 1, 15.0)
            # read back in bf16: each k and v off by 2^-8 of itself, |dt| <= 2^-8 scale sum |q k|, and p s in fp16
            q = np.abs(r.q_last[b, h].double().cpu().numpy())
            dt = 2.0 ** -8 * D ** -0.5 * np.max(np.abs(k) @ q)
            assert np.all(np.abs(out4[b, h].double().cpu().numpy() - o[0]) <= (2 * dt + 2.0 ** -7) * np.max(np.abs(v)))
        at += s


def test_replayed_from_a_graph_and_on_another_stream():
    eager = _Prompt(4)
    eager.go()
    want = eager.state()
    other = _Prompt(4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other.go()
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(other.state(), want):
        assert torch.equal(a, b)
    rep = _Prompt(4)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rep.go()
    rep.seq4.zero_()
    g.replay()
    for a, b in zip(rep.state(), want):
        assert torch.equal(a, b)


def test_the_last_row_is_the_bf16_decode_step():
    """Without a cap the prompt's last row is what kvsel_decode_attn gives for that query over the same pages."""
    r = _Prompt(6)
    K.kvsel_prefill_attn(r.kv, r.table, r.seq, r.q, r.off, r.out, r.ws)
    ws = K.workspace(K.kvsel_decode_attn_workspace(r.kv, 2, 176, False))
    K.kvsel_decode_attn(r.kv, r.table, r.seq.clone(), r.q_last, r.out4, ws, max_len=176)
    assert K.read_status(ws) == 0 and K.read_status(r.ws) == 0
    top = max(float(p.abs().max()) for p in r.pools)
    assert float((r.out[r.last] - r.out4).abs().max()) <= 2 * 2.0 ** -8 * top      # both round p to bf16


def test_empty_call_and_shapes():
    r = _Prompt(7)
    empty = torch.zeros(0, 8, D, dtype=torch.bfloat16, device="cuda")
    K.kvsel_prefill_attn(r.kv, r.table, r.seq, empty, ints([0, 0, 0]), empty, r.ws)
    for bad in (dict(q=r.q[:, :7].contiguous()), dict(q=r.q.float()), dict(out=r.out[:5]), dict(off=ints([0, 1])),
                dict(lse=r.lse[:3]), dict(prefix=ints([1])), dict(doc=ints([0])), dict(q=r.q.cpu())):
        a = dict(q=r.q, out=r.out, off=r.off, lse=None, prefix=None, doc=None)
        a.update(bad)
        with pytest.raises(ValueError):
            K.kvsel_prefill_attn(r.kv, r.table, r.seq, a["q"], a["off"], a["out"], r.ws, lse=a["lse"], prefix=a["prefix"],
                                 doc_start=a["doc"])
