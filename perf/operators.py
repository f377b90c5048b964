"""Cases and plain forms of the 4-bit KV cache's operators and of the prompt attention with capped, biased and masked scores.

Operators:

* ``append``   quantise new K/V rows (one token a sequence, or whole ragged prompts) into a paged 4-bit cache, and read
               them back as the values that the cache now stands for.
* ``decode``   one query token per sequence against the 4-bit cache: capped, distance-biased or windowed scores, each
               key's probability, the H2O cumulative score, optionally the append of the new token.
* ``evict``    H2O eviction of a 4-bit cache by its accumulated attention weight: select, then compact in place; the kept
               rows are read back.
* ``prefill``  attention of a chunk of prompt tokens over the paged bf16 cache: causal, with a prefix that everyone sees,
               documents that do not see each other, a sliding window, a tanh cap and a bias that falls with distance.

The cache's number format: a row of 128 values is four groups of 32.  A group has the minimum ``z`` (bf16, exact), the scale
``s`` = (max - min) / 15 rounded to bf16 (below 2^-100: 0) and codes ``n`` = (x - z) / s rounded to nearest, ties to even,
held within 0..15 (0 where s is 0).  It stands for s * n + z.  Byte i of a row holds value 2i in its low half.
"""
import math

import torch

own = False

D = 128          # head dimension
GROUP = 32       # values that share a scale and a minimum
DEV = "cuda"


# ----------------------------------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # every sequence of a serving batch gets one token: nothing but latency
        dict(name="append_step", op="append", B=64, Hkv=8, page=16, ctx=1999, new=1, ragged=False),
        # prompts of several requests go into the cache at once, behind what is already there
        dict(name="append_prompts", op="append", B=6, Hkv=8, page=64, ctx=1001, new=9000, ragged=True),
        # one short conversation (16/8 heads): latency of a decode step that also keeps probabilities and H2O scores
        dict(name="decode_short", op="decode", B=1, Hq=16, Hkv=8, page=16, S=1600, ragged=False, cap=0.0, alibi=False,
             window=0, sink=0, append=True, evicted=False, probs=True, cum=True),
        # the 70B layer's step (64/8 heads, 8 x 32K) with H2O scores: the stream of the cache
        dict(name="decode_70b", op="decode", B=8, Hq=64, Hkv=8, page=16, S=32768, ragged=False, cap=0.0, alibi=False,
             window=0, sink=0, append=False, evicted=False, probs=False, cum=True),
        # capped scores and a sliding window behind sinks, 7 query heads a kv head, ragged lengths
        dict(name="decode_cap_window", op="decode", B=16, Hq=28, Hkv=4, page=64, S=20011, ragged=True, cap=50.0,
             alibi=False, window=4096, sink=4, append=True, evicted=False, probs=False, cum=True),
        # a cache after evictions: positions come from its map, the bias falls with the original distance
        dict(name="decode_alibi_evicted", op="decode", B=32, Hq=32, Hkv=32, page=32, S=2171, ragged=True, cap=0.0,
             alibi=True, window=0, sink=0, append=True, evicted=True, probs=True, cum=True),
        # eviction of one short conversation down to 256 slots
        dict(name="evict_short", op="evict", B=1, Hkv=8, page=16, S=1664, budget=256, sink=4, window=64, ragged=False),
        # eviction of the 70B layer's batch to a fifth
        dict(name="evict_70b", op="evict", B=8, Hkv=8, page=16, S=32800, budget=6553, sink=4, window=1024, ragged=False),
        # a few tokens per sequence behind cached prompts (speculated tokens, the tail of a chunked prompt)
        dict(name="prefill_tail", op="prefill", B=4, Hq=16, Hkv=8, page=16, S=1600, new=16, ragged=True, cap=0.0,
             alibi=False, window=0, prefix=0, docs=0),
        # a whole prompt, causal, capped scores
        dict(name="prefill_capped", op="prefill", B=1, Hq=32, Hkv=8, page=64, S=8192, new=8192, ragged=False, cap=50.0,
             alibi=False, window=0, prefix=0, docs=0),
        # packed documents with a bias on distance, 7 query heads a kv head, padding rows that see nothing
        dict(name="prefill_documents", op="prefill", B=2, Hq=28, Hkv=4, page=16, S=7001, new=7001, ragged=True, cap=0.0,
             alibi=True, window=0, prefix=0, docs=900),
        # a chunk behind cached context: a prefix that all of it sees, a sliding window behind that
        dict(name="prefill_prefix", op="prefill", B=3, Hq=32, Hkv=8, page=128, S=6007, new=2500, ragged=True, cap=0.0,
             alibi=False, window=1024, prefix=777, docs=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "evict", "prefill", "prefill"])
    page = rng.choice([16, 32, 64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 5, 7, 8, 12, 16])
    if op == "append":
        B = _log(rng, 1, 64)
        new = 1 if rng.random() < 0.3 else _log(rng, 1, max(2, 200000 // (B * Hkv)))
        return dict(op=op, B=B, Hkv=Hkv, page=page, ctx=rng.randint(0, 1500), new=new, ragged=rng.random() < 0.7)
    if op == "decode":
        B = _log(rng, 1, 32)
        S = _log(rng, 1, max(2, 1600000 // (B * Hkv)))
        windowed = rng.random() < 0.4
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, page=page, S=S, ragged=rng.random() < 0.6,
                    cap=rng.choice([0.0, 0.0, 30.0, 50.0]), alibi=rng.random() < 0.4,
                    window=_log(rng, 1, 5000) if windowed else 0, sink=rng.choice([0, 4, 33]) if windowed else 0,
                    append=rng.random() < 0.6, evicted=rng.random() < 0.3, probs=rng.random() < 0.4,
                    cum=rng.random() < 0.6)
    if op == "evict":
        B = _log(rng, 1, 16)
        S = _log(rng, 20, max(40, 1200000 // (B * Hkv)))
        budget = max(4, int(S * rng.uniform(0.1, 0.9)))
        sink = min(rng.choice([0, 1, 4]), budget)
        return dict(op=op, B=B, Hkv=Hkv, page=page, S=S, budget=budget, sink=sink,
                    window=rng.randint(0, budget - sink), ragged=rng.random() < 0.5)
    B = _log(rng, 1, 4)
    S = _log(rng, 17, 6000 if G * Hkv <= 32 else 2500)
    return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, page=page, S=S, new=min(S, _log(rng, 1, 6000)), ragged=rng.random() < 0.6,
                cap=rng.choice([0.0, 0.0, 30.0, 50.0]), alibi=rng.random() < 0.3,
                window=rng.choice([0, 0, _log(rng, 1, 2000)]), prefix=rng.choice([0, 0, rng.randint(1, S)]),
                docs=rng.choice([0, 0, _log(rng, 3, 2000)]))


def _lengths(n, B, ragged):
    """Fixed ragged lengths of a case (from a third of n to n), so that work() can count them."""
    if not ragged:
        return [n] * B
    return [max(1, n - (n * 2 // 3) * ((b * 7 + 3) % 11) // 11) for b in range(B)]


# ----------------------------------------------------------------------------------------------------------------------
# the number format (plain)
# ----------------------------------------------------------------------------------------------------------------------
def _quantise(x):
    """x [..., 128] -> codes uint8 [..., 64], scales bf16 [..., 4, 2] (scale, minimum).  In 64 bits: the codes and the scale
    are values next to a border."""
    g = x.double().unflatten(-1, (D // GROUP, GROUP))
    z = g.amin(-1) + 0.0
    s = ((g.amax(-1) - z) / 15).bfloat16().double()
    s = torch.where(s < 2.0 ** -100, torch.zeros_like(s), s)
    n = torch.where(s[..., None] > 0, (g - z[..., None]) / s[..., None], torch.zeros_like(g))
    n = n.round().clamp(0, 15).to(torch.uint8).flatten(-2)
    codes = n[..., 0::2] | (n[..., 1::2] << 4)
    return codes, torch.stack([s, z], -1).bfloat16()


def _values(codes, scales):
    """What the cache stands for, fp32 [..., 128]."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).unflatten(-1, (D // GROUP, GROUP)).float()
    s = scales.float()
    return (n * s[..., 0:1] + s[..., 1:2]).flatten(-2)


def _rows(pool, table, n):
    """Logical rows [B, Hkv, n, ...] of a pool [pages, Hkv, page, ...]."""
    page = pool.shape[2]
    t = table[:, :(n + page - 1) // page].clamp_min(0).long()
    return pool[t].transpose(1, 2).flatten(2, 3)[:, :, :n]


# ----------------------------------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------------------------------
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _keys(gen, *shape):
    """Keys have a few channels that are larger than the others, as models' keys do."""
    k = _normal(gen, *shape)
    gain = torch.ones(D, device=DEV)
    gain[torch.randperm(D, generator=gen, device=DEV)[:6]] = 3.0
    return (k * gain).bfloat16()


def _table(gen, B, pages):
    return torch.randperm(B * pages, generator=gen, device=DEV).to(torch.int32).view(B, pages)


def _cache4(gen, B, Hkv, page, n):
    """A 4-bit cache of B x n tokens in permuted pages."""
    pages = (n + page - 1) // page
    k_codes, k_scales = _quantise(_keys(gen, B * pages, Hkv, page, D))
    v_codes, v_scales = _quantise(_normal(gen, B * pages, Hkv, page, D).bfloat16())
    return dict(k_codes=k_codes, k_scales=k_scales, v_codes=v_codes, v_scales=v_scales, table=_table(gen, B, pages))


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _offsets(n):
    return _ints([sum(n[:i]) for i in range(len(n) + 1)])


def _packed(n):
    """(sequence, place in it) of every row of packed sequences."""
    n = torch.tensor(n, device=DEV)
    seq = torch.repeat_interleave(torch.arange(len(n), device=DEV), n)
    first = torch.cumsum(n, 0) - n
    return seq, torch.arange(int(seq.numel()), device=DEV) - first[seq]


def _slopes(Hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return dict(append=_prepare_append, decode=_prepare_decode, evict=_prepare_evict,
                prefill=_prepare_prefill)[case["op"]](case, gen)


def _prepare_append(c, gen):
    B, Hkv, page = c["B"], c["Hkv"], c["page"]
    start, new = _lengths(c["ctx"], B, c["ragged"]) if c["ctx"] else [0] * B, _lengths(c["new"], B, c["ragged"])
    st = dict(c=c, **_cache4(gen, B, Hkv, page, max(a + b for a, b in zip(start, new))))
    total = sum(new)
    st |= dict(start=_ints(start), seq=_ints(start), off=_offsets(new), k=_keys(gen, total, Hkv, D),
               v=_normal(gen, total, Hkv, D).bfloat16(), k_back=torch.zeros(total, Hkv, D, dtype=torch.bfloat16, device=DEV),
               v_back=torch.zeros(total, Hkv, D, dtype=torch.bfloat16, device=DEV))
    st["row_seq"], at = _packed(new)
    st["row_slot"] = at + st["start"].long()[st["row_seq"]]
    if own:
        import attention_guided_kv_gb300 as K
        st["kv"] = K.paged_kv4(st["k_codes"], st["v_codes"], st["k_scales"], st["v_scales"], Hkv)
        st["ws"] = K.workspace(K.kvsel_kv4_append_workspace(st["kv"], B))
    return st


def _prepare_decode(c, gen):
    B, Hq, Hkv, page = c["B"], c["Hq"], c["Hkv"], c["page"]
    S = _lengths(c["S"], B, c["ragged"])                 # live keys, the appended one included
    if not c["append"]:
        live = S
    else:
        live = [s - 1 for s in S]
    cap = max(S)
    st = dict(c=c, S=_ints(S), cap=cap, **_cache4(gen, B, Hkv, page, cap))
    st |= dict(live=_ints(live), seq=_ints(live), q=(_normal(gen, B, Hq, D) * 1.5).bfloat16(),
               out=torch.zeros(B, Hq, D, dtype=torch.bfloat16, device=DEV),
               probs=torch.zeros(B, Hq, cap, device=DEV) if c["probs"] else None,
               cum0=_normal(gen, B, Hkv, cap).square() if c["cum"] else None,
               slopes=_slopes(Hq) if c["alibi"] else None, k_new=None, v_new=None, pos=None, pos0=None, next0=None,
               next=None)
    st["cum"] = st["cum0"].clone() if c["cum"] else None
    if c["append"]:
        st["k_new"], st["v_new"] = _keys(gen, B, Hkv, D), _normal(gen, B, Hkv, D).bfloat16()
    if c["evicted"]:                                     # ascending original positions with gaps
        step = torch.randint(1, 6, (B, Hkv, cap), generator=gen, device=DEV)
        pos = torch.cumsum(step, -1) - 1
        st["pos"] = pos.to(torch.int32)
        st["next0"] = (pos.amax((1, 2)) + 1).to(torch.int32)
        st["next"] = st["next0"].clone()
    if own:
        import attention_guided_kv_gb300 as K
        st["kv"] = K.paged_kv4(st["k_codes"], st["v_codes"], st["k_scales"], st["v_scales"], Hq)
        st["ws"] = K.workspace(K.kvsel_kv4_decode_attn_workspace(st["kv"], B, cap, c["probs"], c["cum"]))
    return st


def _prepare_evict(c, gen):
    B, Hkv, page = c["B"], c["Hkv"], c["page"]
    S = _lengths(c["S"], B, c["ragged"])
    cap = max(S)
    kept = [min(s, c["budget"]) for s in S]
    st = dict(c=c, cap=cap, **_cache4(gen, B, Hkv, page, cap))
    # cumulative scores: a few heavy hitters, many near nothing, ties among them
    cum = torch.exp(2.5 * _normal(gen, B, Hkv, cap))
    cum = torch.where(torch.rand(B, Hkv, cap, generator=gen, device=DEV) < 0.1, (cum * 8).floor() / 8, cum)
    total = sum(kept)
    st |= dict(S=_ints(S), seq=_ints(S), table0=st["table"].clone(), cum0=cum, cum=cum.clone(),
               pos0=torch.arange(cap, dtype=torch.int32, device=DEV).expand(B, Hkv, cap).contiguous(), off=_offsets(kept),
               keep=torch.zeros(B, Hkv, c["budget"], dtype=torch.int32, device=DEV), freed=torch.zeros_like(st["table"]),
               k_back=torch.zeros(total, Hkv, D, dtype=torch.bfloat16, device=DEV),
               v_back=torch.zeros(total, Hkv, D, dtype=torch.bfloat16, device=DEV))
    st["pos"] = st["pos0"].clone()
    st["row_seq"], st["row_slot"] = _packed(kept)
    if own:
        import attention_guided_kv_gb300 as K
        st["kv"] = K.paged_kv4(st["k_codes"], st["v_codes"], st["k_scales"], st["v_scales"], Hkv)
        st["ws"] = K.workspace(K.kvsel_kv4_evict_workspace(st["kv"], B, c["budget"]))
    return st


def _prepare_prefill(c, gen):
    B, Hq, Hkv, page = c["B"], c["Hq"], c["Hkv"], c["page"]
    S = _lengths(c["S"], B, c["ragged"])
    new = [min(a, b) for a, b in zip(_lengths(c["new"], B, c["ragged"]), S)]
    cap, total = max(S), sum(new)
    pages = (cap + page - 1) // page
    st = dict(c=c, cap=cap, n_max=max(new), k_pool=_keys(gen, B * pages, Hkv, page, D),
              v_pool=_normal(gen, B * pages, Hkv, page, D).bfloat16(), table=_table(gen, B, pages))
    st |= dict(S=_ints(S), new=_ints(new), off=_offsets(new), q=(_normal(gen, total, Hq, D) * 1.5).bfloat16(),
               slopes=_slopes(Hq) if c["alibi"] else None, prefix=None, docs=None,
               out=torch.zeros(total, Hq, D, dtype=torch.bfloat16, device=DEV), lse=torch.zeros(total, Hq, device=DEV))
    st["row_seq"], st["row_at"] = _packed(new)
    if c["prefix"]:
        st["prefix"] = _ints([max(0, c["prefix"] - 5 * b) for b in range(B)])
    if c["docs"]:                                        # documents of about `docs` tokens; the last rows are padding
        edge = torch.rand(B, cap, generator=gen, device=DEV) < 1.0 / c["docs"]
        edge[:, 0] = True
        first = torch.where(edge, torch.arange(cap, device=DEV), torch.zeros((), dtype=torch.long, device=DEV))
        first = torch.cummax(first, 1).values
        pos = st["row_at"] + (st["S"] - st["new"]).long()[st["row_seq"]]
        first = first[st["row_seq"], pos]
        pad = pos >= (st["S"].long() - min(3, min(new) - 1))[st["row_seq"]]
        st["docs"] = torch.where(pad, cap, first).to(torch.int32)
    if own:
        import attention_guided_kv_gb300 as K
        st["kv"] = K.paged_kv(st["k_pool"], st["v_pool"], Hq)
        st["ws"] = K.workspace(K.kvsel_prefill_attn_workspace(st["kv"], B, total))
    return st


# ----------------------------------------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------------------------------------
def run(st):
    return dict(append=_run_append, decode=_run_decode, evict=_run_evict, prefill=_run_prefill)[st["c"]["op"]](st)


def _put(st, seq, slot, k, v):
    """Rows k, v [n, Hkv, 128] into slots of sequences."""
    page = st["k_codes"].shape[2]
    at = st["table"][seq, slot // page].long()
    for side, x in (("k", k), ("v", v)):
        codes, scales = _quantise(x)
        st[side + "_codes"][at, :, slot % page] = codes
        st[side + "_scales"][at, :, slot % page] = scales


def _back(st):
    """The values of the rows (row_seq, row_slot), bf16 [n, Hkv, 128]."""
    page = st["k_codes"].shape[2]
    at, r = st["table"][st["row_seq"], st["row_slot"] // page].long(), st["row_slot"] % page
    return [_values(st[s + "_codes"][at, :, r], st[s + "_scales"][at, :, r]).bfloat16() for s in "kv"]


def _run_append(st):
    st["seq"].copy_(st["start"])
    if own:
        import attention_guided_kv_gb300 as K
        K.kvsel_kv4_append(st["kv"], st["table"], st["seq"], st["off"], st["k"], st["v"], st["ws"])
        K.kvsel_kv4_read(st["kv"], st["table"], st["seq"], st["off"], st["k_back"], st["v_back"], st["ws"],
                         start=st["start"])
        return dict(k=st["k_back"], v=st["v_back"], seq=st["seq"])
    _put(st, st["row_seq"], st["row_slot"], st["k"], st["v"])
    st["seq"] += st["off"][1:] - st["off"][:-1]
    k, v = _back(st)
    return dict(k=k, v=v, seq=st["seq"])


def _run_decode(st):
    c = st["c"]
    st["seq"].copy_(st["live"])
    if c["cum"]:
        st["cum"].copy_(st["cum0"])
    if c["evicted"]:
        st["next"].copy_(st["next0"])
    if own:
        import attention_guided_kv_gb300 as K
        K.kvsel_kv4_decode_attn(st["kv"], st["table"], st["seq"], st["q"], st["out"], st["ws"], k_new=st["k_new"],
                                v_new=st["v_new"], pos_map=st["pos"], next_pos=st["next"], softcap=c["cap"],
                                slopes=st["slopes"], window=c["window"], n_sink=c["sink"], probs=st["probs"],
                                h2o_cum=st["cum"], max_len=st["cap"])
        return {k: st[k] for k in ("out", "probs", "cum", "seq", "pos", "next") if st[k] is not None}
    B, Hq, Hkv, cap = c["B"], c["Hq"], c["Hkv"], st["cap"]
    if c["append"]:
        b = torch.arange(B, device=DEV)
        slot = st["live"].long()
        _put(st, b, slot, st["k_new"], st["v_new"])
        if c["evicted"]:
            st["pos"][b, :, slot] = st["next"][:, None]
        if c["cum"]:
            st["cum"][b, :, slot] = 0
        st["seq"] += 1
    S = st["seq"].long()
    k = _values(_rows(st["k_codes"], st["table"], cap), _rows(st["k_scales"], st["table"], cap))
    v = _values(_rows(st["v_codes"], st["table"], cap), _rows(st["v_scales"], st["table"], cap))
    s = torch.matmul(st["q"].float().view(B, Hkv, -1, D), k.transpose(-1, -2)) * D ** -0.5
    if c["cap"]:
        s = c["cap"] * torch.tanh(s / c["cap"])
    slot = torch.arange(cap, device=DEV)
    if c["evicted"]:
        pos = st["pos"].long()
        here = pos.gather(2, (S - 1)[:, None, None].expand(B, Hkv, 1))
        if c["append"]:
            here = st["next"].long()[:, None, None].expand(B, Hkv, 1)
    else:
        pos, here = slot.expand(B, Hkv, cap), (S - 1)[:, None, None].expand(B, Hkv, 1)
    if c["alibi"]:
        s = s - st["slopes"].view(Hkv, -1, 1) * (here - pos).abs()[:, :, None].float()
    seen = (slot < S[:, None, None]).expand(B, Hkv, cap)
    if c["window"]:
        seen = seen & ((here - pos < c["window"]) | (pos < c["sink"]))
    s = torch.where(seen[:, :, None], s, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    st["out"].copy_(torch.matmul(p, torch.where((slot < S[:, None, None])[..., None], v, 0.0)).view(B, Hq, D))
    if c["probs"]:
        live = (slot < S[:, None])[:, None]
        st["probs"].copy_(torch.where(live, p.view(B, Hq, cap), st["probs"]))
    if c["cum"]:
        st["cum"] += p.sum(2)
    if c["evicted"] and c["append"]:
        st["next"] += 1
    return {k: st[k] for k in ("out", "probs", "cum", "seq", "pos", "next") if st[k] is not None}


def _run_evict(st):
    c = st["c"]
    st["seq"].copy_(st["S"])
    st["table"].copy_(st["table0"])
    st["cum"].copy_(st["cum0"])
    st["pos"].copy_(st["pos0"])
    names = ("keep", "freed", "table", "seq", "cum", "pos")
    if own:
        import attention_guided_kv_gb300 as K
        K.kvsel_kv4_evict(st["kv"], st["table"], st["seq"], st["cum"], st["ws"], budget=c["budget"], n_sink=c["sink"],
                          window=c["window"], compact=True, pos_map=st["pos"], keep_out=st["keep"], freed_pages=st["freed"])
        K.kvsel_kv4_read(st["kv"], st["table"], st["seq"], st["off"], st["k_back"], st["v_back"], st["ws"])
        return dict(k=st["k_back"], v=st["v_back"], **{n: st[n] for n in names})
    B, Hkv, page, budget, cap = c["B"], c["Hkv"], c["page"], c["budget"], st["cap"]
    S = st["S"].long()[:, None, None]
    slot = torch.arange(cap, device=DEV).expand(B, Hkv, cap)
    locked = (slot < c["sink"]) | (slot >= S - c["window"])
    rank = torch.where(locked, math.inf, st["cum"])      # scores are finite and not negative
    rank = torch.where(slot < S, rank, -math.inf)
    best = torch.sort(rank, dim=-1, descending=True, stable=True).indices[:, :, :min(budget, cap)]
    keep = torch.sort(best, dim=-1).values
    first = torch.arange(keep.shape[-1], device=DEV)
    full = S > budget
    keep = torch.where(full, keep, first)                # nothing is evicted from a sequence within the budget
    n = torch.minimum(S, torch.tensor(budget, device=DEV))
    st["keep"].fill_(-1)
    st["keep"][:, :, :keep.shape[-1]] = torch.where(first < n, st["pos"].gather(2, keep), -1).to(torch.int32)
    b, h = torch.arange(B, device=DEV)[:, None, None], torch.arange(Hkv, device=DEV)[None, :, None]
    src, dst = torch.where(first < n, keep, first), first.expand_as(keep)
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        pool = st[name]
        rows = pool[st["table"][b, src // page].long(), h, src % page]
        pool[st["table"][b, dst // page].long(), h, dst % page] = rows
    for name in ("cum", "pos"):
        st[name][:, :, :keep.shape[-1]] = st[name].gather(2, src)
    old, now = (S[:, :, 0] + page - 1) // page, (n[:, :, 0] + page - 1) // page
    p = torch.arange(st["table"].shape[1], device=DEV)
    shifted = st["table"].gather(1, (p + now).clamp_max(p.numel() - 1))
    st["freed"].copy_(torch.where(now + p < old, shifted, -1))
    k, v = _back(st)
    st["table"].copy_(torch.where((p >= now) & (p < old), -1, st["table"]))
    st["seq"].copy_(n[:, 0, 0])
    return dict(k=k, v=v, **{n: st[n] for n in names})


def _run_prefill(st):
    c = st["c"]
    if own:
        import attention_guided_kv_gb300 as K
        K.kvsel_prefill_attn(st["kv"], st["table"], st["S"], st["q"], st["off"], st["out"], st["ws"], softcap=c["cap"],
                             slopes=st["slopes"], window=c["window"], prefix=st["prefix"], doc_start=st["docs"],
                             lse=st["lse"])
        return dict(out=st["out"], lse=st["lse"])
    B, Hq, Hkv, cap, n = c["B"], c["Hq"], c["Hkv"], st["cap"], st["n_max"]
    G = Hq // Hkv
    k = _rows(st["k_pool"], st["table"], cap).float()
    v = _rows(st["v_pool"], st["table"], cap).float()
    q = torch.zeros(B, n, Hq, D, device=DEV)
    q[st["row_seq"], st["row_at"]] = st["q"].float()
    q = q.view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(D ** -0.5)
    if c["cap"]:
        s = (s / c["cap"]).tanh_().mul_(c["cap"])
    s = s.view(B, Hkv, G, n, cap)
    i = torch.arange(n, device=DEV)[None, :, None] + (st["S"] - st["new"]).long()[:, None, None]
    j = torch.arange(cap, device=DEV)[None, None, :]
    if c["alibi"]:
        s = s - st["slopes"].view(1, Hkv, G, 1, 1) * (i - j).abs().float()[:, None, None]
    seen = j <= i
    if c["window"]:
        seen = seen & (i - j < c["window"])
    if c["prefix"]:
        seen = seen | (j < st["prefix"].long()[:, None, None])
    if c["docs"]:
        first = torch.zeros(B, n, dtype=torch.long, device=DEV)
        first[st["row_seq"], st["row_at"]] = st["docs"].long()
        seen = seen & (j >= first[:, :, None])
    seen = seen & (j < st["S"].long()[:, None, None])
    s = torch.where(seen[:, None, None], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, G * n, cap), v).view(B, Hkv, G, n, D) / torch.where(l > 0, l, 1.0)
    lse = (torch.log(l) + m)[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)[st["row_seq"], st["row_at"]]
    lse = lse.permute(0, 3, 1, 2).reshape(B, n, Hq)[st["row_seq"], st["row_at"]]
    return dict(out=o.bfloat16(), lse=lse)


# ----------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------------------------------------------------
ROW = 64 + 16      # bytes of one row of 128 values in 4 bits, with its scales and minima


def work(c):
    B, Hkv = c["B"], c["Hkv"]
    if c["op"] == "append":
        rows = 2 * Hkv * sum(_lengths(c["new"], B, c["ragged"]))
        return dict(bytes=rows * (256 + ROW + ROW + 256), flops=rows * D * 6)
    if c["op"] == "decode":
        G = c["Hq"] // Hkv
        S = _lengths(c["S"], B, c["ragged"])
        seen = [min(s, c["window"] + c["sink"]) if c["window"] and not c["evicted"] else s for s in S]
        nbytes = sum(seen) * Hkv * 2 * ROW + 4 * B * c["Hq"] * D
        nbytes += Hkv * (4 * G * c["probs"] * sum(S) + 8 * c["cum"] * sum(seen) + 4 * c["evicted"] * sum(S))
        return dict(bytes=nbytes, flops=sum(seen) * c["Hq"] * D * 4)
    if c["op"] == "evict":
        S = _lengths(c["S"], B, c["ragged"])
        kept = sum(min(s, c["budget"]) for s in S)
        moved = sum(c["budget"] for s in S if s > c["budget"])
        nbytes = sum(S) * Hkv * 4 + moved * Hkv * (4 * ROW + 16 + 4) + kept * Hkv * 2 * (ROW + 256)
        return dict(bytes=nbytes, flops=sum(S) * Hkv)
    G = c["Hq"] // Hkv
    S = _lengths(c["S"], B, c["ragged"])
    new = [min(a, b) for a, b in zip(_lengths(c["new"], B, c["ragged"]), S)]
    pairs = keys = 0
    for b, (s, n) in enumerate(zip(S, new)):
        prefix = max(0, c["prefix"] - 5 * b) if c["prefix"] else 0
        keys += s
        for i in range(s - n, s):
            w = min(i + 1, c["window"] or i + 1, c["docs"] or i + 1)   # a document's mean length counts for it
            pairs += min(s, w + max(0, min(prefix, i + 1 - w) if prefix <= i else prefix - w)) if not c["docs"] else w
    return dict(bytes=keys * Hkv * 512 + sum(new) * c["Hq"] * (512 + 4), flops=4 * D * pairs * c["Hq"])


# ----------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits, one sequence and kv head at a time
# ----------------------------------------------------------------------------------------------------------------------
def _held(x):
    """What the format makes of one row set x [n, 128], from its definition: each group's codes by comparing with all 16 levels'
    borders."""
    g = x.double().reshape(-1, GROUP)
    low, high = g.min(1, keepdim=True).values, g.max(1, keepdim=True).values
    step = ((high - low) / 15).bfloat16().double()
    step[step < 2.0 ** -100] = 0
    border = torch.arange(15, device=x.device, dtype=torch.float64) + 0.5
    gap = (g - low)[..., None]
    over = gap > border * step[..., None]
    tie = (gap == border * step[..., None]) & (step[..., None] > 0)
    odd = torch.arange(15, device=x.device) % 2 == 1     # the border over an odd code goes up, to the even one
    n = (over | (tie & odd)).sum(-1).double()
    return (torch.where(step > 0, n * step, torch.zeros_like(n)) + low).reshape(x.shape)


def _level(codes, scales, b, h, table, n):
    """fp64 values of the first n slots of one sequence and kv head."""
    page = codes.shape[2]
    t = table[b, :(n + page - 1) // page].long()
    c = codes[t, h].reshape(-1, D // 2)[:n]
    s = scales[t, h].reshape(-1, D // GROUP, 2)[:n].double()
    n4 = torch.empty(c.shape[0], D, dtype=torch.float64, device=c.device)
    n4[:, 0::2], n4[:, 1::2] = (c % 16).double(), torch.div(c, 16, rounding_mode="floor").double()
    return n4 * s[..., 0].repeat_interleave(GROUP, 1) + s[..., 1].repeat_interleave(GROUP, 1)


def exact(case, seed):
    c = case
    if c["op"] == "evict":
        return None                                      # it moves values and computes none
    st = prepare(case, seed)
    if c["op"] == "append":
        return dict(k=_held(st["k"].reshape(-1, D)).view_as(st["k"]), v=_held(st["v"].reshape(-1, D)).view_as(st["v"]), seq=None)
    Hq, Hkv = c["Hq"], c["Hkv"]
    G = Hq // Hkv
    if c["op"] == "decode":
        out = torch.zeros(c["B"], Hq, D, dtype=torch.float64, device=DEV)
        probs = torch.zeros(c["B"], Hq, st["cap"], dtype=torch.float64, device=DEV)
        cum = st["cum0"].double() if c["cum"] else None
        for b in range(c["B"]):
            n = int(st["S"][b])
            for h in range(Hkv):
                k = _level(st["k_codes"], st["k_scales"], b, h, st["table"], n)
                v = _level(st["v_codes"], st["v_scales"], b, h, st["table"], n)
                pos = st["pos"][b, h, :n].double() if c["evicted"] else torch.arange(n, dtype=torch.float64, device=DEV)
                here = pos[n - 1].clone()
                if c["append"]:
                    k[n - 1], v[n - 1] = _held(st["k_new"][b, h][None])[0], _held(st["v_new"][b, h][None])[0]
                    if c["evicted"]:
                        here = st["next0"][b].double()
                        pos[n - 1] = here
                    if c["cum"]:
                        cum[b, h, n - 1] = 0
                x = st["q"][b, h * G:(h + 1) * G].double() @ k.T / math.sqrt(D)
                if c["cap"]:
                    x = c["cap"] * torch.tanh(x / c["cap"])
                if c["alibi"]:
                    x -= st["slopes"][h * G:(h + 1) * G].double()[:, None] * (here - pos).abs()
                if c["window"]:
                    x[:, (here - pos >= c["window"]) & (pos >= c["sink"])] = -math.inf
                p = torch.softmax(x, -1)
                out[b, h * G:(h + 1) * G] = p @ v
                probs[b, h * G:(h + 1) * G, :n] = p
                if c["cum"]:
                    cum[b, h, :n] += p.sum(0)
        return {k: v for k, v in dict(out=out, probs=probs if c["probs"] else None, cum=cum).items() if v is not None}
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(st["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    for b in range(c["B"]):
        n, m, a = int(st["S"][b]), int(st["new"][b]), int(st["off"][b])
        t = st["table"][b].long()
        j = torch.arange(n, device=DEV)
        i = (torch.arange(m, device=DEV) + n - m)[:, None]
        seen = j <= i
        if c["window"]:
            seen = seen & (j > i - c["window"])
        if c["prefix"]:
            seen = seen | (j < int(st["prefix"][b]))
        if c["docs"]:
            seen = seen & (j >= st["docs"][a:a + m, None])
        for h in range(Hq):
            k = st["k_pool"][t, h // G].reshape(-1, D)[:n].double()
            v = st["v_pool"][t, h // G].reshape(-1, D)[:n].double()
            x = st["q"][a:a + m, h].double() @ k.T / math.sqrt(D)
            if c["cap"]:
                x = c["cap"] * torch.tanh(x / c["cap"])
            if c["alibi"]:
                x -= st["slopes"][h].double() * (i - j).abs()
            x.masked_fill_(~seen, -math.inf)
            lse[a:a + m, h] = torch.logsumexp(x, -1)
            out[a:a + m, h] = torch.nan_to_num(torch.softmax(x, -1), nan=0.0) @ v
    return dict(out=out, lse=lse)
