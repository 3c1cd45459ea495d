"""Cases for the operators around the NVFP4 product in a serving step: the paged
4-bit key/value cache (append, attention, the weight each slot got, eviction)
and the choice of the next token.

A sequence s of length n = kv_lens[s] has nq = q_starts[s + 1] - q_starts[s]
new tokens, the last nq of its slots.  A cache page holds 64 slots; the record
of one (page, kv head) is 72 D bytes:

  0     K codes   [64 slots][D / 2]            low nibble = even dim
  32 D  V codes   [8 blocks][D][4 bytes]       nibble i = slot 8 block + i
  64 D  K scales  [4 a][4 r][4 b][2 h][2 t][D / 64 j]
                  slot = 32 h + 8 a + 4 t + r, 16-dim group = b D / 64 + j
  68 D  V scales  [8 blocks][D / 16 groups][8 slots]
"""
import math
import random

import torch

own = False

PAGE = 64
K_SCALE, V_SCALE = 2.0 ** -6, 2.0 ** -7      # static tensor scales of the cache
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
STEPS = 2.0 ** 30                            # a token's weight is held in steps of 2^-30 of the top one's


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one conversation, one new token: the latency of a short cache
        dict(name="attend_one", op="attend", seqs=1, new=1, new_to=1, kv=777, kv_to=777, mix=1,
             heads=32, kv_heads=8, dim=128, window=0, cap=0.0),
        # a serving batch of one-token steps, from a cache of a few slots to one of 131,071
        dict(name="attend_batch", op="attend", seqs=32, new=1, new_to=1, kv=3, kv_to=131071, mix=2,
             heads=32, kv_heads=8, dim=128, window=0, cap=0.0),
        # a verify round of five drafted tokens in a layer with a window and capped scores, wide heads
        dict(name="attend_verify", op="attend", seqs=16, new=5, new_to=5, kv=200, kv_to=9001, mix=3,
             heads=16, kv_heads=8, dim=256, window=1500, cap=50.0),
        # ragged prompt chunks over a cache that already holds their beginnings
        dict(name="attend_prompt", op="attend", seqs=4, new=700, new_to=4099, kv=4100, kv_to=8192, mix=4,
             heads=32, kv_heads=8, dim=128, window=0, cap=0.0),
        # the new token of each conversation goes into the cache
        dict(name="append_step", op="append", seqs=48, new=1, new_to=1, kv=10, kv_to=8000, mix=5, kv_heads=8, dim=128),
        # whole prompts go into the cache
        dict(name="append_prompts", op="append", seqs=7, new=33, new_to=8191, kv=8192, kv_to=9000, mix=6,
             kv_heads=8, dim=128),
        # the weights of one step, kept up for later eviction
        dict(name="weigh_step", op="weigh", seqs=16, new=1, new_to=1, kv=100, kv_to=16383, mix=7,
             heads=32, kv_heads=8, dim=128, window=0, cap=0.0),
        # the weights that a prompt's last 32 tokens give
        dict(name="weigh_prompt", op="weigh", seqs=4, new=32, new_to=32, kv=9001, kv_to=32768, mix=8,
             heads=32, kv_heads=8, dim=128, window=0, cap=0.0),
        # one short conversation is cut to 512 slots
        dict(name="evict_one", op="evict", seqs=1, kv=1501, kv_to=1501, mix=9, kv_heads=8, dim=128, keep=512, sink=4, recent=64),
        # a batch of long ones is cut to 4000
        dict(name="evict_batch", op="evict", seqs=8, kv=3000, kv_to=65000, mix=10, kv_heads=8, dim=128, keep=4000, sink=4, recent=500),
        # one conversation's next token, from the output head's logits
        dict(name="sample_one", op="sample", rows=1, vocab=151552, type="float32", mix=11),
        # a large batch's next tokens, each row with parameters of its own
        dict(name="sample_batch", op="sample", rows=192, vocab=151552, type="float32", mix=12),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("attend", "attend", "attend", "append", "weigh", "evict", "sample"))
    mix = rng.randrange(1 << 30)
    if op == "sample":
        return dict(op=op, rows=_log(rng, 1, 192), vocab=_log(rng, 1000, 151552), type=rng.choice(("float32", "bfloat16")), mix=mix)
    dim, kv_heads = rng.choice((64, 128, 128, 256)), rng.choice((1, 2, 4, 8))
    heads = kv_heads * rng.choice((1, 2, 3, 4, 5, 8))
    kind = rng.choice(("step", "step", "verify", "prompt"))
    new = {"step": 1, "verify": rng.randint(2, 32), "prompt": _log(rng, 33, 2048)}[kind]
    seqs = _log(rng, 1, 4 if kind == "prompt" else 48)
    most = max(2 * new, min(131072, 400000 // seqs // (4 if kind == "prompt" else 1)))
    kv_to = _log(rng, max(new, 16), most)
    kv = rng.randint(max(new, 1), kv_to)
    case = dict(op=op, seqs=seqs, kv=kv, kv_to=kv_to, mix=mix, kv_heads=kv_heads, dim=dim)
    if op == "evict":
        keep = rng.randint(8, max(9, min(4096, kv_to)))
        return dict(case, keep=keep, sink=rng.randint(0, 4), recent=rng.randint(0, keep // 2))
    case.update(new=rng.randint(1, new), new_to=new)
    if op == "append":
        return case
    return dict(case, heads=heads, window=rng.choice((0, 0, rng.randint(1, 4096))), cap=rng.choice((0.0, 0.0, 30.0)))


def _lens(case):
    """The lengths of a case's sequences and their numbers of new tokens; the first and the last are the range's ends."""
    rng = random.Random(case["mix"])
    kv = [_log(rng, case["kv"], case["kv_to"]) for _ in range(case["seqs"])]
    kv[0], kv[-1] = case["kv"], case["kv_to"]
    if case["op"] == "evict":
        return kv, [min(case["keep"], n) for n in kv]
    new = [min(n, rng.randint(case["new"], case["new_to"])) for n in kv]
    new[-1] = case["new_to"]
    return kv, new


def _pairs(case):
    """(query, slot) pairs that see each other, and the slots that any query sees, over all sequences."""
    pairs = slots = 0
    w = case["window"] or (1 << 40)
    for n, nq in zip(*_lens(case)):
        first = n - nq + 1                   # slots the first query sees without a window, one more for each next
        a = max(0, min(nq, w - first))       # queries whose whole past is inside the window
        pairs += a * first + a * (a - 1) // 2 + (nq - a) * w if w < (1 << 40) else nq * first + nq * (nq - 1) // 2
        slots += min(n, w + nq - 1)
    return pairs, slots


def work(case):
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (4 if case["type"] == "float32" else 2) + case["rows"] * 28, "flops": 4 * n}
    d, hk = case["dim"], case["kv_heads"]
    row = d * 9 // 16                        # bytes of one K or V row of one head
    kv, new = _lens(case)
    if case["op"] == "append":               # rows in (bf16), rows stored, and read back as values
        t = sum(new) * hk * 2
        return {"bytes": t * (2 * d + 2 * row + 2 * d), "flops": t * d * 4}
    if case["op"] == "evict":                # weights, kept rows read and written, kept weights and slots, and values
        kept = sum(new) * hk
        return {"bytes": sum(kv) * hk * 4 + kept * (2 * row * 3 + 2 * d * 2 + 8), "flops": sum(kv) * hk * 4}
    pairs, slots = _pairs(case)
    q = sum(new) * case["heads"]
    if case["op"] == "weigh":
        return {"bytes": slots * hk * row + sum(kv) * hk * 8 + q * (2 * d + 4), "flops": 2 * d * pairs * case["heads"]}
    return {"bytes": slots * hk * 2 * row + q * (4 * d + 4), "flops": 4 * d * pairs * case["heads"]}


# ---------------------------------------------------------------- inputs

def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _e4m3_up(u):
    return u.clamp(max=448.0).to(torch.float8_e4m3fn)


def _codes(x, t):
    """e2m1 codes and e4m3 scales (as bytes) of x [..., D] at the tensor scale t."""
    g = x.float().unflatten(-1, (-1, 16))
    s = _e4m3_up(g.abs().amax(-1) / 6.0 / t)
    big = (s.float() * t).unsqueeze(-1)
    v = torch.where(big > 0, g / torch.where(big > 0, big, torch.ones_like(big)), torch.zeros_like(g))
    a = v.abs()
    m = (a > 0.25).to(torch.uint8)
    for at, on in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        m += (a >= at) if on else (a > at)
    return (m | ((v < 0) & (m > 0)).to(torch.uint8) << 3).flatten(-2), s.view(torch.uint8)


def _pages(k, v):
    """Cache pages [..., 72 D] of K and V rows [..., 64, D]."""
    d = k.shape[-1]
    kc, ks = _codes(k, K_SCALE)
    vc, vs = _codes(v, V_SCALE)
    kb = kc[..., 0::2] | kc[..., 1::2] << 4
    vt = vc.unflatten(-2, (8, 8)).transpose(-1, -2)                       # [..., block, D, slot]
    vb = vt[..., 0::2] | vt[..., 1::2] << 4
    ks = ks.unflatten(-2, (2, 4, 2, 4)).unflatten(-1, (4, d // 64))       # h a t r b j
    ks = ks.movedim((-5, -3, -2, -6, -4, -1), (-6, -5, -4, -3, -2, -1))   # a r b h t j
    vs = vs.unflatten(-2, (8, 8)).transpose(-1, -2)
    return torch.cat([kb.flatten(-2), vb.flatten(-3), ks.flatten(-6), vs.flatten(-3)], -1)


def _cache(gen, pages, kv_heads, dim):
    """Filled pages: normal rows, K with a factor of its own for each channel, as trained keys have."""
    dev = gen.device
    data = torch.empty(pages, kv_heads, 72 * dim, dtype=torch.uint8, device=dev)
    spread = torch.exp(0.5 * torch.randn(kv_heads, 1, dim, generator=gen, device=dev))
    step = max(1, (1 << 27) // (kv_heads * PAGE * dim))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        k = torch.randn(n, kv_heads, PAGE, dim, generator=gen, device=dev) * spread
        v = torch.randn(n, kv_heads, PAGE, dim, generator=gen, device=dev)
        data[p:p + n] = _pages(k.bfloat16(), v.bfloat16())
    return data


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(seed)
    st = dict(case)
    if case["op"] == "sample":
        b, n = case["rows"], case["vocab"]
        # a few likely tokens over a broad tail, as a head's logits are
        x = torch.randn(b, n, generator=gen, device=dev) * 2.0
        at = torch.randint(0, n, (b, 40), generator=gen, device=dev)
        x.scatter_add_(1, at, 8.0 + 3.0 * torch.randn(b, 40, generator=gen, device=dev))
        st["logits"] = x.to(getattr(torch, case["type"]))
        rng = random.Random(case["mix"])
        row = [rng.choice(((0.7, 50, 0.95, 0.0), (1.0, 0, 0.9, 0.0), (0.9, 0, 1.0, 0.05), (1.0, 0, 1.0, 0.0),
                           (0.0, 0, 1.0, 0.0), (1.3, 1000, 0.8, 0.01), (0.6, 20, 0.95, 0.0))) for _ in range(b)]
        row[0] = (0.7, 50, 0.95, 0.0)
        for i, (name, kind) in enumerate((("temperature", torch.float32), ("top_k", torch.int32), ("top_p", torch.float32), ("min_p", torch.float32))):
            st[name] = torch.tensor([r[i] for r in row], dtype=kind, device=dev)
        st["u"] = torch.rand(b, generator=gen, device=dev)
        return st
    kv, new = _lens(case)
    s, hk, d = case["seqs"], case["kv_heads"], case["dim"]
    need = [-(-n // PAGE) for n in kv]
    spare = -(-case["keep"] // PAGE) * s if case["op"] == "evict" else 0
    total = sum(need) + spare
    order = torch.randperm(total, generator=gen, device=dev).int().tolist()
    table = torch.zeros(s, max(need), dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = torch.tensor(order[at:at + n])
        at += n
    st["table"] = table.to(dev)
    st["data"] = _cache(gen, total, hk, d)
    st["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    st["max_kv"] = max(kv)
    if case["op"] == "evict":
        st["dst_table"] = torch.tensor(order[at:], dtype=torch.int32).view(s, -1).to(dev)
        # accumulated softmax weights: many small ones, a few large ones, and ties at zero
        x = torch.rand(s, hk, max(kv), generator=gen, device=dev)
        st["weights"] = torch.where(x < 0.2, torch.zeros_like(x), 1e-3 * x ** 8 / (1.0001 - x))
        new = [case["keep"]] * s
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    st["q_starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    st["total"], st["max_q"] = starts[-1], max(new)
    if case["op"] == "append":
        kv_in = torch.randn(starts[-1], 2 * hk, d, generator=gen, device=dev).bfloat16()
        st["k"], st["v"] = kv_in[:, :hk], kv_in[:, hk:]              # views of one projection's output
    if case["op"] in ("attend", "weigh"):
        h = case["heads"]
        qkv = torch.randn(starts[-1], (h + 2 * hk) * d, generator=gen, device=dev).bfloat16()
        st["q"] = qkv[:, :h * d].view(starts[-1], h, d)              # a view of one projection's output
    if case["op"] == "weigh":
        st["lse"] = _plain_attend(st)[1]
        st["prior"] = torch.rand(s, hk, max(kv), generator=gen, device=dev)
    if own:
        import verify_nvfp4_w4a16_amd as nv
        st["cache"] = nv.KvCache(st["data"], hk, d, K_SCALE, V_SCALE)
    return st


# ---------------------------------------------------------------- plain forms

def _nibbles(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _values(c):
    sign_and_size = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=c.device)
    return sign_and_size[c.int()]


def _decoded(rec, d):
    """K and V of records [..., 72 D] in 32 bits: [..., 64, D] each."""
    kc, vc, ks, vs = rec.split([32 * d, 32 * d, 4 * d, 4 * d], -1)
    k = _values(_nibbles(kc.unflatten(-1, (PAGE, d // 2))))
    ks = ks.contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (4, 4, 4, 2, 2, d // 64))
    ks = ks.movedim((-6, -5, -4, -3, -2, -1), (-5, -3, -2, -6, -4, -1)).flatten(-2).flatten(-5, -2)
    k = (k.unflatten(-1, (-1, 16)) * (ks * K_SCALE).unsqueeze(-1)).flatten(-2)
    v = _values(_nibbles(vc.unflatten(-1, (8, d, 4)))).transpose(-1, -2)  # [..., block, slot, D]
    vs = vs.contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (8, d // 16, 8)).transpose(-1, -2)
    v = (v.unflatten(-1, (-1, 16)) * (vs * V_SCALE).unsqueeze(-1)).flatten(-2).flatten(-3, -2)
    return k, v


def _rows(st, table):
    """K and V of whole tables in 32 bits: [S, heads, pages 64, D] each."""
    return tuple(x.flatten(2, 3) for x in _decoded(st["data"][table.long()].transpose(1, 2), st["dim"]))


def _scores(st, k):
    """Scores of padded queries [S, KH, G max_q, slots] with -inf where a slot is not seen, and where each padded query is among the packed ones."""
    s, hk, d, mq = st["seqs"], st["kv_heads"], st["dim"], st["max_q"]
    g = st["heads"] // hk
    lens, starts = st["kv_lens"].long(), st["q_starts"].long()
    new = starts[1:] - starts[:-1]
    i = torch.arange(mq, device=k.device)
    there = i < new[:, None]                                              # [S, mq]
    at = (starts[:-1, None] + i).clamp(max=max(0, st["total"] - 1))
    q = st["q"].float()[at].view(s, mq, hk, g, d).permute(0, 2, 3, 1, 4).reshape(s, hk, g * mq, d)
    z = torch.matmul(q, k.transpose(-1, -2)) * d ** -0.5
    if st["cap"]:
        z = st["cap"] * torch.tanh(z / st["cap"])
    place = (lens - new)[:, None] + i                                     # the slot of each query
    j = torch.arange(k.shape[2], device=k.device)
    seen = (j <= place[..., None]) & (j < lens[:, None, None]) & there[..., None]
    if st["window"]:
        seen &= j > place[..., None] - st["window"]
    z = z.view(s, hk, g, mq, -1).masked_fill_(~seen[:, None, None], float("-inf"))
    return z, at, there


def _plain_attend(st):
    k, v = _rows(st, st["table"])
    z, at, there = _scores(st, k)
    s, hk, g, mq, n = z.shape
    top = z.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e.view(s, hk, g * mq, n), v).view(s, hk, g, mq, -1) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (torch.log(total) + top).squeeze(-1)
    pick = torch.nonzero(there.reshape(-1)).squeeze(-1)
    out = out.permute(0, 3, 1, 2, 4).reshape(s * mq, hk * g, -1)[pick]
    lse = lse.permute(0, 3, 1, 2).reshape(s * mq, hk * g)[pick]
    return out.bfloat16(), lse


def _plain_weigh(st):
    k, _ = _rows(st, st["table"])
    z, at, there = _scores(st, k)
    lse = st["lse"][at].unflatten(-1, (st["kv_heads"], -1)).permute(0, 2, 3, 1)[..., None]
    p = torch.exp(z - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)).sum((2, 3))[..., :st["max_kv"]]
    here = torch.arange(st["max_kv"], device=p.device) < st["kv_lens"][:, None, None]
    return torch.where(here, st["prior"] + p, torch.zeros_like(p))


def _plain_append(st):
    """The new rows' stored values: the pages they lie in are taken out, filled and put back."""
    starts = st["q_starts"].long()
    t = torch.arange(st["total"], device=starts.device)
    s = torch.searchsorted(starts[1:], t, right=True)
    slot = st["kv_lens"].long()[s] - starts[s + 1] + t
    page, at, d = st["table"].long()[s, slot // PAGE], slot % PAGE, st["dim"]
    kc, ks = _codes(st["k"], K_SCALE)
    vc, vs = _codes(st["v"], V_SCALE)
    data = st["data"]
    pages, inverse = torch.unique(page, return_inverse=True)
    rec = data[pages]
    rec[..., :32 * d].unflatten(-1, (PAGE, d // 2))[inverse, :, at] = kc[..., 0::2] | kc[..., 1::2] << 4
    vt = _nibbles(rec[..., 32 * d:64 * d].unflatten(-1, (8, d, 4)))       # [pages, H, block, D, slot]
    vt[inverse, :, at // 8, :, at % 8] = vc
    rec[..., 32 * d:64 * d] = (vt[..., 0::2] | vt[..., 1::2] << 4).flatten(-3)
    scales = rec[..., 64 * d:68 * d].unflatten(-1, (4, 4, 4, 2, 2, d // 64))
    scales[inverse, :, at // 8 % 4, at % 4, :, at // 32, at // 4 % 2] = ks.unflatten(-1, (4, d // 64))
    rec[..., 68 * d:].unflatten(-1, (8, d // 16, 8))[inverse, :, at // 8, :, at % 8] = vs
    data[pages] = rec
    return tuple(x[inverse, :, at].bfloat16() for x in _decoded(rec, d))


def _plain_evict(st):
    lens, keep, sink, recent = st["kv_lens"].long(), st["keep"], st["sink"], st["recent"]
    w, d = st["weights"], st["dim"]
    s, hk, m = w.shape
    j = torch.arange(m, device=w.device)
    n = lens[:, None, None]
    rank = torch.where((j < sink) | (j >= n - recent), torch.full_like(w, float("inf")), torch.nan_to_num(w, nan=float("-inf")))
    rank = torch.where(j < n, rank, torch.full_like(w, float("-inf")))
    order = torch.sort(torch.where(j < n, rank, torch.full_like(w, float("-inf"))), dim=-1, descending=True, stable=True).indices
    if m < keep:
        order = torch.nn.functional.pad(order, (0, keep - m), value=m)
    order = order[..., :keep]
    kept = torch.sort(torch.where(order < n, order, torch.full_like(order, 1 << 40)), dim=-1).values
    there = kept < (1 << 40)
    at = torch.where(there, kept, torch.zeros_like(kept))
    kept_weights = torch.where(there, w.gather(-1, at), torch.zeros_like(w[..., :1]))
    new_lens = torch.minimum(lens, torch.full_like(lens, keep)).int()
    k, v = _rows(st, st["table"])
    rows = []
    for x in (k, v):
        x = x.gather(2, at[..., None].expand(-1, -1, -1, d))              # [S, H, keep, D], the kept rows from the first slot on
        slot = new_lens.long()[:, None] - keep + torch.arange(keep, device=w.device)
        x = x.gather(2, slot.clamp(min=0)[:, None, :, None].expand(-1, hk, -1, d))
        rows.append(torch.where((slot >= 0)[:, None, :, None], x, torch.zeros((), device=x.device)).transpose(1, 2).reshape(s * keep, hk, d).bfloat16())
    return torch.where(there, kept, torch.full_like(kept, -1)).int(), kept_weights, new_lens, rows[0], rows[1]


def _plain_sample(st):
    x = torch.nan_to_num(st["logits"].float(), nan=float("-inf"), posinf=float("inf"), neginf=float("-inf"))
    top = x.amax(-1, keepdim=True)
    t = st["temperature"][:, None]
    inverse = torch.where(t > 0, 1.0 / torch.where(t > 0, t, torch.ones_like(t)), torch.zeros_like(t))
    w = torch.where(t > 0, torch.floor(torch.exp((x - top) * inverse) * STEPS), torch.zeros_like(x))
    w = torch.where(x == top, torch.full_like(w, STEPS), w).long()
    w = torch.where(torch.isinf(top) & (top < 0), torch.zeros_like(w), w)
    down, order = torch.sort(w, dim=-1, descending=True, stable=True)
    place = torch.arange(x.shape[1], device=x.device)
    k = torch.where(t > 0, st["top_k"].long()[:, None], torch.ones_like(t, dtype=torch.int64))
    down = torch.where((k > 0) & (place >= k), torch.zeros_like(down), down)
    total = torch.cumsum(down, -1)
    before = total - down
    limit = st["top_p"].double()[:, None] * total[:, -1:].double()
    low = st["min_p"].double()[:, None] * STEPS
    stays = ((before.double() < limit) & (down.double() >= low)) | (place == 0)
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(stays, down, torch.zeros_like(down)))
    running = torch.cumsum(kept, -1)
    mass = running[:, -1:]
    target = torch.minimum((st["u"].double()[:, None] * mass.double()).long(), mass - 1)
    token = (running <= target).sum(-1)
    token = torch.where(mass[:, 0] > 0, token, torch.full_like(token, -1))
    picked = kept.gather(1, token.clamp(min=0)[:, None])
    return token.int(), torch.log((picked.double() / mass.clamp(min=1).double()).float()).squeeze(1)


def run(state):
    st, op = state, state["op"]
    if not own:
        return {"attend": _plain_attend, "append": _plain_append, "weigh": _plain_weigh, "evict": _plain_evict, "sample": _plain_sample}[op](st)
    import verify_nvfp4_w4a16_amd as nv
    if op == "sample":
        return nv.sample(st["logits"], st["u"], st["temperature"], st["top_k"], st["top_p"], st["min_p"])
    if op == "attend":
        return nv.kv_attention(st["q"], st["cache"], st["table"], st["kv_lens"], st["q_starts"], st["max_q"], st["max_kv"],
                               window=st["window"], softcap=st["cap"])
    if op == "weigh":
        return nv.kv_weights(st["q"], st["lse"], st["cache"], st["table"], st["kv_lens"], st["q_starts"], st["max_q"], st["max_kv"],
                             window=st["window"], softcap=st["cap"], prior=st["prior"])
    if op == "append":
        nv.kv_append(st["cache"], st["k"], st["v"], st["table"], st["kv_lens"], st["q_starts"])
        return nv.kv_read(st["cache"], st["table"], st["kv_lens"], st["q_starts"], st["total"])
    kept, kept_weights, new_lens = nv.kv_evict(st["weights"], st["cache"], st["table"], st["kv_lens"], st["dst_table"], st["keep"],
                                               sink=st["sink"], recent=st["recent"])
    k, v = nv.kv_read(st["cache"], st["dst_table"], new_lens, st["q_starts"], st["total"])
    return kept, kept_weights, new_lens, k, v


# ---------------------------------------------------------------- the definition in 64 bits

def _slots64(st, i, table=None):
    """K and V rows of one sequence, one page after the other by the layout's own words: [heads, slots, D] in 64 bits."""
    d = st["dim"]
    hk = st["kv_heads"]
    grid = torch.tensor([(-1.0 if c & 8 else 1.0) * ((c & 1) * 0.5 if c & 6 == 0 else (1 + 0.5 * (c & 1)) * 2.0 ** ((c >> 1 & 3) - 1)) for c in range(16)],
                        dtype=torch.float64, device=st["data"].device)
    e4m3 = torch.tensor([(b & 7) * 2.0 ** -9 if b >> 3 == 0 else (8 + (b & 7)) * 2.0 ** ((b >> 3) - 10) for b in range(128)],
                        dtype=torch.float64, device=st["data"].device)
    n = int(st["kv_lens"][i])
    pages = (st["table"] if table is None else table)[i, :-(-n // PAGE)].long()
    rec = st["data"][pages]                                               # [P, H, 72 D]
    slot = torch.arange(PAGE, device=rec.device)[:, None]
    dim = torch.arange(d, device=rec.device)[None]
    group = dim // 16
    per = d // 64
    k_at = slot * (d // 2) + dim // 2
    v_at = 32 * d + (slot // 8 * d + dim) * 4 + slot % 8 // 2
    h, a, t, r = slot // 32, slot // 8 % 4, slot // 4 % 2, slot % 4
    ks_at = 64 * d + ((((a * 4 + r) * 4 + group // per) * 2 + h) * 2 + t) * per + group % per
    vs_at = 68 * d + (slot // 8 * (d // 16) + group) * 8 + slot % 8
    k = grid[(rec[..., k_at] >> 4 * (dim % 2).to(torch.uint8) & 15).long()] * e4m3[rec[..., ks_at].long()] * K_SCALE
    v = grid[(rec[..., v_at] >> 4 * (slot % 2).to(torch.uint8) & 15).long()] * e4m3[rec[..., vs_at].long()] * V_SCALE
    return (x.transpose(0, 1).reshape(hk, -1, d)[:, :n] for x in (k, v))


def _probabilities64(st, i, k, lse=None):
    """Sequence i's (start, end, scores [H, G, nq, n] in 64 bits)."""
    a, b = int(st["q_starts"][i]), int(st["q_starts"][i + 1])
    n, hk = k.shape[1], st["kv_heads"]
    q = st["q"][a:b].double().view(b - a, hk, -1, st["dim"]).permute(1, 2, 0, 3)
    z = (q.reshape(hk, -1, st["dim"]) @ k.mT.contiguous()).view(hk, -1, b - a, n) / math.sqrt(st["dim"])
    if st["cap"]:
        z = torch.tanh(z / st["cap"]) * st["cap"]
    place = n - (b - a) + torch.arange(b - a, device=k.device)[:, None]
    j = torch.arange(n, device=k.device)[None]
    hidden = j > place
    if st["window"]:
        hidden = hidden | (place - j >= st["window"])
    return a, b, z.masked_fill(hidden, -math.inf)


def _quantised64(x, t):
    g = x.double().unflatten(-1, (-1, 16))
    u = (g.abs().amax(-1) / 6 / t).clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(u.clamp(min=2.0 ** -6))) - 3)
    s = (torch.round(u / step) * step).clamp(max=448.0) * t
    v = torch.where(s[..., None] > 0, g / s[..., None].clamp(min=1e-300), torch.zeros_like(g)).clamp(-6, 6)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=1.0))) - 1)
    return (torch.round(v / step) * step * s[..., None]).flatten(-2)


def _evicted64(st):
    """The kept weights and rows of every sequence and head; slots and lengths are whole numbers."""
    keep, hk, d = st["keep"], st["kv_heads"], st["dim"]
    weights = torch.zeros(st["seqs"], hk, keep, dtype=torch.float64, device=st["data"].device)
    k_out, v_out = (torch.zeros(st["seqs"], keep, hk, d, dtype=torch.float64, device=weights.device) for _ in range(2))
    for i in range(st["seqs"]):
        k, v = _slots64(st, i)
        n = k.shape[1]
        for h in range(hk):
            w = st["weights"][i, h, :n].double()
            slots = torch.arange(n, device=w.device)
            if n > keep:
                middle = slots[st["sink"]:n - st["recent"]]
                best = torch.sort(w[middle], descending=True, stable=True).indices[:keep - st["sink"] - st["recent"]]
                slots = torch.cat([slots[:st["sink"]], middle[best].sort().values, slots[n - st["recent"]:]])
            weights[i, h, :len(slots)] = w[slots]
            k_out[i, keep - len(slots):, h], v_out[i, keep - len(slots):, h] = k[h, slots], v[h, slots]
    return None, weights, None, k_out.flatten(0, 1), v_out.flatten(0, 1)


def exact(case, seed):
    if case["op"] in ("attend", "weigh") and _pairs(case)[0] * case["heads"] * case["dim"] > 2e11:
        return None
    global own
    was, own = own, False
    st = prepare(case, seed)
    own = was
    op, dev = case["op"], st["u"].device if "u" in st else st["data"].device
    if op == "append":
        return tuple(_quantised64(st[x], t) for x, t in (("k", K_SCALE), ("v", V_SCALE)))
    if op == "attend":
        outs, lses = [], []
        for i in range(case["seqs"]):
            k, v = _slots64(st, i)
            a, b, z = _probabilities64(st, i, k)
            lse = torch.logsumexp(z, -1)
            p = torch.exp(z - lse[..., None])
            o = (p.reshape(p.shape[0], -1, p.shape[-1]) @ v).view(*p.shape[:3], -1)
            outs.append(o.permute(2, 0, 1, 3).reshape(b - a, case["heads"], -1))
            lses.append(lse.permute(2, 0, 1).reshape(b - a, case["heads"]))
        return torch.cat(outs), torch.cat(lses)
    if op == "weigh":
        out = torch.zeros(st["prior"].shape, dtype=torch.float64, device=dev)
        for i in range(case["seqs"]):
            k, _ = _slots64(st, i)
            a, b, z = _probabilities64(st, i, k)
            lse = st["lse"][a:b].double().view(b - a, case["kv_heads"], -1).permute(1, 2, 0)
            out[i, :, :k.shape[1]] = st["prior"][i, :, :k.shape[1]].double() + torch.exp(z - lse[..., None]).sum((1, 2))
        return out
    if op == "evict":
        return _evicted64(st)
    logits = st["logits"].double()
    logprob = torch.zeros(case["rows"], dtype=torch.float64, device=dev)
    for b in range(case["rows"]):
        x, t = logits[b], float(st["temperature"][b])
        if t > 0:
            w = torch.floor(torch.exp((x - x.max()) * float(1.0 / st["temperature"][b])) * STEPS)
            rank = torch.sort(w, descending=True, stable=True)
            many = int(st["top_k"][b]) or w.numel()
            mass = rank.values[:many]
            mass = mass[(torch.cumsum(mass, 0) - mass < float(st["top_p"][b]) * mass.sum()) & (mass >= float(st["min_p"][b]) * STEPS)]
            kept = torch.zeros_like(w)
            kept[rank.indices[:mass.numel()]] = mass
            token = int((torch.cumsum(kept, 0) <= math.floor(float(st["u"][b]) * float(mass.sum()))).sum())
            logprob[b] = torch.log(kept[token] / mass.sum())
    return None, logprob
