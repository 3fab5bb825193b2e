"""The paged-cache operators as measured workloads: what they are given, one
pass of each, the bytes and operations a pass cannot do without, and its
results in 64 bits.

Three operators keep a key/value cache in pages beside the statistics its
eviction goes by:

- append: new tokens' keys (rotated by their positions) and values go to the
  pages, their accumulated weight starts at zero;
- attend: attention of one new token per sequence over its cached tokens,
  which may add every token's softmax weight, summed over the query heads of
  its KV head, to the token's accumulated weight;
- evict: of the cached tokens of a (sequence, KV head) the `keep` heaviest
  stay (the first `sinks` positions and the last `recent` ones always), the
  kept tokens behind slot `keep` move into the slots the others leave.

`step` is a run of the three, as a bounded cache decodes one token.

The cache: k_pages, v_pages [n_pages, Hkv, page, d]; page_table [B, max_pages]
int32; weight fp32 and token_pos int32 [B, Hkv, max_pages * page].
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------- cases
def _case(name, op, dtype, batch, hq, hkv, d, theta, page, lo, hi, weights=False, new_lo=1, new_hi=1, keep=0,
          sinks=0, recent=0):
    c = dict(op=op, dtype=dtype, batch=batch, hq=hq, hkv=hkv, d=d, theta=theta, page=page, lo=lo, hi=hi,
             weights=weights, new_lo=new_lo, new_hi=new_hi, keep=keep, sinks=sinks, recent=recent)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step's new tokens for a batch of 32 sequences of very different lengths
        _case("append_decode_b32", "append", "bf16", 32, 32, 8, 128, 1e6, 16, 0, 2047),
        # the prompts of eight requests, from a few tokens to 4096, written in one call
        _case("append_prompts_b8", "append", "bf16", 8, 32, 8, 128, 5e5, 64, 0, 512, new_lo=3, new_hi=4096),
        # a small fp32 model's chunk of a prompt, odd lengths, behind what is cached
        _case("append_f32_d64", "append", "f32", 4, 4, 2, 64, 1e4, 32, 1, 77, new_lo=1, new_hi=201),
        # the smallest call: one sequence of a small fp32 model, latency alone
        _case("attend_f32_ctx1k", "attend", "f32", 1, 4, 2, 64, 1e4, 64, 1023, 1023, weights=True),
        # one long sequence: few rows, the cache's length has to be split
        _case("attend_ctx32k", "attend", "bf16", 1, 32, 8, 128, 5e5, 64, 32768, 32768),
        # batch 8 of 16K, seven query heads to a KV head, small pages, weights kept for eviction
        _case("attend_b8_ctx16k_g7", "attend", "bf16", 8, 28, 4, 128, 1e6, 16, 16384, 16384, weights=True),
        # serving: 32 sequences of 4K to 32K
        _case("attend_b32_ragged", "attend", "bf16", 32, 32, 8, 128, 1e6, 32, 4096, 32768),
        # four sequences of 128K with their weights
        _case("attend_b4_ctx128k", "attend", "bf16", 4, 32, 8, 128, 5e5, 64, 131072, 131072, weights=True),
        # many short sequences, an empty one among them, one query head to a KV head
        _case("attend_b64_short_d64", "attend", "bf16", 64, 8, 8, 64, 1e4, 16, 0, 1000),
        # a 32K prompt cut down to 4096 tokens after it was read
        _case("evict_ctx32k_to_4k", "evict", "bf16", 1, 32, 8, 128, 5e5, 64, 32768, 32768, keep=4096, sinks=4,
              recent=256),
        # 32 sequences around their bound: most are under it or a few tokens over
        _case("evict_b32_around_2k", "evict", "bf16", 32, 32, 8, 128, 1e6, 16, 1900, 2080, keep=2048, sinks=4,
              recent=128),
        # one token of eight full bounded caches: append, attend with weights, evict
        _case("step_b8_keep4k", "step", "bf16", 8, 32, 8, 128, 5e5, 16, 4096, 4096, weights=True, keep=4096,
              sinks=4, recent=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "evict", "step"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    theta = rng.choice([1e4, 5e5, 1e6])
    batch = _log(rng, 1, 48)
    row = hkv * d * (2 if dtype == "bf16" else 4) * 2  # K and V of a token
    if op == "append":
        hi = _log(rng, 1, 1500)
        new = max(1, min(_log(rng, 1, 4096), 4096 * 8 * 256 // (batch * row) * 4))
        return _case("", op, dtype, batch, hq, hkv, d, theta, page, rng.randint(0, hi), hi,
                     new_lo=rng.randint(1, new), new_hi=new)
    most = max(64, int(1.5e9) // (batch * row))
    if op == "attend":
        hi = _log(rng, 1, min(65536, most))
        return _case("", op, dtype, batch, hq, hkv, d, theta, page, rng.randint(0, hi), hi,
                     weights=rng.random() < 0.5)
    hi = _log(rng, 40, min(32768 if op == "evict" else 8192, most))
    if op == "step":
        recent = rng.randint(1, max(1, hi // 4))
        return _case("", op, dtype, batch, hq, hkv, d, theta, page, hi, hi, weights=True, keep=hi,
                     sinks=rng.randint(0, 8), recent=recent)
    keep = _log(rng, 20, hi)
    return _case("", op, dtype, batch, hq, hkv, d, theta, page, rng.randint(hi // 2, hi), hi, keep=keep,
                 sinks=rng.randint(0, 8), recent=rng.randint(0, keep // 2))


def _spread(lo, hi, n):
    """n whole numbers spread over lo..hi, both ends among them where n > 1 (the same for every seed)."""
    if n == 1:
        return [hi]
    out = [lo + int(round((hi - lo) * ((i * 0.6180339887498949) % 1.0))) for i in range(n)]
    out[n // 2] = hi
    return out


def _lens(c):
    return _spread(c["lo"], c["hi"], c["batch"])


def _news(c):
    return _spread(c["new_lo"], c["new_hi"], c["batch"])[::-1]


# -------------------------------------------------------------------- inputs
def prepare(case, seed):
    c = dict(case)
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]
    B, hkv, d, page, op = c["batch"], c["hkv"], c["d"], c["page"], c["op"]
    lens = _lens(c)
    news = _news(c) if op == "append" else [1] * B
    grow = op in ("append", "step")
    cap = max(n + (m if grow else 0) for n, m in zip(lens, news))
    max_pages = max(1, -(-cap // page))
    n_pages = B * max_pages + 3
    T = max_pages * page

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    def rows(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=dt)

    s = dict(case=c)
    # the pages of a sequence lie anywhere in the pool
    s["page_table"] = torch.randperm(n_pages, generator=g, device=dev)[:B * max_pages].to(torch.int32).view(
        B, max_pages).contiguous()
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["k_pages"] = rows(n_pages, hkv, page, d)
    s["v_pages"] = rows(n_pages, hkv, page, d)
    # weights that earlier steps have added up: few tokens carry much
    s["weight"] = torch.exp(1.5 * normal(B, hkv, T))
    # positions in the order they came; an eviction has taken out some before
    gaps = torch.randint(1, 4, (B, hkv, T), generator=g, device=dev, dtype=torch.int32)
    s["token_pos"] = (torch.cumsum(gaps, dim=-1, dtype=torch.int32) - 1).contiguous()
    last = torch.tensor([max(n - 1, 0) for n in lens], device=dev).view(B, 1, 1).expand(B, hkv, 1)
    newest = torch.gather(s["token_pos"], 2, last).amax(dim=(1, 2))
    # the query logits spread by about 2: some tokens matter, none alone
    s["q"] = (2.0 * normal(B, c["hq"], d)).to(dt)
    n_tok = sum(news)
    s["k_new"] = rows(n_tok, hkv, d)
    s["v_new"] = rows(n_tok, hkv, d)
    s["pos"] = (newest + (1 if op == "append" else 0)).to(torch.int32).contiguous()
    s["cu_new"] = torch.tensor([sum(news[:i]) for i in range(B + 1)], dtype=torch.int32, device=dev)
    s["lens_after"] = (s["seq_lens"] + torch.tensor(news if grow else [0] * B, dtype=torch.int32, device=dev))
    s["new_lens"] = torch.zeros(B, dtype=torch.int32, device=dev)
    s["out"] = torch.zeros(B, c["hq"], d, dtype=torch.float32, device=dev)
    s["weight_out"] = torch.zeros_like(s["weight"])
    s["token_pos_out"] = torch.zeros_like(s["token_pos"])
    # room for what the calls keep on the device meanwhile: partial results, scores, lists
    s["workspace"] = torch.empty(64 * 1024 * 1024 + 4 * B * (c["hq"] + 2 * hkv) * T, dtype=torch.uint8, device=dev)
    s["one_each"] = op == "step" or all(m == 1 for m in news)
    s["n_pages"], s["max_pages"] = n_pages, max_pages
    return s


# ------------------------------------------------------------- plain operators
def _angles(pos, c):
    """cos and sin of pos * theta^(-2i/d), in 64 bits: far positions turn many times."""
    i = torch.arange(c["d"] // 2, device=pos.device, dtype=torch.float64)
    a = pos.double().unsqueeze(-1) * torch.pow(torch.tensor(c["theta"], dtype=torch.float64, device=pos.device),
                                               -2.0 * i / c["d"])
    return torch.cos(a).float(), torch.sin(a).float()


def _rotate(x, pos, c):
    """x [N, H, d] in 32 bits, its pairs (2i, 2i+1) turned by pos [N]."""
    cos, sin = _angles(pos, c)
    cos, sin = cos.unsqueeze(1), sin.unsqueeze(1)
    a, b = x[..., 0::2].float(), x[..., 1::2].float()
    return torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)


def _plain_append(s, c):
    n_tok = s["k_new"].shape[0]
    j = torch.arange(n_tok, device=s["pos"].device)
    seq = torch.searchsorted(s["cu_new"], j.to(torch.int32), right=True) - 1
    nth = j - s["cu_new"][seq]
    slot = s["seq_lens"][seq] + nth
    pos = s["pos"][seq] + nth
    page = s["page_table"][seq, slot // c["page"]].long()
    at = slot % c["page"]
    s["k_pages"][page, :, at] = _rotate(s["k_new"], pos, c).to(s["k_pages"].dtype)
    s["v_pages"][page, :, at] = s["v_new"]
    s["weight"][seq, :, slot] = 0.0
    s["token_pos"][seq, :, slot] = pos.to(torch.int32).unsqueeze(1)


def _gathered(pages, s, c):
    """[B, Hkv, T, d] in 32 bits."""
    x = pages[s["page_table"].long()]  # [B, max_pages, Hkv, page, d]
    return x.permute(0, 2, 1, 3, 4).reshape(c["batch"], c["hkv"], -1, c["d"]).float()


def _plain_attend(s, c, lens, weights):
    B, hkv, G, d = c["batch"], c["hkv"], c["hq"] // c["hkv"], c["d"]
    q = _rotate(s["q"], s["pos"], c).view(B, hkv, G, d)
    k = _gathered(s["k_pages"], s, c)
    score = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)  # [B, Hkv, G, T]
    del k
    valid = (torch.arange(score.shape[-1], device=q.device) < lens.unsqueeze(-1)).view(B, 1, 1, -1)
    score = score.masked_fill(~valid, -math.inf)
    most = score.amax(dim=-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isfinite(most), most, torch.zeros_like(most)))
    p = p / p.sum(dim=-1, keepdim=True).clamp_min(1e-30)  # a sequence with no token: zeros
    # what the page rows behind a sequence's end hold counts for nothing, whatever it is
    v = _gathered(s["v_pages"], s, c).masked_fill(~valid.view(B, 1, -1, 1), 0.0)
    s["out"].copy_(torch.matmul(p, v).reshape(B, c["hq"], d))
    if weights:
        s["weight"].add_(p.sum(dim=2))


def _plain_evict(s, c, lens, weight_out, token_pos_out):
    B, hkv, keep = c["batch"], c["hkv"], c["keep"]
    w, tp = s["weight"].clone(), s["token_pos"].clone()
    T = w.shape[-1]
    slots = torch.arange(T, device=w.device)
    n = lens.view(B, 1, 1)
    valid = (slots < n).expand(B, hkv, T)
    held = (tp < c["sinks"]) | (tp > s["pos"].view(B, 1, 1) - c["recent"])
    key = torch.where(held, torch.full_like(w, math.inf), w)
    key = torch.where(valid, key, torch.full_like(w, -math.inf))
    order = torch.argsort(key, dim=-1, descending=True, stable=True)  # equal weights: the lower slot first
    rank = torch.empty_like(order).scatter_(2, order, slots.expand(B, hkv, T))
    kept = valid & (rank < keep)
    hole = torch.nonzero(valid & ~kept & (slots < keep))
    mover = torch.nonzero(kept & (slots >= keep))  # as many as holes in every (sequence, head), in the same order
    b, h, dst, src = hole[:, 0], hole[:, 1], hole[:, 2], mover[:, 2]
    pd, ps = s["page_table"][b, dst // c["page"]].long(), s["page_table"][b, src // c["page"]].long()
    od, os_ = dst % c["page"], src % c["page"]
    s["k_pages"][pd, h, od] = s["k_pages"][ps, h, os_]
    s["v_pages"][pd, h, od] = s["v_pages"][ps, h, os_]
    w[b, h, dst], tp[b, h, dst] = w[b, h, src], tp[b, h, src]
    left = slots < torch.clamp(n, max=keep)
    weight_out.copy_(torch.where(left, w, weight_out))
    token_pos_out.copy_(torch.where(left, tp, token_pos_out))
    s["new_lens"].copy_(torch.clamp(lens, max=keep))


# ----------------------------------------------------------- the framework's
def _dims(s, c):
    from kv_cache_token_tip_gb300 import FASA_BF16, FASA_F32, FasaPagedDims
    if "dims" not in s:
        s["dims"] = FasaPagedDims(c["batch"], c["hq"], c["hkv"], c["d"], c["page"], s["n_pages"], s["max_pages"],
                                  FASA_BF16 if c["dtype"] == "bf16" else FASA_F32, c["theta"])
    return s["dims"]


def _own_append(s, c):
    from kv_cache_token_tip_gb300 import fasa_paged_append
    fasa_paged_append(s["k_new"], s["v_new"], s["pos"], s["k_pages"], s["v_pages"], s["page_table"], s["seq_lens"],
                      cu_new=None if s["one_each"] else s["cu_new"], weight=s["weight"], token_pos=s["token_pos"],
                      dims=_dims(s, c))


def _own_attend(s, c, lens, weights):
    from kv_cache_token_tip_gb300 import fasa_paged_attention
    fasa_paged_attention(s["q"], s["pos"], s["k_pages"], s["v_pages"], s["page_table"], lens, s["out"],
                         weight=s["weight"] if weights else None, workspace=s["workspace"], dims=_dims(s, c))


def _own_evict(s, c, lens, weight_out, token_pos_out):
    from kv_cache_token_tip_gb300 import fasa_paged_evict
    fasa_paged_evict(s["weight"], s["token_pos"], s["pos"], s["k_pages"], s["v_pages"], s["page_table"], lens,
                     c["keep"], s["new_lens"], sinks=c["sinks"], recent=c["recent"], weight_out=weight_out,
                     token_pos_out=token_pos_out, workspace=s["workspace"], dims=_dims(s, c))


# ---------------------------------------------------------------------- a pass
def run(state):
    s, c = state, state["case"]
    append, attend, evict = (_own_append, _own_attend, _own_evict) if own else (_plain_append, _plain_attend,
                                                                                 _plain_evict)
    cache = ("k_pages", "v_pages", "weight", "token_pos")
    if c["op"] == "append":
        append(s, c)
        return {k: s[k] for k in cache}
    if c["op"] == "attend":
        attend(s, c, s["seq_lens"], c["weights"])
        return {k: s[k] for k in (("out", "weight") if c["weights"] else ("out",))}
    if c["op"] == "evict":
        # into other statistics than it reads, so that a pass leaves the next one as much to do
        evict(s, c, s["seq_lens"], s["weight_out"], s["token_pos_out"])
        return {k: s[k] for k in ("k_pages", "v_pages", "weight_out", "token_pos_out", "new_lens")}
    # a decode step of a full cache: the next position, its token, its attention, one token out
    s["pos"].add_(1)
    append(s, c)
    attend(s, c, s["lens_after"], True)
    evict(s, c, s["lens_after"], s["weight"], s["token_pos"])
    return {k: s[k] for k in ("out", "new_lens") + cache}


# ------------------------------------------------------------------------ work
def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    B, hq, hkv, d, op = c["batch"], c["hq"], c["hkv"], c["d"], c["op"]
    lens = _lens(c)
    tables = 4 * sum(-(-n // c["page"]) for n in lens) + 12 * B
    by = fl = 0.0

    def append(n_tok):
        # the new rows in and out, a zero weight and the position of each
        return n_tok * hkv * (4 * d * es + 8), 3.0 * n_tok * hkv * d

    def attend(lens):
        n = sum(lens)
        return (n * hkv * (2 * d * es + (8 if c["weights"] else 0)) + B * hq * d * (es + 4),
                4.0 * n * hq * d + 4.0 * n * hq)

    def evict(lens, apart):
        over = [n for n in lens if n > c["keep"]]
        # a kept token lies behind slot `keep` as often as not, but for the share that does
        moved = sum(c["keep"] * (1.0 - c["keep"] / n) for n in over)
        by = hkv * (8.0 * sum(lens if apart else over) + moved * (4 * d * es + (0 if apart else 16)))
        return by + (8.0 * hkv * sum(min(n, c["keep"]) for n in lens) if apart else 0), 2.0 * hkv * sum(lens)

    if op == "append":
        by, fl = append(sum(_news(c)))
    elif op == "attend":
        by, fl = attend(lens)
    elif op == "evict":
        by, fl = evict(lens, True)
    else:
        after = [n + 1 for n in lens]
        for x, y in (append(B), attend(after), evict(after, False)):
            by, fl = by + x, fl + y
    return {"bytes": by + tables, "flops": fl}


# ----------------------------------------------------------------------- exact
def _turned(x, pos, theta):
    """Rows x [..., d] in 64 bits as complex numbers times exp(i pos theta_j)."""
    d = x.shape[-1]
    j = torch.arange(0, d, 2, dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.ones_like(j), float(pos) * torch.exp(-j / d * math.log(theta)))
    z = torch.view_as_complex(x.double().reshape(*x.shape[:-1], d // 2, 2).contiguous()) * turn
    return torch.view_as_real(z).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op, page, hkv, G = c["op"], c["page"], c["hkv"], c["hq"] // c["hkv"]
    lens, news = _lens(c), (_news(c) if c["op"] == "append" else [1] * c["batch"])
    table = s["page_table"].tolist()
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    w, tp = s["weight"].double(), s["token_pos"].clone()
    pos = [p + (1 if op == "step" else 0) for p in s["pos"].tolist()]
    stored = DTYPES[c["dtype"]]
    if op in ("append", "step"):
        at = 0
        for b, (n, m) in enumerate(zip(lens, news)):
            steps = torch.arange(m, device=kp.device)
            slot = n + steps
            pg = s["page_table"][b].long()[slot // page]
            j = torch.arange(0, c["d"], 2, dtype=torch.float64, device=kp.device)
            a = (pos[b] + steps.double()).view(-1, 1, 1) * torch.exp(-j / c["d"] * math.log(c["theta"]))
            z = torch.view_as_complex(s["k_new"][at:at + m].double().view(m, hkv, -1, 2))
            new = torch.view_as_real(z * torch.polar(torch.ones_like(a), a)).reshape(m, hkv, c["d"])
            if op == "step":  # what the attention then reads is what the cache can hold
                new = new.to(stored).double()
            kp[pg, :, slot % page], vp[pg, :, slot % page] = new, s["v_new"][at:at + m].double()
            w[b, :, n:n + m] = 0.0
            tp[b, :, n:n + m] = (pos[b] + steps).to(torch.int32)
            at += m
    if op == "append":
        return {"k_pages": kp, "v_pages": vp, "weight": w, "token_pos": None}
    if op == "step":
        lens = [n + 1 for n in lens]
    out = torch.zeros(c["batch"], c["hq"], c["d"], dtype=torch.float64, device=kp.device)
    if op in ("attend", "step"):
        for b, n in enumerate(lens):
            if n == 0:
                continue
            used = s["page_table"][b, :-(-n // page)].long()
            for h in range(hkv):
                k = kp[used, h].reshape(-1, c["d"])[:n]
                q = _turned(s["q"][b, h * G:(h + 1) * G], pos[b], c["theta"])
                p = torch.softmax((k @ q.T) / math.sqrt(c["d"]), dim=0)  # [n, G]
                out[b, h * G:(h + 1) * G] = p.T @ vp[used, h].reshape(-1, c["d"])[:n]
                w[b, h, :n] += p.sum(dim=1)
    if op == "attend":
        return {"out": out, "weight": w} if c["weights"] else {"out": out}
    wo, to = (w, tp) if op == "step" else (s["weight_out"].double(), s["token_pos_out"])
    for b, n in enumerate(lens):
        m = min(n, c["keep"])
        for h in range(hkv):
            wb, tb = w[b, h, :n].clone(), tp[b, h, :n].clone()
            if n > m:
                must = (tb < c["sinks"]) | (tb > pos[b] - c["recent"])
                rank = torch.where(must, torch.full_like(wb, math.inf), wb)
                least = torch.topk(rank, c["keep"]).values[-1]
                sure, tie = rank > least, rank == least
                sure[torch.nonzero(tie).flatten()[:c["keep"] - int(sure.sum())]] = True
                dst = torch.nonzero(~sure[:m]).flatten()
                src = torch.nonzero(sure[m:]).flatten() + m
                row = torch.tensor(table[b], device=kp.device)
                for x in (kp, vp):
                    x[row[dst // page], h, dst % page] = x[row[src // page], h, src % page]
                wb[dst], tb[dst] = wb[src], tb[src]
            wo[b, h, :m], to[b, h, :m] = wb[:m], tb[:m]
    if op == "step":
        return {"out": out, "new_lens": None, "k_pages": kp, "v_pages": vp, "weight": wo, "token_pos": None}
    return {"k_pages": kp, "v_pages": vp, "weight_out": wo, "token_pos_out": None, "new_lens": None}
