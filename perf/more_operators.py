"""What a server does around the paged cache, as measured workloads: what the
operators are given, one pass of each, the bytes and operations a pass cannot do
without, and its results in 64 bits.

- assign: from the lengths that sequences have and want, the pages that they give
  back and take, their new lengths, where each sequence's new tokens begin, and
  for every new token its sequence, slot, page and position;
- rope: the new tokens' queries and keys are turned by their positions (pairs
  interleaved or in halves, the whole head or its first part, plain or scaled
  frequencies); the queries go to a buffer, keys and values to the pages, the
  tokens' statistics begin;
- chunk: attention of each sequence's new tokens over its cached ones, themselves
  among them, every token over the slots up to its own; it may add every slot's
  softmax weights, summed over the queries, to its accumulated weight.

`serve` is a run of the three, as a server takes one step of prompts' chunks and
single tokens together.

The cache: k_pages, v_pages [n_pages, Hkv, page, d]; page_table [B, max_pages]
int32; weight fp32 and token_pos int32 [B, Hkv, max_pages * page]; the free pages
are the first free_count entries of free_pages [n_pages], taken from the end.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------- cases
def _case(name, op, dtype, batch, hq, hkv, d, page, lo, hi, new_lo, new_hi, prompts=0, finish=0, spare=8, pad=0,
          weights=False, layout="half", rotary=0, theta=5e5, scaling="plain", factor=1.0):
    """lo..hi: tokens that a sequence has; new_lo..new_hi: those that it gets.  In assign and serve the first
    `prompts` sequences get new_lo..new_hi, the last `finish` of them end, and the others get one.  spare: free pages
    beyond those that are needed (below 0: too few).  pad: rows of the map and the inputs behind the last token."""
    c = dict(op=op, dtype=dtype, batch=batch, hq=hq, hkv=hkv, d=d, page=page, lo=lo, hi=hi, new_lo=new_lo,
             new_hi=new_hi, prompts=prompts, finish=finish, spare=spare, pad=pad, weights=weights, layout=layout,
             rotary=rotary or d, theta=theta, scaling=scaling, factor=factor)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a decode step of 64 sequences: one in sixteen needs a page
        _case("assign_decode_b64", "assign", "bf16", 64, 32, 8, 128, 16, 100, 4000, 1, 1),
        # a busy server: of 256 sequences 24 bring prompts of up to 4096 tokens, 20 have ended
        _case("assign_mixed_b256", "assign", "bf16", 256, 32, 8, 128, 16, 1, 16384, 33, 4096, prompts=24, finish=20,
              pad=500),
        # one token each of 32 sequences, frequencies scaled by their wavelengths
        _case("rope_decode_b32", "rope", "bf16", 32, 32, 8, 128, 16, 100, 2047, 1, 1, scaling="wavelength", factor=8.0),
        # eight prompts, 16.5K tokens, frequencies scaled along a ramp
        _case("rope_prompts_b8", "rope", "bf16", 8, 28, 4, 128, 64, 0, 512, 3, 4096, theta=1e6, scaling="ramp",
              factor=4.0),
        # a small fp32 model, half of the head turned, pairs side by side, odd lengths
        _case("rope_f32_d64_part", "rope", "f32", 4, 4, 2, 64, 32, 1, 77, 1, 201, layout="interleaved", rotary=32,
              theta=1e4, scaling="linear", factor=2.0),
        # the smallest call: a small fp32 model's chunk behind a few hundred tokens, with weights
        _case("chunk_f32_ctx1k", "chunk", "f32", 1, 4, 2, 64, 64, 959, 959, 65, 65, weights=True),
        # drafted tokens of 16 sequences are checked: few rows over long caches
        _case("chunk_drafts_b16", "chunk", "bf16", 16, 32, 8, 128, 16, 4096, 16384, 3, 8),
        # eight prompts of very different lengths, seven query heads to a KV head
        _case("chunk_prompts_b8_g7", "chunk", "bf16", 8, 28, 4, 128, 64, 0, 512, 37, 4096),
        # a chunk of a long prompt behind what is cached
        _case("chunk_2k_ctx32k", "chunk", "bf16", 1, 32, 8, 128, 64, 30720, 30720, 2048, 2048),
        # a whole prompt with the weights that its eviction will go by
        _case("chunk_16k_weights", "chunk", "bf16", 1, 32, 8, 128, 64, 0, 0, 16384, 16384, weights=True),
        # fp32 prompts of heads of 128 dims
        _case("chunk_f32_prompts_b2", "chunk", "f32", 2, 8, 2, 128, 32, 100, 300, 1000, 1501),
        # one step of a server: 30 sequences decode, two prompts go on by up to 1024 tokens
        _case("serve_b32", "serve", "bf16", 32, 32, 8, 128, 16, 500, 8000, 700, 1024, prompts=2, pad=37, weights=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["assign", "rope", "chunk", "chunk", "chunk", "serve"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    kw = dict(layout=rng.choice(["half", "half", "interleaved"]), rotary=rng.choice([d, d, d // 2, d // 4]),
              theta=rng.choice([1e4, 5e5, 1e6]), scaling=rng.choice(["plain", "linear", "wavelength", "ramp"]),
              factor=rng.choice([2.0, 4.0, 8.0]), pad=rng.choice([0, 0, 1, 77]))
    es = 2 if dtype == "bf16" else 4
    if op == "assign":
        batch = _log(rng, 1, 400)
        hi = _log(rng, 1, 16384)
        prompts = rng.randint(0, batch)
        new = _log(rng, 1, max(1, min(8192, 100000 // max(1, prompts))))
        return _case("", op, dtype, batch, g * hkv, hkv, d, page, rng.randint(0, hi), hi, rng.randint(1, new), new,
                     prompts=prompts, finish=rng.randint(0, batch - prompts),
                     spare=rng.choice([0, 5, 1000, -1, -20]), **kw)
    batch = _log(rng, 1, 40)
    if op == "rope":
        new = _log(rng, 1, max(1, min(4096, 16384 // batch)))
        hi = _log(rng, 1, 1500)
        return _case("", op, dtype, batch, g * hkv, hkv, d, page, rng.randint(0, hi), hi, rng.randint(1, new), new,
                     **kw)
    # operations of the attention, and the cache's bytes
    flops, room = (6e11 if dtype == "bf16" else 2e10), int(1.5e9) // (batch * hkv * d * 2 * es)
    hi = _log(rng, 1, max(1, min(32768, room)))
    prompts = batch if op == "chunk" else rng.randint(0, min(3, batch))
    new = max(1, min(4096, room, int(flops / (4.0 * d * hkv * g * max(1, prompts) * (hi + 1)))))
    new = _log(rng, 1, new)
    while prompts * 4.0 * d * hkv * g * new * (hi + new / 2) > flops and new > 1:
        new = new * 3 // 4
    return _case("", op, dtype, batch, g * hkv, hkv, d, page, rng.randint(0, hi), hi, rng.randint(1, new), new,
                 prompts=prompts if op == "serve" else 0, weights=rng.random() < 0.5, **kw)


def _spread(lo, hi, n):
    """n whole numbers spread over lo..hi, both ends among them where n > 1 (the same for every seed)."""
    if n < 2:
        return [hi] * n
    out = [lo + int(round((hi - lo) * ((i * 0.6180339887498949) % 1.0))) for i in range(n)]
    out[n // 2] = hi
    return out


def _lens(c):
    """Tokens that each sequence has and wants, all of which it gets where the pages last."""
    have = _spread(c["lo"], c["hi"], c["batch"])
    if c["op"] in ("rope", "chunk"):
        return have, [h + m for h, m in zip(have, _spread(c["new_lo"], c["new_hi"], c["batch"])[::-1])]
    new = _spread(c["new_lo"], c["new_hi"], c["prompts"]) + [1] * (c["batch"] - c["prompts"])
    want = [h + m for h, m in zip(have, new)]
    if c["finish"]:
        want[-c["finish"]:] = [0] * c["finish"]
    return have, want


# -------------------------------------------------------------------- inputs
def prepare(case, seed):
    c = dict(case)
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]
    B, hq, hkv, d, page, op = c["batch"], c["hq"], c["hkv"], c["d"], c["page"], c["op"]
    have, want = _lens(c)
    grown = [max(0, w - h) for h, w in zip(have, want)]
    n_tok = sum(grown) + c["pad"]
    max_pages = max(1, -(-max(max(h, w) for h, w in zip(have, want)) // page))
    T = max_pages * page
    held = [-(-h // page) for h in have]
    takes = [max(0, -(-w // page) - p) for w, p in zip(want, held)]
    gives = [max(0, p - -(-w // page)) for w, p in zip(want, held)]
    free = max(0, sum(takes) - sum(gives) + c["spare"])
    n_pages = sum(held) + max(free, sum(takes)) + 3

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    s = dict(case=c, n_pages=n_pages, max_pages=max_pages, max_tokens=n_tok)
    # the pages of a sequence lie anywhere in the pool
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    e = torch.arange(max_pages, device=dev).view(1, -1)
    held_t, at = ints(held).view(-1, 1), torch.cumsum(ints([0] + held[:-1]), 0).view(-1, 1)
    table = torch.where(e < held_t, order[(at + e).clamp(max=n_pages - 1)], torch.full_like(order[:1], -1))
    s["page_table"] = table.to(torch.int32).contiguous()
    s["free_pages"] = torch.full((n_pages,), -1, dtype=torch.int32, device=dev)
    s["free_pages"][:free] = order[sum(held):sum(held) + free]
    if op in ("rope", "chunk"):  # the new tokens' pages are there
        more = torch.tensor([0] + takes[:-1], device=dev).cumsum(0).view(-1, 1)
        fresh = (e >= held_t) & (e < held_t + ints(takes).view(-1, 1))
        place = (sum(held) + more + e - held_t).clamp(min=0, max=n_pages - 1)
        s["page_table"] = torch.where(fresh, order[place], s["page_table"]).contiguous()
    s["free_count"], s["free_count_out"] = ints([free]), ints([0])
    s["have"], s["want"], s["lens"] = ints(have), ints(want), ints([0] * B)
    # positions go on behind what evictions have taken out
    s["pos"] = (s["have"] + torch.randint(0, 1000, (B,), generator=g, device=dev, dtype=torch.int32)).contiguous()
    cu = [0]
    for m in grown:
        cu.append(cu[-1] + m)
    s["cu_new"] = ints(cu)
    s["token_map"] = torch.full((n_tok, 4), -1, dtype=torch.int32, device=dev)
    if op == "assign":
        s["cu_new"].zero_()
        return _handles(s)
    if op == "rope":
        x = torch.arange(n_tok, device=dev)
        b = (torch.searchsorted(s["cu_new"], x.to(torch.int32), right=True) - 1).clamp(max=B - 1)
        nth = x - s["cu_new"][b]
        slot = s["have"][b] + nth
        m = torch.stack((b, slot, s["page_table"][b, (slot // page).clamp(max=max_pages - 1)].long(),
                         s["pos"][b] + nth), dim=1)
        s["token_map"] = torch.where((x < cu[-1]).view(-1, 1), m, torch.full_like(m, -1)).to(torch.int32).contiguous()
    s["k_pages"] = torch.randn((n_pages, hkv, page, d), generator=g, device=dev, dtype=dt)
    s["v_pages"] = torch.randn((n_pages, hkv, page, d), generator=g, device=dev, dtype=dt)
    if op in ("rope", "serve"):
        # what one projection gave: queries, keys and values of a token side by side; the logits spread by about 2
        qkv = normal(n_tok, hq + 2 * hkv, d)
        qkv[:, :hq] *= 2.0
        qkv = qkv.to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_rot"] = torch.zeros((n_tok, hq, d), dtype=dt, device=dev)
    else:
        s["q_rot"] = (2.0 * normal(n_tok, hq, d)).to(dt)
    s["out"] = torch.zeros((n_tok, hq, d), dtype=dt, device=dev)
    s["weight"] = torch.exp(1.5 * normal(B, hkv, T))
    s["token_pos"] = torch.arange(T, dtype=torch.int32, device=dev).expand(B, hkv, T).contiguous()
    return _handles(s)


def _handles(s):
    """What a user's program keeps beside its tensors: the shapes, and a workspace."""
    c = s["case"]
    if own:
        import kv_cache_token_tip_gb300 as F
        s["dims"] = F.FasaPagedDims(c["batch"], c["hq"], c["hkv"], c["d"], c["page"], s["n_pages"], s["max_pages"],
                                    F.FASA_BF16 if c["dtype"] == "bf16" else F.FASA_F32, c["theta"])
        s["rope"] = F.FasaRope(
            layout=F.FASA_ROPE_HALF if c["layout"] == "half" else F.FASA_ROPE_INTERLEAVED, rotary_dim=c["rotary"],
            scaling={"plain": F.FASA_ROPE_PLAIN, "linear": F.FASA_ROPE_LINEAR, "wavelength": F.FASA_ROPE_WAVELENGTH,
                     "ramp": F.FASA_ROPE_RAMP}[c["scaling"]],
            rope_theta=c["theta"], factor=c["factor"], **_SCALES.get(c["scaling"], {}))
        if c["op"] in ("chunk", "serve"):
            s["workspace"] = torch.empty(F.fasa_paged_chunk_workspace_size(s["dims"], s["max_tokens"], c["weights"]),
                                         dtype=torch.uint8, device="cuda")
    return s


# The scaled frequencies' bounds: turns that a frequency makes within the `original` positions, and what a turned pair
# is multiplied by.
_SCALES = {"wavelength": dict(low=1.0, high=4.0, original=8192.0, magnitude=1.0),
           "ramp": dict(low=1.0, high=32.0, original=4096.0, magnitude=1.1386294361119891)}


# ------------------------------------------------------------- plain operators
def _plain_assign(s, c):
    page, dev = c["page"], s["have"].device
    have, want = s["have"].long(), s["want"].long()
    ph, pw = (have + page - 1) // page, (want + page - 1) // page
    gives, takes = (ph - pw).clamp(min=0), (pw - ph).clamp(min=0)
    grows = (want - have).clamp(min=0)
    n = s["free_count"].long()
    avail = n + gives.sum()
    # in order, as long as the pages and the map's rows last
    fits = (torch.cumsum(takes, 0) <= avail) & (torch.cumsum(grows, 0) <= s["max_tokens"])
    fits = fits | (grows == 0)
    lens = torch.where(fits, want, have)
    takes, grows = torch.where(fits, takes, 0), torch.where(fits, grows, 0)
    e = torch.arange(s["max_pages"], device=dev).view(1, -1)
    table = s["page_table"]
    back = (e >= pw.view(-1, 1)) & (e < ph.view(-1, 1))
    pushed = table[back]  # sequence by sequence, entry by entry
    s["free_pages"].index_copy_(0, n + torch.arange(pushed.shape[0], device=dev), pushed)
    nth = (torch.cumsum(takes, 0) - takes).view(-1, 1) + e - ph.view(-1, 1)
    fresh = (e >= ph.view(-1, 1)) & (e < (ph + takes).view(-1, 1))
    taken = s["free_pages"][(avail - 1 - nth).clamp(min=0, max=s["n_pages"] - 1)]
    table.copy_(torch.where(fresh, taken, table))
    s["free_count_out"].copy_(avail - takes.sum())
    s["lens"].copy_(lens)
    s["cu_new"][0] = 0
    s["cu_new"][1:].copy_(torch.cumsum(grows, 0))
    x = torch.arange(s["max_tokens"], device=dev)
    b = (torch.searchsorted(s["cu_new"], x.to(torch.int32), right=True) - 1).clamp(max=c["batch"] - 1)
    j = x - s["cu_new"][b]
    slot = have[b] + j
    m = torch.stack((b, slot, table[b, (slot // page).clamp(max=s["max_pages"] - 1)].long(), s["pos"][b] + j), dim=1)
    s["token_map"].copy_(torch.where((x < s["cu_new"][-1]).view(-1, 1), m, torch.full_like(m, -1)))


def _frequencies(c):
    """The turned pairs' angles per position, in 64 bits (a list), and what a turned pair is multiplied by."""
    rd, theta, kind = c["rotary"], c["theta"], c["scaling"]
    f = [theta ** (-2.0 * i / rd) for i in range(rd // 2)]
    s = _SCALES.get(kind, {})
    if kind == "linear":
        f = [x / c["factor"] for x in f]
    elif kind == "wavelength":  # slow ones are stretched, fast ones stay, by the turns that they make
        for i, x in enumerate(f):
            w = (s["original"] * x / (2 * math.pi) - s["low"]) / (s["high"] - s["low"])
            w = min(1.0, max(0.0, w))
            f[i] = x * (w + (1.0 - w) / c["factor"])
    elif kind == "ramp":  # the same between two whole indexes, linear in the index
        def index(turns):
            return rd * math.log(s["original"] / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(index(s["high"])), 0), min(math.ceil(index(s["low"])), rd - 1)
        for i, x in enumerate(f):
            w = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f[i] = x * ((1.0 - w) + w / c["factor"])
    return f, s.get("magnitude", 1.0)


def _turn(x, pos, c):
    """x [N, H, d] in 32 bits, turned by pos [N]."""
    f, mag = _frequencies(c)
    a = pos.double().unsqueeze(-1) * torch.tensor(f, dtype=torch.float64, device=x.device)
    cos, sin = (torch.cos(a) * mag).float().unsqueeze(1), (torch.sin(a) * mag).float().unsqueeze(1)
    rd = c["rotary"]
    y = x.float().clone()
    i = slice(0, rd, 2) if c["layout"] == "interleaved" else slice(0, rd // 2)
    j = slice(1, rd, 2) if c["layout"] == "interleaved" else slice(rd // 2, rd)
    u, v = x[..., i].float(), x[..., j].float()
    y[..., i], y[..., j] = u * cos - v * sin, u * sin + v * cos
    return y


def _plain_rope(s, c):
    live = torch.nonzero(s["token_map"][:, 0] >= 0).flatten()
    b, slot, page, pos = (s["token_map"][live, i].long() for i in range(4))
    s["q_rot"][live] = _turn(s["q"][live], pos, c).to(s["q_rot"].dtype)
    at = slot % c["page"]
    s["k_pages"][page, :, at] = _turn(s["k"][live], pos, c).to(s["k_pages"].dtype)
    s["v_pages"][page, :, at] = s["v"][live]
    s["weight"][b, :, slot] = 0.0
    s["token_pos"][b, :, slot] = pos.to(torch.int32).unsqueeze(1)


def _plain_chunk(s, c, lens):
    hkv, G, d, page = c["hkv"], c["hq"] // c["hkv"], c["d"], c["page"]
    for b, (n, x0, x1) in enumerate(lens):
        m = x1 - x0
        if m == 0:
            continue
        used = s["page_table"][b, :-(-n // page)].long()
        k = s["k_pages"][used].transpose(0, 1).reshape(hkv, -1, d)[:, :n].float()
        v = s["v_pages"][used].transpose(0, 1).reshape(hkv, -1, d)[:, :n].float()
        step = max(1, int(2.5e8) // (c["hq"] * n))
        for j0 in range(0, m, step):
            j1 = min(m, j0 + step)
            see = n - m + j1  # slots that the last of these sees
            q = s["q_rot"][x0 + j0:x0 + j1].float().view(j1 - j0, hkv, G, d).permute(1, 0, 2, 3).reshape(hkv, -1, d)
            score = (torch.matmul(q, k[:, :see].transpose(1, 2)) / math.sqrt(d)).view(hkv, j1 - j0, G, see)
            mine = torch.arange(n - m + j0, n - m + j1, device=q.device).view(1, -1, 1, 1)
            score.masked_fill_(torch.arange(see, device=q.device) > mine, -math.inf)
            p = torch.exp(score - score.amax(dim=-1, keepdim=True))
            p = p / p.sum(dim=-1, keepdim=True)
            o = torch.matmul(p.view(hkv, -1, see), v[:, :see]).view(hkv, j1 - j0, G, d)
            s["out"][x0 + j0:x0 + j1] = o.permute(1, 0, 2, 3).reshape(j1 - j0, c["hq"], d).to(s["out"].dtype)
            if c["weights"]:
                s["weight"][b, :, :see].add_(p.sum(dim=(1, 2)))


# ------------------------------------------------------------------- one pass
def run(s):
    c, op = s["case"], s["case"]["op"]
    if own:
        import kv_cache_token_tip_gb300 as F
        if op in ("assign", "serve"):
            F.fasa_paged_assign(s["have"], s["want"], s["page_table"], s["free_pages"], s["free_count"], s["lens"],
                                s["cu_new"], s["token_map"], pos=s["pos"], free_count_out=s["free_count_out"],
                                dims=s["dims"])
        if op in ("rope", "serve"):
            F.fasa_paged_rope_append(s["q"], s["k"], s["v"], s["token_map"], s["q_rot"], s["k_pages"], s["v_pages"],
                                     weight=s["weight"], token_pos=s["token_pos"], rope=s["rope"], dims=s["dims"])
        if op in ("chunk", "serve"):
            F.fasa_paged_chunk_attention(s["q_rot"], s["k_pages"], s["v_pages"], s["page_table"],
                                         s["want"] if op == "chunk" else s["lens"], s["out"], cu_new=s["cu_new"],
                                         weight=s["weight"] if c["weights"] else None, workspace=s["workspace"],
                                         dims=s["dims"])
    else:
        if op in ("assign", "serve"):
            _plain_assign(s, c)
        if op in ("rope", "serve"):
            _plain_rope(s, c)
        if op in ("chunk", "serve"):
            cu = [int(x) for x in s["cu_new"].tolist()]
            n = (s["want"] if op == "chunk" else s["lens"]).tolist()
            _plain_chunk(s, c, [(n[b], cu[b], cu[b + 1]) for b in range(c["batch"])])
    out = {}
    if op in ("assign", "serve"):
        out.update({k: s[k] for k in ("page_table", "free_pages", "free_count_out", "lens", "cu_new", "token_map")})
    if op in ("rope", "serve"):
        out.update({k: s[k] for k in ("q_rot", "k_pages", "v_pages", "weight", "token_pos")})
    if op in ("chunk", "serve"):
        out["out"] = s["out"]
        if c["weights"]:
            out["weight"] = s["weight"]
    return out


# ------------------------------------------------------------------ the work
def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    have, want = _lens(c)
    op, d, hq, hkv, page = c["op"], c["d"], c["hq"], c["hkv"], c["page"]
    grown = [max(0, w - h) for h, w in zip(have, want)]
    tokens = sum(grown)
    bytes_, flops = 0, 0
    if op in ("assign", "serve"):
        moved = sum(abs(-(-h // page) - -(-w // page)) for h, w in zip(have, want))
        bytes_ += c["batch"] * (12 + 8) + moved * 8 + (tokens + c["pad"]) * 16
    if op in ("rope", "serve"):
        bytes_ += tokens * (2 * (hq + 2 * hkv) * d * es + 16 + 8 * hkv)
        flops += tokens * (hq + hkv) * c["rotary"] // 2 * 6
    if op in ("chunk", "serve"):
        for h, m in zip(have, grown):
            if m == 0:
                continue
            n = h + m
            bytes_ += 2 * m * hq * d * es + 2 * n * hkv * d * es + (8 * n * hkv if c["weights"] else 0)
            seen = m * h + m * (m + 1) // 2
            flops += 4 * d * hq * seen
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------- results in 64 bits
def exact(case, seed):
    """By the definitions, token by token or sequence by sequence, apart from the forms above.  (`serve`: its queries
    and keys are turned and stored before the attention reads them, so it goes by their stored values.)"""
    c = dict(case)
    op, hkv, G, d, page = c["op"], c["hkv"], c["hq"] // c["hkv"], c["d"], c["page"]
    if op == "assign":
        return None  # whole numbers alone
    s = prepare(case, seed)
    have, want = _lens(c)
    if op == "serve" and any(w < h for h, w in zip(have, want)):
        return None
    out = {}
    table = s["page_table"]
    tokens = [(b, have[b] + j, j) for b in range(c["batch"]) for j in range(max(0, want[b] - have[b]))]
    if op == "serve":
        # pages as the list gives them, from its end
        free, t = s["free_pages"].tolist()[:int(s["free_count"])], table.tolist()
        total = 0
        for b in range(c["batch"]):
            total += want[b] - have[b]
            first, last = -(-have[b] // page), -(-want[b] // page)
            if len(free) < last - first or total > s["max_tokens"]:
                return None
            for e in range(first, last):
                t[b][e] = free.pop()
        table = torch.tensor(t, dtype=torch.int32, device=table.device)
        out.update(page_table=None, free_pages=None, free_count_out=None, lens=None, cu_new=None, token_map=None)
    w = s["weight"].double()
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    q = s["q_rot"].double()
    if op in ("rope", "serve"):
        dev = q.device
        b = torch.tensor([x[0] for x in tokens], device=dev)
        slot = torch.tensor([x[1] for x in tokens], device=dev)
        pos = s["pos"].long()[b] + torch.tensor([x[2] for x in tokens], device=dev)
        f, mag = _frequencies(c)
        rd, n = c["rotary"], len(tokens)
        a = pos.double().view(-1, 1, 1) * torch.tensor(f, dtype=torch.float64, device=dev)
        turn = torch.polar(torch.full_like(a, mag), a)

        def turned(x):
            x = x[:n].double()
            h = x.shape[1]
            head = x[..., :rd]
            if c["layout"] == "interleaved":
                z = torch.view_as_complex(head.reshape(n, h, rd // 2, 2).contiguous()) * turn
                y = torch.view_as_real(z).reshape(n, h, rd)
            else:
                z = torch.complex(head[..., :rd // 2].contiguous(), head[..., rd // 2:].contiguous()) * turn
                y = torch.cat((z.real, z.imag), dim=-1)
            return torch.cat((y, x[..., rd:]), dim=-1)

        pg, at = table.long()[b, slot // page], slot % page
        kp[pg, :, at], vp[pg, :, at] = turned(s["k"]), s["v"][:n].double()
        q[:n] = turned(s["q"])
        w[b, :, slot] = 0.0
        out.update(q_rot=q, k_pages=kp, v_pages=vp, weight=w, token_pos=None)
        if op == "rope":
            return out
        stored = s["q_rot"].dtype
        q, kp = q.to(stored).double(), kp.to(stored).double()
    o = torch.zeros_like(q)
    x = 0
    for b in range(c["batch"]):
        n, m = want[b], want[b] - have[b]
        if m == 0:
            continue
        pages = table[b, :-(-n // page)].long()
        for h in range(hkv):
            k, v = kp[pages, h].reshape(-1, d)[:n], vp[pages, h].reshape(-1, d)[:n]
            for j0 in range(0, m, 512):
                j1 = min(m, j0 + 512)
                see = n - m + j1
                qh = q[x + j0:x + j1, h * G:(h + 1) * G].reshape(-1, d)
                z = (qh @ k[:see].T / math.sqrt(d)).view(j1 - j0, G, see)
                hidden = torch.ones(j1 - j0, see, dtype=torch.bool, device=z.device).triu(see - (j1 - j0) + 1)
                p = torch.softmax(z.masked_fill(hidden.unsqueeze(1), -math.inf), dim=-1)
                o[x + j0:x + j1, h * G:(h + 1) * G] = (p.view(-1, see) @ v[:see]).view(j1 - j0, G, d)
                if c["weights"]:
                    w[b, h, :see] += p.sum(dim=(0, 1))
        x += m
    out["out"] = o
    if c["weights"]:
        out["weight"] = w
    return out
