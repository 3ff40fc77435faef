"""The paged key-value cache and the attention of new tokens over it: what is measured.

Three operators, each as elementary torch operations in 32 bits (``own`` false) or as the
framework's calls (``own`` true):

append  K and V rows of new tokens written into the pages of a cache, as bf16 or as e4m3
        codes with one power-of-two scale per row.
read    the rows of a cache, gathered from their pages into contiguous bf16 [B,H,N,d].
decode  attention of the last T tokens of each sequence over its cached keys and values,
        with grouped heads, ragged lengths and, optionally, lists of kept pages.

Lengths follow from the case alone (the bytes of a pass do); values, page tables and kept
lists follow from the seed. Table entries past a sequence's last page are -1.
"""
import math

import torch

own = False

SPARE_PAGES = 3   # pages of the pool that no sequence owns


# ------------------------------------------------------------------ cases
def _case(name, op, **kw):
    base = dict(op=op, B=1, H=16, G=1, T=1, d=128, page=64, cache="bf16", out="bf16",
                longest=4096, shortest=0, first=0, keep=0, lse=False, token_major=False)
    base.update(kw)
    if name:
        base["name"] = name
    return base


def listed():
    return [
        # a small model's single stream, two heads of 64, 4,096 cached tokens: latency counts
        _case("decode-2heads-4096-d64", "decode", H=2, d=64, longest=4096, out="f32"),
        # one token after one cached frame of 1,560 tokens: latency counts
        _case("decode-1frame-bf16", "decode", H=16, longest=1560),
        # four world-model rollouts with the whole cache of 41 frames of 1,560 tokens
        _case("decode-4x63960-bf16", "decode", B=4, H=16, longest=63960),
        # one 720p-sized cache of 40 heads in 8 bits, large pages
        _case("decode-75600-40heads-e4m3", "decode", H=40, longest=75600, page=128, cache="e4m3"),
        # many requests of very different lengths (none at all among them), grouped heads, small pages
        _case("decode-64ragged-gqa-e4m3", "decode", B=64, H=8, G=4, longest=8191, shortest=1,
              page=16, cache="e4m3"),
        # four new tokens checked at once on long caches with eight query heads per key head
        _case("decode-4tokens-gqa-f32", "decode", B=2, H=2, G=8, T=4, longest=63957,
              shortest=40001, page=32, out="f32", lse=True),
        # the same rollouts with a tenth of the pages kept by a routing step
        _case("decode-4x63960-kept-bf16", "decode", B=4, H=16, longest=63960, keep=100, lse=True),
        # one token per rollout stored in 8 bits: the smallest call
        _case("append-1token-e4m3", "append", B=4, H=16, T=1, first=63959, cache="e4m3"),
        # one frame per rollout, straight from a token-major projection
        _case("append-frame-e4m3", "append", B=4, H=16, T=1560, first=62400, cache="e4m3",
              token_major=True),
        # a whole 720p-sized prompt of 40 heads
        _case("append-75600-40heads-bf16", "append", H=40, T=75600, page=128),
        # the last frame of a cache of each type read back, and a whole 8-bit cache
        _case("read-frame-bf16", "read", B=4, H=16, longest=63960, first=62400),
        _case("read-4x63960-e4m3", "read", B=4, H=16, longest=63960, cache="e4m3"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "read"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    cache = rng.choice(["bf16", "e4m3"])
    B, H = _log_int(rng, 1, 64), _log_int(rng, 1, 40)
    longest = _log_int(rng, 1, 75600)
    # no drawn case moves more bytes, or takes more operations, than the largest listed one
    longest = max(1, min(longest, 3_000_000 // (B * H)))
    if op == "decode":
        G = rng.choice([1, 1, 2, 4, 5, 8, 16])
        T = rng.choice([1, 1, 1, 2, 3, 8])
        longest = max(1, min(longest, 8_000_000 // (B * H * G * T)))
        pages = -(-longest // page)
        keep = rng.choice([0, 0, max(1, pages // 10)])
        return _case(None, op, B=B, H=H, G=G, T=T, d=d, page=page, cache=cache,
                     out=rng.choice(["bf16", "f32"]), longest=longest,
                     shortest=rng.choice([0, 1, max(1, longest // 2)]), keep=keep,
                     lse=rng.random() < 0.5)
    if op == "append":
        T = longest
        return _case(None, op, B=B, H=H, T=T, d=d, page=page, cache=cache,
                     first=_log_int(rng, 1, 4096) - 1, shortest=rng.choice([0, 1]),
                     token_major=rng.random() < 0.5)
    return _case(None, op, B=B, H=H, d=d, page=page, cache=cache, longest=longest,
                 shortest=rng.choice([0, 1, max(1, longest // 2)]),
                 first=rng.choice([0, longest // 2]))


def _spread(B, lo, hi):
    """B whole numbers of [lo, hi] spread evenly in no order: hi first, then lo."""
    got = [hi, lo]
    got += [lo + int((hi - lo) * math.modf(i * 0.6180339887498949)[0]) for i in range(2, B)]
    return got[:B]


def _lengths(case):
    """(first row, rows) that each sequence brings: appended, read, or cached for decode."""
    B = case["B"]
    if case["op"] == "append":
        first = _spread(B, max(0, case["first"] - 7), case["first"])
        count = _spread(B, 0 if case["shortest"] else case["T"], case["T"])
        return first, count
    longest = case["longest"]
    shortest = case["shortest"] - 1 if case["shortest"] else longest   # 0: all equal
    lens = _spread(B, shortest, longest)
    if case["op"] == "read":
        return [min(case["first"], n) for n in lens], lens
    return [0] * B, lens


# ------------------------------------------------------------------ inputs
def _quantise(x):
    """(e4m3 codes, E8M0 scales) of rows of x: the scale is the smallest power of two that
    brings the row's largest finite magnitude to at most 448 (1 for a row of zeros)."""
    x = x.float()
    top = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1)
    mant, e = torch.frexp(top)                      # top = mant * 2^e, mant in [0.5, 1)
    e = torch.where(mant > 0.875, e - 8, e - 9)     # 448 = 0.875 * 2^9
    e = torch.where(top > 0, e.clamp(min=-126), torch.zeros_like(e))
    codes = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _scale_values(s):
    return torch.ldexp(torch.ones(s.shape, device=s.device), s.view(torch.uint8).int() - 127)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    B, H, T, d, page = case["B"], case["H"], case["T"], case["d"], case["page"]
    randn = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    first, rows = _lengths(case)
    ends = [f + n for f, n in zip(first, rows)] if case["op"] == "append" else rows
    used = [-(-n // page) for n in ends]
    width, total = max(1, max(used)), sum(used) + SPARE_PAGES
    perm = torch.randperm(total, generator=g, device=dev).int()
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    cols = torch.arange(width, device=dev)
    owned = cols[None, :] < torch.tensor(used, device=dev)[:, None]
    table[owned] = perm[:sum(used)]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    st = dict(case=case, table=table)
    if case["op"] == "append":
        shape = (B, T, H, d) if case["token_major"] else (B, H, T, d)
        k, v = randn(*shape).bfloat16(), randn(*shape).bfloat16()
        if case["token_major"]:
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        dt = torch.bfloat16 if case["cache"] == "bf16" else torch.float8_e4m3fn
        st.update(k_new=k, v_new=v, start=ints(first), count=ints(rows),
                  k=torch.zeros(total, H, page, d, device=dev).to(dt),
                  v=torch.zeros(total, H, page, d, device=dev).to(dt), k_scale=None, v_scale=None)
        if case["cache"] == "e4m3":
            st.update({n: torch.full((total, H, page), 127, dtype=torch.uint8, device=dev)
                       .view(torch.float8_e8m0fnu) for n in ("k_scale", "v_scale")})
        return st
    # keys near one centre per page, a few of them outliers; values without structure
    centre = randn(total, H, 1, d)
    k = centre + 0.3 * randn(total, H, page, d)
    k[torch.rand(total, H, page, generator=g, device=dev) < 0.02] *= 2
    k, v = k.bfloat16(), randn(total, H, page, d).bfloat16()
    st.update(k=k, v=v, k_scale=None, v_scale=None, lens=ints(rows))
    if case["cache"] == "e4m3":
        st["k"], st["k_scale"] = _quantise(k)
        st["v"], st["v_scale"] = _quantise(v)
    if case["op"] == "read":
        st.update(first=ints(first),
                  k_out=torch.zeros(B, H, max(1, case["longest"]), d, dtype=torch.bfloat16, device=dev),
                  v_out=torch.zeros(B, H, max(1, case["longest"]), d, dtype=torch.bfloat16, device=dev))
        return st
    G = case["G"]
    at = torch.randint(0, total, (B, H, G, T), generator=g, device=dev)
    q = centre[at, torch.arange(H, device=dev)[None, :, None, None], 0] + 0.5 * randn(B, H, G, T, d)
    st["q"] = (0.7 * q).reshape(B, H * G, T, d).bfloat16()
    st["idx"] = st["cnt"] = None
    if case["keep"]:
        # random distinct pages of each sequence in ascending order, as a routing step lists them
        score = torch.rand(B, H, width, generator=g, device=dev)
        score = score.masked_fill(~owned[:, None, :], 2.0)
        picked = score.argsort(-1)[..., :case["keep"]]
        cnt = torch.minimum(ints(used), ints([case["keep"]] * B))
        live = torch.arange(picked.shape[-1], device=dev)[None, None, :] < cnt[:, None, None]
        st["idx"] = picked.masked_fill(~live, width).sort(-1).values.int().contiguous()
        st["cnt"] = cnt[:, None].expand(B, H).contiguous()
    return st


# ------------------------------------------------------------------ plain forms
def _plain_append(st):
    page = st["case"]["page"]
    B, H, T, d = st["k_new"].shape
    t = torch.arange(T, device="cuda")
    pos = st["start"].long()[:, None] + t
    live = t < st["count"][:, None]
    b, t = live.nonzero(as_tuple=True)
    pos = pos[b, t]
    pg = st["table"][b, pos // page].long()
    for name in ("k", "v"):
        x = st[name + "_new"][b, :, t].float()      # [rows, H, d]
        if st["k_scale"] is None:
            st[name][pg, :, pos % page] = x.bfloat16()
        else:
            codes, scales = _quantise(x)
            st[name].view(torch.uint8)[pg, :, pos % page] = codes.view(torch.uint8)
            st[name + "_scale"].view(torch.uint8)[pg, :, pos % page] = scales.view(torch.uint8)


def _values(st, name, pages):
    """fp32 rows of the pages: [..., H, page, d]."""
    x = st[name].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float() \
        if st["k_scale"] is not None else st[name][pages].float()
    if st["k_scale"] is not None:
        x *= _scale_values(st[name + "_scale"])[pages][..., None]
    return x


def _plain_read(st):
    page, N = st["case"]["page"], st["k_out"].shape[2]
    t = torch.arange(N, device="cuda")
    live = (t >= st["first"][:, None]) & (t < st["lens"][:, None])
    b, t = live.nonzero(as_tuple=True)
    pg = st["table"][b, t // page].long()
    for name in ("k", "v"):
        if st["k_scale"] is None:
            st[name + "_out"][b, :, t] = st[name][pg, :, t % page]
        else:
            x = st[name].view(torch.uint8)[pg, :, t % page].view(torch.float8_e4m3fn).float()
            s = _scale_values(st[name + "_scale"].view(torch.uint8)[pg, :, t % page])
            st[name + "_out"][b, :, t] = (x * s[..., None]).bfloat16()


def _plain_decode(st):
    c = st["case"]
    B, H, G, T, d, page = c["B"], c["H"], c["G"], c["T"], c["d"], c["page"]
    q = st["q"].float().view(B, H, G * T, d)
    width = st["table"].shape[1]
    if st["idx"] is None:
        pages = st["table"].clamp(min=0).long()                       # [B, W]
        k, v = (_values(st, n, pages).transpose(1, 2).reshape(B, H, -1, d) for n in ("k", "v"))
        pos = torch.arange(width * page, device="cuda").expand(B, H, -1)
    else:
        logical = st["idx"].long()                                    # [B, H, cap]
        bb = torch.arange(B, device="cuda")[:, None, None]
        hh = torch.arange(H, device="cuda")[None, :, None]
        pages = st["table"][bb, logical.clamp(max=width - 1)].clamp(min=0).long()
        k, v = (_listed_values(st, n, pages, hh).reshape(B, H, -1, d) for n in ("k", "v"))
        listed_page = torch.arange(logical.shape[-1], device="cuda") < st["cnt"][..., None]
        pos = logical[..., None] * page + torch.arange(page, device="cuda")
        pos = torch.where(listed_page[..., None], pos, torch.full_like(pos, 1 << 40)).reshape(B, H, -1)
    s = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)           # [B, H, G*T, keys]
    sees = st["lens"].long()[:, None] - torch.arange(T - 1, -1, -1, device="cuda")   # [B, T]
    mask = pos[:, :, None, :] < sees[:, None, :, None]                # [B, H, T, keys]
    mask = mask[:, :, None].expand(B, H, G, T, -1).reshape(B, H, G * T, -1)
    s = s.masked_fill(~mask, float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m.clamp(min=-3e38))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / total.clamp(min=1e-30)
    out = o.view(B, H * G, T, d).to(torch.bfloat16 if c["out"] == "bf16" else torch.float32)
    lse = (m + total.log()).view(B, H * G, T)
    return out, torch.where(lse.isnan(), torch.full_like(lse, float("-inf")), lse)


def _listed_values(st, name, pages, heads):
    """fp32 rows of the listed pages of each head: [B, H, cap, page, d]."""
    if st["k_scale"] is None:
        return st[name][pages, heads].float()
    x = st[name].view(torch.uint8)[pages, heads].view(torch.float8_e4m3fn).float()
    return x * _scale_values(st[name + "_scale"].view(torch.uint8)[pages, heads])[..., None]


# ------------------------------------------------------------------ one pass
def run(state):
    st, c = state, state["case"]
    if own:
        from free_block_sparse_kv_b200 import paged_cache as P
        cache = P.PagedCache(st["k"], st["v"], st["k_scale"], st["v_scale"])
        if c["op"] == "append":
            P.cache_append(cache, st["k_new"], st["v_new"], st["table"], st["start"], st["count"])
        elif c["op"] == "read":
            P.cache_read(cache, st["table"], st["lens"], st["k_out"], st["v_out"], first=st["first"])
        else:
            out = P.decode(st["q"], cache, st["table"], st["lens"], kv_idx=st["idx"], kv_cnt=st["cnt"],
                           out_dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32,
                           return_lse=c["lse"])
            return {"out": out[0], "lse": out[1]} if c["lse"] else {"out": out}
    elif c["op"] == "append":
        _plain_append(st)
    elif c["op"] == "read":
        _plain_read(st)
    else:
        out, lse = _plain_decode(st)
        return {"out": out, "lse": lse} if c["lse"] else {"out": out}
    if c["op"] == "append":
        got = {"k": st["k"], "v": st["v"]}
        if st["k_scale"] is not None:
            got.update(k_scale=st["k_scale"], v_scale=st["v_scale"])
        return got
    return {"k": st["k_out"], "v": st["v_out"]}


def work(case):
    H, d, T = case["H"], case["d"], case["T"]
    first, rows = _lengths(case)
    held = 2 * (2 * d if case["cache"] == "bf16" else d + 1)     # K and V of a cached row
    if case["op"] == "append":
        n = sum(rows) * H
        return {"bytes": n * (4 * d + held), "flops": 4 * n * d if case["cache"] == "e4m3" else 0}
    if case["op"] == "read":
        n = sum(e - f for f, e in zip(first, rows)) * H
        return {"bytes": n * (4 * d + held), "flops": 2 * n * d if case["cache"] == "e4m3" else 0}
    keys = [min(n, case["keep"] * case["page"]) if case["keep"] else n for n in rows]
    R = case["G"] * T
    io = len(rows) * H * R * (2 * d + (2 if case["out"] == "bf16" else 4) * d + 4 * case["lse"])
    return {"bytes": sum(keys) * H * held + io, "flops": 4.0 * sum(keys) * H * R * d}


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _e4m3_64(y):
    """y rounded to the nearest e4m3 value (ties to even), |y| <= 448: three significand
    bits after the first, spacing 2^-9 below 2^-6."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step


def _held_64(st, name, b, h):
    """Rows of sequence b, head h in position order, in 64 bits, over its owned pages."""
    pages = st["table"][b]
    pages = pages[pages >= 0].long()
    x = st[name].view(torch.uint8)[pages, h].view(torch.float8_e4m3fn).double() \
        if st["k_scale"] is not None else st[name][pages, h].double()
    if st["k_scale"] is not None:
        e = st[name + "_scale"].view(torch.uint8)[pages, h].double()
        x = x * torch.exp2(e - 127)[..., None]
    return x.reshape(-1, x.shape[-1])


def exact(case, seed):
    st = prepare(case, seed)
    B, H, G, T, d, page = (case[n] for n in ("B", "H", "G", "T", "d", "page"))
    if case["op"] == "append":
        if B * H * T > 8_000_000:
            return None
        got = {n: st[n].double() for n in ("k", "v")}
        if case["cache"] == "e4m3":
            got.update({n: torch.ones(st[n].shape, dtype=torch.float64, device="cuda")
                        for n in ("k_scale", "v_scale")})
        for b in range(B):
            n, s = int(st["count"][b]), int(st["start"][b])
            if not n:
                continue
            at = torch.arange(s, s + n, device="cuda")
            pg, row = st["table"][b][at // page].long(), at % page
            for name in ("k", "v"):
                x = st[name + "_new"][b, :, :n].transpose(0, 1).double()
                if case["cache"] == "e4m3":
                    top = x.abs().amax(-1)
                    scale = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** -100) / 448)))
                    scale = torch.where(top > 0, scale, torch.ones_like(scale))
                    got[name + "_scale"][pg, :, row] = scale
                    x = _e4m3_64(x / scale[..., None])
                got[name][pg, :, row] = x
        return got
    if case["op"] == "read":
        got = {"k": st["k_out"].double(), "v": st["v_out"].double()}
        for b in range(B):
            f, n = int(st["first"][b]), int(st["lens"][b])
            for h in range(H):
                for name in ("k", "v"):
                    got[name][b, h, f:n] = _held_64(st, name, b, h)[f:n]
        return got
    out = torch.zeros(B, H * G, T, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H * G, T), float("-inf"), dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(st["lens"][b])
        for h in range(H):
            if n == 0:
                continue
            at = torch.arange(n, device="cuda")
            if st["idx"] is not None:
                kept = st["idx"][b, h, :int(st["cnt"][b, h])].long()
                at = at[torch.isin(at // page, kept)]
            k, v = _held_64(st, "k", b, h)[at], _held_64(st, "v", b, h)[at]
            seen = at[None, :] <= n - T + torch.arange(T, device="cuda")[:, None]      # [T, keys]
            logit = st["q"][b, h * G:(h + 1) * G].double() @ k.T / math.sqrt(d)        # [G, T, keys]
            logit = torch.where(seen, logit, torch.full_like(logit, float("-inf")))
            total = torch.logsumexp(logit, -1)
            share = torch.where(seen, torch.exp(logit - total[..., None]), torch.zeros_like(logit))
            lse[b, h * G:(h + 1) * G] = total
            out[b, h * G:(h + 1) * G] = share @ v
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
