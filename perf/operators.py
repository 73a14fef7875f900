"""The operators around an 8-bit paged KV cache: what is measured, and their plain forms.

* rope:   rotary positions of query and key rows (kt_apply_rope);
* append: rotate, code to 8 bits and write new tokens into the paged cache, with the
          representatives of the blocks they complete (kt_append_kv_f8);
* read:   tokens of the cache back as binary16 rows (kt_read_kv_f8);
* attend: decode attention over the cache, dense, over a given block selection, or as the
          decode step that also makes the selection (kt_dense_decode_attn_f8,
          kt_sparse_decode_attn_f8, kt_sparse_decode_step_f8).

The cache: e4m3 codes [pages][KV heads][128 tokens][128 channels] and one binary32 scale per
(page, KV head), a power of two 2^e: the least e in [-15, 8] with amax <= 448 2^e over the values
the block has held since it was begun.  A value is code * scale; rows are rounded to binary16
before they are coded, and codes are at most 240 where e is 8, so that a value is a finite
binary16.

`own` false: elementary torch operations in 32 bits (64 for angles and block scores).  `own`
true: the framework's calls.
"""
import math

import torch

own = False

D = 128   # channels of a head
BS = 128  # tokens of a block
F8 = torch.float8_e4m3fn
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


# ---- cases ------------------------------------------------------------------------------
def listed():
    return [
        # one decode step of 16 sequences: the packed projection's q and k heads, rotated
        rope_case("rope-decode-16", tokens=16, q=32, kv=8, dtype="bf16", layout="half", rot=128,
                  scaling="plain", theta=1e6, factor=1.0, far=65536),
        # a prefill chunk of a long-context model (NTK-scaled base)
        rope_case("rope-prefill-8k", tokens=8192, q=32, kv=8, dtype="bf16", layout="half", rot=128,
                  scaling="ntk", theta=5e6, factor=4.0, far=131072),
        # binary32 rows, half of each head rotated in neighbouring pairs, positions up to 1M
        rope_case("rope-partial-1m", tokens=5003, q=16, kv=4, dtype="f32", layout="pairs", rot=64,
                  scaling="yarn", theta=1e4, factor=32.0, far=1048576),
        # one decoded token for each of 16 sequences of 8K to 64K, queries rotated in the same call
        append_case("append-decode-16", batch=16, least=1, most=1, start=65536, q=32, kv=8,
                    dtype="bf16", rope=True, rep="quest"),
        # the last chunk of a 128K prompt, from the middle of a block
        append_case("append-prefill-16k", batch=1, least=16384, most=16384, start=114000, q=32,
                    kv=8, dtype="bf16", rope=True, rep="quest"),
        # mixed prefill and decode rows of 7 sequences, already rotated
        append_case("append-ragged-7", batch=7, least=1, most=6000, start=5000, q=0, kv=4,
                    dtype="f16", rope=False, rep="mean"),
        # the ends of 5 cached sequences, for a kernel that takes contiguous binary16 rows
        read_case("read-ragged-5", batch=5, least=1, most=700, start=3000, kv=8),
        # a whole 128K prefix
        read_case("read-prefix-128k", batch=1, least=131072, most=131072, start=0, kv=8),
        # the first decode steps of short chats: 8 sequences of 1 to 300 tokens
        attend_case("dense-short-8", how="dense", batch=8, least=1, most=300, q=32, kv=8),
        # a dense layer over one 128K sequence
        attend_case("dense-128k", how="dense", batch=1, least=131072, most=131072, q=32, kv=8),
        # a batch of 16 at mixed lengths, the selection reused from an earlier layer
        attend_case("sparse-ragged-16", how="sparse", batch=16, least=8192, most=65536, q=32, kv=8,
                    initial=1, local=16, top_k=16, mode="separate"),
        # the 128K decode step: score the blocks' representatives, pick 32, attend
        attend_case("step-128k", how="step", batch=1, least=131072, most=131072, q=32, kv=8,
                    initial=1, local=32, top_k=32, mode="shared"),
    ]


def rope_case(name, **kw):
    return dict(name=name, op="rope", **kw)


def append_case(name, **kw):
    return dict(name=name, op="append", **kw)


def read_case(name, **kw):
    return dict(name=name, op="read", **kw)


def attend_case(name, initial=0, local=0, top_k=0, mode="shared", **kw):
    return dict(name=name, op="attend", initial=initial, local=local, top_k=top_k, mode=mode, **kw)


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "attend", "attend"])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 8])
    if op == "rope":
        scaling = rng.choice(["plain", "linear", "ntk", "yarn"])
        case = rope_case("", tokens=_spread(rng, 1, 8192), q=kv * group, kv=kv,
                         dtype=rng.choice(["f16", "bf16", "f32"]),
                         layout=rng.choice(["half", "pairs"]),
                         rot=rng.choice([128, 128, 64, 96, 32, 2 * rng.randint(2, 63)]),
                         scaling=scaling, theta=rng.choice([1e4, 1e6, 5e7]),
                         factor=1.0 if scaling == "plain" else float(rng.choice([2, 4, 8, 40])),
                         far=_spread(rng, 64, 1048576))
    elif op == "append":
        batch = rng.choice([1, 2, 5, 16])
        most = _spread(rng, 1, 16384 // batch)
        case = append_case("", batch=batch, least=rng.choice([1, most]), most=most,
                           start=_spread(rng, 1, 65536 // batch), q=rng.choice([0, kv * group]),
                           kv=kv, dtype=rng.choice(["f16", "bf16", "f32"]),
                           rope=rng.random() < 0.7, rep=rng.choice(["max", "mean", "quest", "fix"]))
    elif op == "read":
        batch = rng.choice([1, 3, 8])
        most = _spread(rng, 1, 131072 // batch)
        case = read_case("", batch=batch, least=rng.choice([1, most]), most=most,
                         start=_spread(rng, 1, 4096), kv=kv)
    else:
        how = rng.choice(["dense", "sparse", "step"])
        batch = rng.choice([1, 2, 7, 16])
        most = _spread(rng, 1 if how == "dense" else 2048, 131072 // batch)
        kept = {} if how == "dense" else dict(initial=rng.choice([0, 1, 2]),
                                              local=rng.choice([1, 4, 16]),
                                              top_k=rng.choice([4, 8, 16, 32]),
                                              mode=rng.choice(["shared", "separate"]))
        case = attend_case("", how=how, batch=batch, least=max(1, most // rng.choice([1, 2, 4])),
                           most=most, q=kv * group, kv=kv, **kept)
    del case["name"]
    return case


# ---- inputs -----------------------------------------------------------------------------
def _lengths(least, most, batch):
    """`batch` whole numbers from `most` down to `least`: the same for every seed."""
    return [most - (most - least) * i // max(1, batch - 1) for i in range(batch)]


def _starts(least, most, batch, gen):
    """`batch` whole numbers of [least, most], the first one `most`."""
    x = torch.rand(batch, generator=gen).mul_(most - least + 1).to(torch.int64).add_(least)
    x[0] = most
    return x.clamp_(max=most).to(torch.int32)


def _projection(gen, tokens, heads, dtype):
    """Rows of the packed projection [tokens][heads][128], a few channels of them large."""
    x = torch.randn(tokens, heads, D, generator=gen, device=DEV)
    x[:, :, [5, 37, 66, 101]] *= 4.0
    return x.to(dtype)


def _pages(gen, batch, blocks):
    """A block table over a shuffled pool with a few spare pages, and the pool's pages."""
    pages = batch * blocks + 3
    order = torch.randperm(pages, generator=gen, device=DEV)[: batch * blocks]
    return order.to(torch.int32).reshape(batch, blocks).contiguous(), pages


def _cache(gen, pages, kv):
    """A filled cache: codes and scales of random values, in slices of pages."""
    code = torch.empty(pages, kv, BS, D, dtype=F8, device=DEV)
    scale = torch.empty(pages, kv, dtype=torch.float32, device=DEV)
    for lo in range(0, pages, 256):
        n = min(256, pages - lo)
        x = torch.randn(n, kv, BS, D, generator=gen, device=DEV)
        x[..., [9, 77]] *= 6.0
        x = x * torch.exp2(torch.randint(-1, 2, (n, kv, 1, 1), generator=gen, device=DEV).float())
        s = block_scale(x.abs().amax(dim=(2, 3)))
        code[lo:lo + n] = (x / s[:, :, None, None]).to(F8)
        scale[lo:lo + n] = s
    return code, scale


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    cpu = torch.Generator()
    cpu.manual_seed(int(seed))
    c = dict(case)
    st = {"case": c}
    if c["op"] == "rope":
        heads = c["q"] + 2 * c["kv"]  # q, k and v heads of one packed projection
        st["qkv"] = _projection(gen, c["tokens"], heads, TYPES[c["dtype"]])
        top = torch.randint(0, c["far"], (1,), generator=gen, device=DEV)
        st["positions"] = (top + torch.arange(c["tokens"], device=DEV)).to(torch.int32)
        st["q_out"] = torch.zeros(c["tokens"], c["q"], D, dtype=torch.float16, device=DEV)
        st["k_out"] = torch.zeros(c["tokens"], c["kv"], D, dtype=torch.float16, device=DEV)
        return st
    batch, kv = c["batch"], c["kv"]
    if c["op"] == "append":
        new = torch.tensor(_lengths(c["least"], c["most"], batch), dtype=torch.int32)
        start = _starts(c["start"] // 2, c["start"], batch, cpu)
        total = int(new.sum())
        blocks = -(-int((start + new).max()) // BS)
        st["table"], pages = _pages(gen, batch, blocks)
        st["k_code"], st["k_scale"] = _cache(gen, pages, kv)
        st["v_code"], st["v_scale"] = _cache(gen, pages, kv)
        st["lens"] = start.to(DEV)
        st["new_lens"] = torch.zeros_like(st["lens"])
        cu = torch.zeros(batch + 1, dtype=torch.int32)
        cu[1:] = new.cumsum(0)
        st["cu"], st["tokens"] = cu.to(DEV), total
        st["qkv"] = _projection(gen, total, c["q"] + 2 * kv, TYPES[c["dtype"]])
        st["q_out"] = torch.zeros(total, c["q"], D, dtype=torch.float16, device=DEV) \
            if c["q"] else None
        rows = {"max": 1, "mean": 1, "quest": 2, "fix": 4}[c["rep"]]
        st["reps"] = torch.zeros(pages, kv, rows, D, device=DEV,
                                 dtype=torch.float32 if c["rep"] == "mean" else torch.float16)
        return st
    if c["op"] == "read":
        new = torch.tensor(_lengths(c["least"], c["most"], batch), dtype=torch.int32)
        first = _starts(c["start"] // 2, c["start"], batch, cpu)
        lens = first + new
        st["table"], pages = _pages(gen, batch, -(-int(lens.max()) // BS))
        st["k_code"], st["k_scale"] = _cache(gen, pages, kv)
        st["v_code"], st["v_scale"] = _cache(gen, pages, kv)
        cu = torch.zeros(batch + 1, dtype=torch.int32)
        cu[1:] = new.cumsum(0)
        st["cu"], st["tokens"] = cu.to(DEV), int(new.sum())
        st["first"], st["lens"] = first.to(DEV), lens.to(DEV)
        st["k_out"] = torch.zeros(st["tokens"], kv, D, dtype=torch.float16, device=DEV)
        st["v_out"] = torch.zeros_like(st["k_out"])
        return st
    lens = torch.tensor(_lengths(c["least"], c["most"], batch), dtype=torch.int32)
    blocks = -(-int(lens.max()) // BS)
    st["table"], pages = _pages(gen, batch, blocks)
    st["k_code"], st["k_scale"] = _cache(gen, pages, kv)
    st["v_code"], st["v_scale"] = _cache(gen, pages, kv)
    st["lens"] = lens.to(DEV)
    q = torch.randn(batch, c["q"], D, generator=gen, device=DEV).half()
    st["q"] = q
    st["out"] = torch.zeros(batch, c["q"], D, dtype=torch.float32, device=DEV)
    if c["how"] == "dense":
        return st
    units, k = (1 if c["mode"] == "shared" else kv), c["top_k"]
    # a needle workload: in each unit's context, top_k blocks answer to its queries
    sel = torch.zeros(batch, units, k, dtype=torch.int32)
    cnt = torch.zeros(batch, units, dtype=torch.int32)
    for b in range(batch):
        nb = -(-int(lens[b]) // BS)
        c0 = min(c["initial"], nb)
        c1 = max(c0, nb - c["local"])
        for u in range(units):
            n = min(k, c1 - c0)
            ids = (torch.randperm(c1 - c0, generator=cpu)[:n] + c0).sort().values
            sel[b, u, :n], cnt[b, u] = ids.to(torch.int32), n
    if c["how"] == "sparse":
        st["sel"], st["cnt"] = sel.to(DEV), cnt.to(DEV)
        return st
    group = q.float().reshape(batch, kv, c["q"] // kv, D).sum(2)
    toward = 3.0 * group / group.norm(dim=-1, keepdim=True)
    for b in range(batch):
        for h in range(kv):
            u = 0 if units == 1 else h
            page = st["table"][b, sel[b, u, : int(cnt[b, u])].long().to(DEV)].long()
            x = st["k_code"][page, h].float() * st["k_scale"][page, h][:, None, None]
            x = x + toward[b, h]
            s = block_scale(x.abs().amax(dim=(1, 2)))
            st["k_code"][page, h] = (x / s[:, None, None]).to(F8)
            st["k_scale"][page, h] = s
    st["reps"] = torch.empty(pages, kv, 2, D, dtype=torch.float16, device=DEV)
    for lo in range(0, pages, 256):
        x = st["k_code"][lo:lo + 256].float() * st["k_scale"][lo:lo + 256, :, None, None]
        st["reps"][lo:lo + 256, :, 0] = x.amin(2)
        st["reps"][lo:lo + 256, :, 1] = x.amax(2)
    st["sel"] = torch.zeros(batch, units, k, dtype=torch.int32, device=DEV)
    st["cnt"] = torch.zeros(batch, units, dtype=torch.int32, device=DEV)
    return st


# ---- plain forms ------------------------------------------------------------------------
def block_scale(amax):
    """2^e, the least e in [-15, 8] with amax <= 448 2^e."""
    m, e = torch.frexp(amax.double() / 448.0)
    e = torch.where(m > 0.5, e, e - 1).clamp(-15, 8)
    return torch.exp2(torch.where(amax > 0, e, torch.full_like(e, -15)).float())


def frequencies(rot, theta, scaling, factor):
    """Angles per position in 64 bits, and the factor on the rotated channels."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    f = torch.exp(-2.0 * i / rot * math.log(theta))
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        turn = [rot * math.log(8192 / (beta * 2 * math.pi)) / (2 * math.log(theta))
                for beta in (32.0, 1.0)]
        low, high = max(math.floor(turn[0]), 0), min(math.ceil(turn[1]), rot - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
        f = f / factor * ramp + f * (1.0 - ramp)
    return f, (0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0)


def rotate(x, positions, f, amplitude, layout):
    """Rows [tokens][heads][128] rotated by their positions, in 32 bits."""
    half = f.numel()
    angle = torch.remainder(positions.double()[:, None] * f, 2.0 * math.pi)
    cos = (torch.cos(angle) * amplitude).float()[:, None]
    sin = (torch.sin(angle) * amplitude).float()[:, None]
    x = x.float()
    if layout == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        parts = [a * cos - b * sin, b * cos + a * sin]
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        parts = [torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)]
    return torch.cat(parts + [x[..., 2 * half:]], dim=-1)


ROPE = {"rot": 128, "theta": 1e6, "scaling": "plain", "factor": 1.0, "layout": "half"}


def plain_rope(st):
    c = st["case"]
    f, amp = frequencies(c["rot"], c["theta"], c["scaling"], c["factor"])
    x = rotate(st["qkv"][:, : c["q"] + c["kv"]], st["positions"], f, amp, c["layout"]).half()
    return x[:, : c["q"]], x[:, c["q"]:]


def token_places(st, first):
    """Sequence, position and page of every row of the call."""
    t = torch.arange(st["tokens"], device=DEV)
    seq = torch.searchsorted(st["cu"][1:].long(), t, right=True)
    pos = first[seq].long() + t - st["cu"][seq].long()
    return seq, pos, st["table"][seq, pos // BS].long()


def write_rows(code, scale, x, page, row, starts, start_row):
    """Code the rows x [tokens][heads][128] (binary16) into (page, row); `starts` are the rows of
    the call that come first in their block, at rows `start_row` of it."""
    heads = x.shape[1]
    seen = torch.zeros(scale.shape, device=DEV)
    seen.index_reduce_(0, page, x.float().abs().amax(-1), "amax")
    at = page[starts]
    fresh = block_scale(seen[at])
    begun = (start_row == 0)[:, None]
    old = torch.where(begun, fresh, scale[at])
    new = torch.maximum(old, fresh)
    before = torch.arange(BS, device=DEV)[None, :] < start_row[:, None]
    held = code[at].float()
    recoded = held * (old / new)[:, :, None, None]
    code[at] = torch.where(before[:, None, :, None], recoded, held).to(F8)
    scale[at] = new
    s = scale[page]
    top = torch.where(s == 256.0, 240.0, 448.0)[..., None]
    y = (x.float() / s[..., None]).clamp(-top, top).to(F8)
    code.view(-1, BS, D)[(page[:, None] * heads + torch.arange(heads, device=DEV)),
                         row[:, None]] = y


def plain_append(st):
    c = st["case"]
    kv, nq = c["kv"], c["q"]
    seq, pos, page = token_places(st, st["lens"])
    x = st["qkv"]
    q, k, v = x[:, :nq], x[:, nq:nq + kv], x[:, nq + kv:].half()
    if c["rope"]:
        f, amp = frequencies(ROPE["rot"], ROPE["theta"], ROPE["scaling"], ROPE["factor"])
        k = rotate(k, pos, f, amp, ROPE["layout"])
        q = rotate(q, pos, f, amp, ROPE["layout"]) if nq else q
    if nq:
        st["q_out"].copy_(q.half())
    row = pos % BS
    starts = torch.nonzero((row == 0) | (pos == st["lens"][seq])).flatten()
    write_rows(st["k_code"], st["k_scale"], k.half(), page, row, starts, row[starts])
    write_rows(st["v_code"], st["v_scale"], v, page, row, starts, row[starts])
    st["new_lens"].copy_(st["lens"] + (st["cu"][1:] - st["cu"][:-1]))
    done = page[row == BS - 1]
    held = st["k_code"][done].float() * st["k_scale"][done][:, :, None, None]
    if c["rep"] == "max":
        st["reps"][done] = held.amax(2, keepdim=True).half()
    elif c["rep"] == "quest":
        st["reps"][done] = torch.stack([held.amin(2), held.amax(2)], dim=2).half()
    elif c["rep"] == "mean":
        st["reps"][done] = (held.double().sum(2, keepdim=True) / BS).float()
    else:
        st["reps"][done] = held[:, :, ::32].half()
    return append_outputs(st)


def append_outputs(st):
    names = ["k_code", "k_scale", "v_code", "v_scale", "new_lens", "reps"]
    return {n: st[n] for n in names + (["q_out"] if st["case"]["q"] else [])}


def plain_read(st):
    _, pos, page = token_places(st, st["first"])
    row = pos % BS
    k = st["k_code"][page, :, row].float() * st["k_scale"][page][..., None]
    v = st["v_code"][page, :, row].float() * st["v_scale"][page][..., None]
    return k.half(), v.half()


def attended(st):
    """Block lists [B][units][blocks] with what each position holds (and whether it does), and the
    selection that the step writes."""
    c = st["case"]
    lens = st["lens"].long()
    nb = (lens + BS - 1) // BS
    every = torch.arange(st["table"].shape[1], device=DEV)
    if c["how"] == "dense":
        return every[None, None], (every < nb[:, None])[:, None], None, None
    c0 = torch.minimum(torch.full_like(nb, c["initial"]), nb)
    c1 = torch.maximum(c0, nb - c["local"])
    if c["how"] == "sparse":
        sel, cnt = st["sel"].long(), st["cnt"]
    else:
        sel, cnt = select(st, c0, c1, every)
    k = c["top_k"]
    units = sel.shape[1]
    ends = torch.arange(c["local"], device=DEV)
    first = torch.arange(c["initial"], device=DEV)
    b = lens.shape[0]
    ids = torch.cat([first.expand(b, units, -1), sel,
                     (c1[:, None] + ends)[:, None].expand(b, units, -1)], dim=-1)
    holds = torch.cat([(first < c0[:, None])[:, None].expand(b, units, -1),
                       torch.arange(k, device=DEV) < cnt[..., None],
                       (c1[:, None] + ends < nb[:, None])[:, None].expand(b, units, -1)], dim=-1)
    return ids, holds, sel, cnt


def select(st, c0, c1, every):
    """The best top_k context blocks of each unit by the bound of their least and largest keys."""
    c = st["case"]
    b, kv = st["lens"].shape[0], c["kv"]
    q = st["q"].double().reshape(b, kv, -1, D)
    reps = st["reps"][st["table"].long()].double()  # [B][blocks][heads][2][128]
    score = torch.einsum("bhd,bjhd->bhj", q.clamp(max=0.0).sum(2), reps[:, :, :, 0])
    score += torch.einsum("bhd,bjhd->bhj", q.clamp(min=0.0).sum(2), reps[:, :, :, 1])
    if c["mode"] == "shared":
        score = score.sum(1, keepdim=True)
    context = (every >= c0[:, None]) & (every < c1[:, None])
    score = score.masked_fill(~context[:, None], -math.inf)
    k = c["top_k"]
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :k]
    cnt = (c1 - c0).clamp(max=k)[:, None].expand(-1, score.shape[1])
    rank = torch.arange(order.shape[-1], device=DEV)
    order = torch.where(rank < cnt[..., None], order, torch.full_like(order, 1 << 40))
    order = torch.sort(order, dim=-1).values
    sel = torch.zeros(b, score.shape[1], k, dtype=torch.int64, device=DEV)
    sel[..., : order.shape[-1]] = torch.where(order < 1 << 40, order, torch.zeros_like(order))
    return sel, cnt.to(torch.int32)


def plain_attend(st):
    c = st["case"]
    b, kv = st["lens"].shape[0], c["kv"]
    ids, holds, sel, cnt = attended(st)
    ids, holds = ids.expand(b, kv, -1), holds.expand(b, kv, -1)
    page = torch.gather(st["table"].long()[:, None].expand(b, kv, -1), 2,
                        ids.clamp(max=st["table"].shape[1] - 1))
    head = torch.arange(kv, device=DEV)[None, :, None]
    k = st["k_code"][page, head].float() * st["k_scale"][page, head][..., None, None]
    token = ids[..., None] * BS + torch.arange(BS, device=DEV)
    live = holds[..., None] & (token < st["lens"].long()[:, None, None, None])
    q = st["q"].float().reshape(b, kv, -1, D)
    s = torch.matmul(q, k.flatten(2, 3).transpose(2, 3)) * D ** -0.5
    del k
    s = s.masked_fill(~live.flatten(2)[:, :, None], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    total = p.sum(-1, keepdim=True)
    v = st["v_code"][page, head].float() * st["v_scale"][page, head][..., None, None]
    out = (torch.matmul(p, v.flatten(2, 3)) / total).reshape(b, -1, D)
    return (out, sel.to(torch.int32), cnt) if c["how"] == "step" else out


def run(st):
    if own:
        return run_own(st)
    return {"rope": plain_rope, "append": plain_append, "read": plain_read,
            "attend": plain_attend}[st["case"]["op"]](st)


# ---- the framework's calls --------------------------------------------------------------
def handles(st):
    """The structs and the workspace that a program keeps beside its buffers."""
    if "handles" in st:
        return st["handles"]
    import block_sparse_long_quest_gb300 as kt
    c = st["case"]
    h = {"kt": kt}
    if c["op"] == "rope" or c.get("rope"):
        r = c if c["op"] == "rope" else ROPE
        scaling = {"plain": kt.KT_ROPE_PLAIN, "linear": kt.KT_ROPE_LINEAR, "ntk": kt.KT_ROPE_NTK,
                   "yarn": kt.KT_ROPE_YARN}[r["scaling"]]
        h["rope"] = kt.rope(r["rot"], theta=r["theta"], scaling=scaling, factor=r["factor"],
                            original_len=8192,
                            layout=kt.KT_ROPE_HALF if r["layout"] == "half" else kt.KT_ROPE_PAIRS)
    if c["op"] != "rope":
        h["kv"] = kt.paged_kv_f8(st["k_code"], st["k_scale"], st["v_code"], st["v_scale"],
                                 st["table"], st["lens"])
    if c["op"] == "append":
        rep = {"max": kt.KT_REP_MAX, "mean": kt.KT_REP_MEAN, "quest": kt.KT_REP_QUEST,
               "fix": kt.KT_REP_FIX}[c["rep"]]
        h["params"] = kt.sparse_params(c["q"] or c["kv"], 1, 16, 16, rep, kt.KT_HEAD_SHARED)
        h["ws"] = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, h["kv"], h["params"])
    if c["op"] == "read":
        h["params"] = kt.sparse_params(c["kv"], 1, 16, 16, kt.KT_REP_QUEST, kt.KT_HEAD_SHARED)
        h["ws"] = kt.workspace_f8(kt.KT_OP_DENSE_ATTN, h["kv"], h["params"])
    if c["op"] == "attend":
        mode = kt.KT_HEAD_SHARED if c["mode"] == "shared" else kt.KT_HEAD_SEPARATE
        h["params"] = kt.sparse_params(c["q"], c["initial"], max(c["local"], 1),
                                       max(c["top_k"], 1), kt.KT_REP_QUEST, mode)
        op = {"dense": kt.KT_OP_DENSE_ATTN, "sparse": kt.KT_OP_SPARSE_ATTN,
              "step": kt.KT_OP_SPARSE_STEP}[c["how"]]
        h["ws"] = kt.workspace_f8(op, h["kv"], h["params"])
    st["handles"] = h
    return h


def run_own(st):
    c, h = st["case"], handles(st)
    kt, nq, kv = h["kt"], c["q"] if "q" in c else 0, c["kv"]
    if c["op"] == "rope":
        x = st["qkv"]
        kt.kt_apply_rope(h["rope"], st["positions"], x[:, :nq], st["q_out"], x[:, nq:nq + kv],
                         st["k_out"])
        return st["q_out"], st["k_out"]
    if c["op"] == "append":
        x = st["qkv"]
        kt.kt_append_kv_f8(h["kv"], h["params"], x[:, nq:nq + kv], x[:, nq + kv:], h["ws"],
                           rope=h.get("rope"), q=x[:, :nq] if nq else None, q_out=st["q_out"],
                           cu_tokens=st["cu"], new_lens=st["new_lens"], reps_pool=st["reps"])
        return append_outputs(st)
    if c["op"] == "read":
        kt.kt_read_kv_f8(h["kv"], st["cu"], st["k_out"], st["v_out"], h["ws"], first=st["first"])
        return st["k_out"], st["v_out"]
    if c["how"] == "dense":
        kt.kt_dense_decode_attn_f8(st["q"], h["kv"], nq, D ** -0.5, st["out"], h["ws"])
        return st["out"]
    if c["how"] == "sparse":
        kt.kt_sparse_decode_attn_f8(st["q"], h["kv"], h["params"], st["sel"], st["cnt"], st["out"],
                                    h["ws"])
        return st["out"]
    kt.kt_sparse_decode_step_f8(st["q"], h["kv"], st["reps"], h["params"], st["sel"], st["cnt"],
                                st["out"], h["ws"])
    return st["out"], st["sel"], st["cnt"]


# ---- work -------------------------------------------------------------------------------
def work(case):
    c = case
    size = {"f16": 2, "bf16": 2, "f32": 4}.get(c.get("dtype"), 2)
    if c["op"] == "rope":
        n = c["tokens"] * (c["q"] + c["kv"])
        return {"bytes": n * D * (size + 2) + 4 * c["tokens"],
                "flops": n * c["rot"] * 3 + c["tokens"] * c["rot"] * 10}
    lens = _lengths(c["least"], c["most"], c["batch"])
    tokens = sum(lens)
    if c["op"] == "append":
        rows = {"max": 2, "mean": 4, "quest": 4, "fix": 8}[c["rep"]] * D
        byte = tokens * D * (c["q"] * (size + 2) + 2 * c["kv"] * (size + 1))
        byte += tokens / BS * c["kv"] * (rows + 8)
        rot = tokens * (c["q"] + c["kv"]) * D * 3 if c["rope"] else 0
        return {"bytes": byte, "flops": rot + tokens * c["kv"] * D * 4}
    if c["op"] == "read":
        return {"bytes": tokens * c["kv"] * 2 * D * 3, "flops": tokens * c["kv"] * 2 * D}
    reps = 0
    if c["how"] != "dense":
        ends = (c["initial"] + c["local"]) * BS
        tokens = sum(min(n, ends + c["top_k"] * BS) for n in lens)
        if c["how"] == "step":
            reps = sum(max(0, n - ends) // BS for n in lens) * c["kv"] * 2 * D * 2
    return {"bytes": tokens * c["kv"] * 2 * D + reps + c["batch"] * c["q"] * D * 6,
            "flops": tokens * c["q"] * D * 4 + reps}


# ---- the operators in 64 bits, written apart --------------------------------------------
def _angles_exact(rot, theta, scaling, factor):
    f = []
    for i in range(rot // 2):
        base = theta * factor ** (rot / (rot - 2)) if scaling == "ntk" else theta
        w = base ** (-2.0 * i / rot)
        if scaling == "linear":
            w /= factor
        if scaling == "yarn":
            edge = [rot / 2 * math.log(8192 / (2 * math.pi * b), base) for b in (32, 1)]
            lo, hi = max(0, math.floor(edge[0])), min(rot - 1, math.ceil(edge[1]))
            t = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
            w = (1 - t) * w + t * w / factor
        f.append(w)
    return torch.tensor(f, dtype=torch.float64, device=DEV), \
        1.0 + 0.1 * math.log(factor) if scaling == "yarn" else 1.0


def _rotate_exact(x, pos, f, amp, layout):
    n = f.numel()
    turn = torch.polar(torch.full((pos.numel(), n), amp, dtype=torch.float64, device=DEV),
                       pos.double()[:, None] * f)[:, None]
    x = x.double().clone()
    at = torch.arange(n, device=DEV)
    re, im = (at, at + n) if layout == "half" else (2 * at, 2 * at + 1)
    z = torch.complex(x[..., re], x[..., im]) * turn
    x[..., re], x[..., im] = z.real, z.imag
    return x


def _code_exact(v):
    """The nearest e4m3 value (ties to even) of 64-bit values within its range."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -9))).clamp(min=-6)
    e = torch.where(v.abs() >= torch.exp2(e + 1), e + 1, e)
    step = torch.exp2(e - 3)
    return torch.round(v / step) * step


def _scale_exact(a):
    e = -15
    while e < 8 and a > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def _append_side_exact(code, scale, rows, st, b, first, last, n0, lo):
    """Rows `rows` (tokens n0 .. of sequence b, from row lo of the call) into blocks first..last."""
    heads = code.shape[1]
    for j in range(first, last):
        page = int(st["table_cpu"][b, j])
        a, z = max(n0, j * BS), min(n0 + rows.shape[0], (j + 1) * BS)
        new = rows[a - n0:z - n0]
        most = new.abs().amax(dim=(0, 2)).tolist()
        r0 = a - j * BS
        s = [_scale_exact(m) for m in most]
        if r0:
            had = scale[page].tolist()
            s = [max(x, y) for x, y in zip(s, had)]
            for h in range(heads):
                if s[h] > had[h]:
                    code[page, h, :r0] = _code_exact(code[page, h, :r0] * (had[h] / s[h]))
        sc = torch.tensor(s, dtype=torch.float64, device=DEV)
        scale[page] = sc
        top = torch.tensor([240.0 if x == 256.0 else 448.0 for x in s], dtype=torch.float64,
                           device=DEV)[:, None]
        y = torch.minimum(torch.maximum(_code_exact(new / sc[:, None]), -top), top)
        code[page, :, r0:r0 + z - a] = y.transpose(0, 1)


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    if c["op"] == "rope":
        f, amp = _angles_exact(c["rot"], c["theta"], c["scaling"], c["factor"])
        x = st["qkv"][:, : c["q"] + c["kv"]]
        y = _rotate_exact(x, st["positions"], f, amp, c["layout"])
        return y[:, : c["q"]], y[:, c["q"]:]
    kv = c["kv"]
    st["table_cpu"] = st["table"].cpu()
    lens = st["lens"].tolist()
    if c["op"] == "append":
        nq = c["q"]
        cu = st["cu"].tolist()
        f, amp = _angles_exact(128, 1e6, "plain", 1.0)
        kc, vc = st["k_code"].double(), st["v_code"].double()
        ks, vs = st["k_scale"].double(), st["v_scale"].double()
        reps = st["reps"].double()
        qs = []
        for b, n0 in enumerate(lens):
            x = st["qkv"][cu[b]:cu[b + 1]]
            pos = n0 + torch.arange(x.shape[0], device=DEV)
            q, k, v = x[:, :nq].double(), x[:, nq:nq + kv].double(), x[:, nq + kv:]
            if c["rope"]:
                q = _rotate_exact(q, pos, f, amp, "half")
                k = _rotate_exact(k, pos, f, amp, "half")
            qs.append(q)
            n1 = n0 + x.shape[0]
            blocks = (n0 // BS, -(-n1 // BS))
            _append_side_exact(kc, ks, k.half().double(), st, b, *blocks, n0, cu[b])
            _append_side_exact(vc, vs, v.half().double(), st, b, *blocks, n0, cu[b])
            for j in range(n0 // BS, n1 // BS):
                page = int(st["table_cpu"][b, j])
                held = kc[page] * ks[page][:, None, None]
                if c["rep"] == "mean":
                    reps[page, :, 0] = held.mean(1)
                elif c["rep"] == "fix":
                    reps[page] = held[:, [0, 32, 64, 96]]
                else:
                    reps[page, :, -1] = held.max(1).values
                    if c["rep"] == "quest":
                        reps[page, :, 0] = held.min(1).values
        out = {"k_code": kc, "k_scale": ks, "v_code": vc, "v_scale": vs, "reps": reps,
               "new_lens": torch.tensor([n + b - a for n, a, b in zip(lens, cu, cu[1:])],
                                        dtype=torch.int32)}
        if nq:
            out["q_out"] = torch.cat(qs)
        return out
    if c["op"] == "read":
        cu, first = st["cu"].tolist(), st["first"].tolist()
        outs = []
        for side in ("k", "v"):
            rows = []
            for b, n0 in enumerate(first):
                t = torch.arange(n0, n0 + cu[b + 1] - cu[b], device=DEV)
                page = st["table"][b].long()[torch.div(t, BS, rounding_mode="floor")]
                rows.append(st[side + "_code"][page, :, t % BS].double()
                            * st[side + "_scale"][page].double()[:, :, None])
            outs.append(torch.cat(rows))
        return tuple(outs)
    group = c["q"] // kv
    out = torch.zeros(len(lens), c["q"], D, dtype=torch.float64, device=DEV)
    units = 1 if c["mode"] == "shared" or c["how"] == "dense" else kv
    sels = torch.zeros(len(lens), units, max(c["top_k"], 1), dtype=torch.int32)
    cnts = torch.zeros(len(lens), units, dtype=torch.int32)
    for b, n in enumerate(lens):
        nb = -(-n // BS)
        c0 = 0 if c["how"] == "dense" else min(c["initial"], nb)
        c1 = 0 if c["how"] == "dense" else max(c0, nb - c["local"])
        chosen = [[]] * units
        if c["how"] == "sparse":
            chosen = [st["sel"][b, u, : int(st["cnt"][b, u])].tolist() for u in range(units)]
        if c["how"] == "step" and c1 > c0:
            page = st["table"][b, c0:c1].long()
            low, high = st["reps"][page, :, 0].double(), st["reps"][page, :, 1].double()
            w = st["q"][b].double().reshape(kv, group, 1, 1, D)
            bound = sum(torch.maximum(w[:, g, 0] * low.transpose(0, 1),
                                      w[:, g, 0] * high.transpose(0, 1)).sum(-1)
                        for g in range(group))
            bound = (bound.sum(0, keepdim=True) if units == 1 else bound).tolist()
            chosen = [sorted(sorted(range(c1 - c0), key=lambda j: (-s[j], j))[: c["top_k"]])
                      for s in bound]
            chosen = [[j + c0 for j in s] for s in chosen]
        for u, s in enumerate(chosen):
            sels[b, u, : len(s)] = torch.tensor(s, dtype=torch.int32)
            cnts[b, u] = len(s)
        for h in range(kv):
            blocks = list(range(c0)) + chosen[0 if units == 1 else h] + list(range(c1, nb))
            page = st["table"][b, torch.tensor(blocks, device=DEV)].long()
            live = torch.cat([torch.arange(j * BS, j * BS + BS) for j in blocks]).to(DEV) < n
            k = (st["k_code"][page, h].double() * st["k_scale"][page, h].double()[:, None, None])
            v = (st["v_code"][page, h].double() * st["v_scale"][page, h].double()[:, None, None])
            s = st["q"][b, h * group:(h + 1) * group].double() @ k.reshape(-1, D)[live].T
            out[b, h * group:(h + 1) * group] = \
                torch.softmax(s / math.sqrt(D), dim=-1) @ v.reshape(-1, D)[live]
    return (out, sels, cnts) if c["how"] == "step" else out
