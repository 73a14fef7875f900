"""Sequences that share pages of the paged caches: what is measured, and the plain forms.

* attend:  decode attention of a batch whose sequences share long prefixes, each shared prefix
           computed once for all of its sequences (kt_prefix_decode_attn over binary16 pools,
           kt_prefix_decode_attn_f8 over the 8-bit cache);
* fork:    the turnover of samples between two decode steps: the old copies are freed, sequences
           are forked into their slots, every sequence gets the page of its next token, and the
           forks' partial last pages are copied in all layers (kt_free_seqs, kt_fork_seqs,
           kt_reserve_pages, kt_copy_pages);
* compact: the pages in use move to the front of the pools (kt_compact_pages, kt_copy_pages).

A sequence b holds the pages table[b][: blocks[b]]; refs[p] counts the table entries that hold
page p, and a page is free where that is 0.  Free pages are taken lowest first.  Sequences of a
group are consecutive, and the first `prefix` blocks of all of them are the same pages.

`own` false: elementary torch operations in 32 bits.  `own` true: the framework's calls.
"""
import math

import torch

own = False

D = 128   # channels of a head
BS = 128  # tokens of a block
F8 = torch.float8_e4m3fn
DEV = "cuda"


# ---- cases ------------------------------------------------------------------------------
def listed():
    return [
        # four samples of one short prompt, just begun
        attend_case("attend-samples-4", groups=1, members=4, ragged=False, prefix=8, tail=200, q=32,
                    kv=8, cache="f16"),
        # 16 chats behind one 4K system prompt
        attend_case("attend-system-16", groups=1, members=16, ragged=False, prefix=32, tail=2000,
                    q=32, kv=8, cache="f16"),
        # 64 questions to one 32K document
        attend_case("attend-document-64", groups=1, members=64, ragged=False, prefix=256, tail=1024,
                    q=32, kv=8, cache="f16"),
        # a mixed batch: 8 groups of 9 to 1 sequences behind prefixes of 16K tokens to none
        attend_case("attend-groups-8", groups=8, members=9, ragged=True, prefix=128, tail=3000, q=28,
                    kv=4, cache="f16"),
        # 32 questions to one 128K document in the 8-bit cache
        attend_case("attend-f8-document-32", groups=1, members=32, ragged=False, prefix=1024,
                    tail=2048, q=32, kv=8, cache="f8"),
        # 5 groups of 12 to 1 sequences in the 8-bit cache, three heads a K/V head
        attend_case("attend-f8-groups-5", groups=5, members=12, ragged=True, prefix=200, tail=700,
                    q=24, kv=8, cache="f8"),
        # one prompt into four samples, one layer
        fork_case("fork-4", parents=1, children=4, most=1000, layers=1, kv=8, cache="f16",
                  spare=9),
        # best-of-6 of 8 prompts, 8 layers with their representatives
        fork_case("fork-48", parents=8, children=6, most=8000, layers=8, kv=4, cache="f16",
                  spare=200),
        # 16 long sequences of the 8-bit cache forked once each, most of a large pool free
        fork_case("fork-long-16", parents=16, children=1, most=131000, layers=1, kv=1, cache="f8",
                  spare=16000),
        # a small pool after a few sequences have left
        compact_case("compact-300", batch=6, most=6000, share=8, layers=1, kv=8, cache="f16",
                     spare=100),
        # many sequences that share prefixes, a third of the pool's pages free, two layers
        compact_case("compact-8k", batch=64, most=16000, share=20, layers=2, kv=4, cache="f16",
                     spare=1000),
        # the 8-bit cache of 16 sequences of up to 64K tokens
        compact_case("compact-f8-8k", batch=16, most=65536, share=40, layers=1, kv=8, cache="f8",
                     spare=500),
    ]


def attend_case(name, **kw):
    return dict(name=name, op="attend", **kw)


def fork_case(name, **kw):
    return dict(name=name, op="fork", **kw)


def compact_case(name, **kw):
    return dict(name=name, op="compact", **kw)


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "fork", "compact"])
    kv, cache = rng.choice([1, 2, 4, 8]), rng.choice(["f16", "f8"])
    if op == "attend":
        groups = rng.choice([1, 1, 2, 3, 8])
        members = _spread(rng, 1, 32 // groups)
        blocks = _spread(rng, 1, (256 if cache == "f16" else 512) // groups)
        case = attend_case("", groups=groups, members=members, ragged=rng.random() < 0.5,
                           prefix=blocks, tail=_spread(rng, 1, 65536 // (groups * members)),
                           q=kv * rng.choice([1, 2, 3, 4, 5, 7, 8]), kv=kv, cache=cache)
    elif op == "fork":
        parents = rng.choice([1, 2, 5, 16])
        case = fork_case("", parents=parents, children=_spread(rng, 1, 48 // parents),
                         most=_spread(rng, 2, 131000 // parents), layers=rng.choice([1, 2, 4]),
                         kv=kv, cache=cache, spare=_spread(rng, 1, 4000 // kv))
    else:
        batch = rng.choice([1, 3, 16, 64])
        case = compact_case("", batch=batch, most=_spread(rng, 2, 320000 // batch),
                            share=rng.choice([0, 1, 5, 20]), layers=rng.choice([1, 2]), kv=kv,
                            cache=cache, spare=_spread(rng, 1, 800))
    del case["name"]
    return case


# ---- inputs -----------------------------------------------------------------------------
def _down(most, least, n):
    """`n` whole numbers from `most` down to `least`: the same for every seed."""
    return [most - (most - least) * i // max(1, n - 1) for i in range(n)]


def _cache(gen, pages, kv, cache):
    """A filled K or V pool: binary16, or e4m3 codes and a scale per (page, head), a power of two."""
    if cache == "f16":
        pool = torch.empty(pages, kv, BS, D, dtype=torch.float16, device=DEV)
        return pool.normal_(generator=gen), None
    code = torch.empty(pages, kv, BS, D, dtype=F8, device=DEV)
    for lo in range(0, pages, 512):
        n = min(512, pages - lo)
        code[lo:lo + n] = (48.0 * torch.randn(n, kv, BS, D, generator=gen, device=DEV)).to(F8)
    scale = torch.exp2(torch.randint(-7, -3, (pages, kv), generator=gen, device=DEV).float())
    return code, scale


def group_shape(c):
    """Members and prefix blocks of every group, and the tokens of every sequence behind its
    prefix."""
    n = c["groups"]
    members = _down(c["members"], 1, n) if c["ragged"] else [c["members"]] * n
    prefix = _down(c["prefix"], 0, n) if n > 1 else [c["prefix"]]
    tails = _down(c["tail"], 1, sum(members))
    tails = tails[::2] + tails[1::2][::-1]  # long and short ones in every group
    return members, prefix, tails


def prepare_attend(c, st, gen):
    members, prefix, tails = group_shape(c)
    batch = len(tails)
    lens = [128 * p + t for p, t in zip([p for m, p in zip(members, prefix) for _ in range(m)], tails)]
    mine = [-(-t // BS) for t in tails]
    pages = sum(prefix) + sum(mine) + 5
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32).tolist()
    table = torch.zeros(batch, max(-(-n // BS) for n in lens), dtype=torch.int32)
    at = b = 0
    for m, p in zip(members, prefix):
        shared = order[at:at + p]
        at += p
        for _ in range(m):
            table[b, :p + mine[b]] = torch.tensor(shared + order[at:at + mine[b]], dtype=torch.int32)
            at += mine[b]
            b += 1
    st["table"], st["lens"] = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    cu = torch.zeros(c["groups"] + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(members).cumsum(0)
    st["cu"], st["prefix"] = cu.to(DEV), torch.tensor(prefix, dtype=torch.int32, device=DEV)
    st["k"], st["k_scale"] = _cache(gen, pages, c["kv"], c["cache"])
    st["v"], st["v_scale"] = _cache(gen, pages, c["kv"], c["cache"])
    st["q"] = torch.randn(batch, c["q"], D, generator=gen, device=DEV).half()
    st["out"] = torch.zeros(batch, c["q"], D, dtype=torch.float32, device=DEV)
    # how far a padded form of the batch reaches (a server knows that from its own lengths)
    st["most"] = (max(members), max(prefix), max(mine))
    return st


def _pools(c, gen, pages):
    """The pools of every layer: K, V, their scales in the 8-bit cache, and representatives."""
    pools = {}
    for layer in range(c["layers"]):
        for side in ("k", "v"):
            pools["%s%d" % (side, layer)], scale = _cache(gen, pages, c["kv"], c["cache"])
            if scale is not None:
                pools["%s_scale%d" % (side, layer)] = scale
        reps = torch.empty(pages, c["kv"], 2, D, dtype=torch.float16, device=DEV)
        pools["reps%d" % layer] = reps.normal_(generator=gen)
    return pools


def prepare_fork(c, st, gen):
    """Parents in the first slots, and in the others copies that an earlier fork has left there."""
    cpu = torch.Generator()
    cpu.manual_seed(int(torch.randint(0, 1 << 30, (1,), generator=gen, device=DEV)))
    np_, nc = c["parents"], c["parents"] * c["children"]
    lens = torch.randint((c["most"] + 1) // 2, c["most"] + 1, (np_,), generator=cpu).tolist()
    lens[0] = c["most"]
    blocks = [-(-n // BS) for n in lens]
    width = -(-(c["most"] + 1) // BS) + 1
    old = [1 + n // 2 for n in blocks]  # blocks of the old copies: the last one is their own
    pages = np_ * -(-c["most"] // BS) + nc + nc + c["spare"]
    order = torch.randperm(pages, generator=cpu).tolist()
    table = torch.zeros(np_ + nc, width, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    at = 0
    src = []
    for i, n in enumerate(blocks):
        table[i, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    for j in range(nc):
        i = j % np_
        src.append((i * 7 + 3) % np_)  # the new copies are of other parents than the old ones
        table[np_ + j, : old[i]] = table[i, : old[i]]
        table[np_ + j, old[i] - 1] = order[at]
        lens.append(old[i] * BS - 5)
        blocks.append(old[i])
        at += 1
    for row, n in zip(table, blocks):
        refs += torch.bincount(row[:n].long(), minlength=pages).to(torch.int32)
    st["table"], st["refs"] = table.to(DEV), refs.to(DEV)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    st["blocks"] = torch.tensor(blocks, dtype=torch.int32, device=DEV)
    st["src"] = torch.tensor(src, dtype=torch.int32, device=DEV)
    st["dst"] = torch.arange(np_, np_ + nc, dtype=torch.int32, device=DEV)
    st["moves"] = torch.zeros(nc, 2, dtype=torch.int32, device=DEV)
    st["num_moves"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    st["pools"] = _pools(c, gen, pages)
    return st


def prepare_compact(c, st, gen):
    """Sequences that share their first blocks in pairs, over a pool with free pages everywhere."""
    cpu = torch.Generator()
    cpu.manual_seed(int(torch.randint(0, 1 << 30, (1,), generator=gen, device=DEV)))
    lens = torch.randint((c["most"] + 1) // 2, c["most"] + 1, (c["batch"],), generator=cpu).tolist()
    blocks = [-(-n // BS) for n in lens]
    pages = c["batch"] * -(-c["most"] // BS) + c["spare"]
    order = torch.randperm(pages, generator=cpu)
    table = torch.zeros(c["batch"], -(-c["most"] // BS) + 2, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n].to(torch.int32)
        at += n
        if b % 2:
            k = min(c["share"], n, blocks[b - 1])
            table[b, :k] = table[b - 1, :k]
        refs += torch.bincount(table[b, :n].long(), minlength=pages).to(torch.int32)
    st["table"], st["refs"] = table.to(DEV), refs.to(DEV)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    st["blocks"] = torch.tensor(blocks, dtype=torch.int32, device=DEV)
    st["new_table"], st["new_refs"] = torch.zeros_like(st["table"]), torch.zeros_like(st["refs"])
    st["moves"] = torch.zeros(pages // 2, 2, dtype=torch.int32, device=DEV)
    st["num_moves"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    st["pools"] = _pools(c, gen, pages)
    return st


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    st = {"case": dict(case)}
    return {"attend": prepare_attend, "fork": prepare_fork,
            "compact": prepare_compact}[case["op"]](st["case"], st, gen)


# ---- plain forms ------------------------------------------------------------------------
def values(pool, scale, page):
    """Pages [n][blocks] of a pool as [n][heads][tokens][128] in 32 bits."""
    x = pool.view(torch.uint8)[page].view(F8).float() if scale is not None else pool[page].float()
    if scale is not None:
        x = x * scale[page][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def plain_attend(st):
    c = st["case"]
    kv, group = c["kv"], c["q"] // c["kv"]
    members, prefix, tail = st["most"]
    cu, lens = st["cu"].long(), st["lens"].long()
    table, batch = st["table"].long(), st["lens"].shape[0]
    every = torch.arange(batch, device=DEV)
    mine = torch.searchsorted(cu[1:], every, right=True)  # the group of every sequence
    place = every - cu[mine]
    q = st["q"].float().reshape(batch, kv, group, D) * D ** -0.5
    # scores against the shared prefixes, one product a group: [groups][kv][members * group][tokens]
    rows = (cu[:-1, None] + torch.arange(members, device=DEV)).clamp(max=batch - 1)
    qg = q[rows].transpose(1, 2).flatten(2, 3)
    page = table[cu[:-1], : max(prefix, 1)]
    token = torch.arange(page.shape[1] * BS, device=DEV)
    seen = token < BS * st["prefix"][:, None]
    sp = torch.matmul(qg, values(st["k"], st["k_scale"], page).transpose(2, 3))
    sp = sp.masked_fill(~seen[:, None, None], -math.inf)
    # scores against what each sequence has of its own
    start = st["prefix"].long()[mine]
    at = start[:, None] + torch.arange(tail, device=DEV)
    own_page = table.gather(1, at.clamp(max=table.shape[1] - 1))
    left = lens - BS * start
    live = torch.arange(tail * BS, device=DEV) < left[:, None]
    ss = torch.matmul(q, values(st["k"], st["k_scale"], own_page).transpose(2, 3))
    ss = ss.masked_fill(~live[:, None, None], -math.inf)
    # the two parts of every row under one maximum
    most_p = sp.amax(-1).reshape(c["groups"], kv, members, group)[mine, :, place]
    most = torch.maximum(most_p, ss.amax(-1))
    back = torch.zeros(c["groups"], members, kv, group, device=DEV)
    back[mine, place] = most
    sp = torch.exp(sp - back.transpose(1, 2).flatten(2, 3)[..., None])
    ss = torch.exp(ss - most[..., None])
    op = torch.matmul(sp, values(st["v"], st["v_scale"], page))
    op = op.reshape(c["groups"], kv, members, group, D)[mine, :, place]
    total = sp.sum(-1).reshape(c["groups"], kv, members, group)[mine, :, place] + ss.sum(-1)
    out = op + torch.matmul(ss, values(st["v"], st["v_scale"], own_page))
    return (out / total[..., None]).reshape(batch, c["q"], D)


def held(st, blocks):
    return torch.arange(st["table"].shape[1], device=DEV) < blocks[:, None]


def free_pages(refs, n):
    """The n lowest pages that nobody holds (all of them are there)."""
    return torch.argsort((refs > 0).to(torch.int8), stable=True)[:n]


def copy_pages(pools, moves, count):
    """Pages from -> to in all pools; rows of `moves` behind `count` are none."""
    source, to = moves[:int(count)].long().unbind(1)
    for x in pools.values():
        x = x.flatten(1).view(torch.uint8)
        x[to] = x[source]


def plain_fork(st):
    table, lens, blocks, refs = st["table"], st["lens"], st["blocks"], st["refs"]
    src, dst = st["src"].long(), st["dst"].long()
    # free the old copies
    gone = torch.where(held(st, blocks)[dst], table[dst].long(), refs.shape[0])
    refs -= torch.bincount(gone.flatten(), minlength=refs.shape[0] + 1)[:-1].to(torch.int32)
    # fork: whole blocks are shared, the partial last one becomes a page of the copy's own
    n = lens[src]
    whole, partial = (n // BS)[:, None], n % BS > 0
    shared = torch.arange(table.shape[1], device=DEV) < whole
    refs += torch.bincount(torch.where(shared, table[src].long(), refs.shape[0]).flatten(),
                           minlength=refs.shape[0] + 1)[:-1].to(torch.int32)
    rank = partial.cumsum(0) - 1
    new = free_pages(refs, dst.shape[0])[rank.clamp(min=0)].to(torch.int32)
    rows = torch.where(shared, table[src], table[dst])
    last = (n // BS).long()[:, None].clamp(max=table.shape[1] - 1)
    tail = table[src].gather(1, last)[:, 0]
    rows.scatter_(1, last, torch.where(partial[:, None], new[:, None], rows.gather(1, last)))
    table[dst] = rows
    lens[dst], blocks[dst] = n, (n + BS - 1) // BS
    taken = torch.where(partial, new.long(), refs.shape[0])
    refs += torch.bincount(taken, minlength=refs.shape[0] + 1)[:-1].to(torch.int32)
    slot = torch.where(partial, rank, dst.shape[0])
    moves = torch.cat([st["moves"], st["moves"][:1]])
    moves[slot] = torch.stack([tail, new], dim=1)
    st["moves"].copy_(moves[:-1])
    st["num_moves"].copy_(partial.sum()[None])
    # the page of every sequence's next token
    need = (lens + BS) // BS - blocks
    rank = need.cumsum(0) - 1
    new = free_pages(refs, lens.shape[0])[rank.clamp(min=0)].to(torch.int32)
    at = blocks.long()[:, None].clamp(max=table.shape[1] - 1)
    table.scatter_(1, at, torch.where(need[:, None] > 0, new[:, None], table.gather(1, at)))
    taken = torch.where(need > 0, new.long(), refs.shape[0])
    refs += torch.bincount(taken, minlength=refs.shape[0] + 1)[:-1].to(torch.int32)
    blocks += need
    copy_pages(st["pools"], st["moves"], st["num_moves"])
    return fork_outputs(st)


def fork_outputs(st):
    names = ["table", "lens", "blocks", "refs", "moves", "num_moves"]
    return {**{n: st[n] for n in names}, **st["pools"]}


def plain_compact(st):
    refs, pages = st["refs"], st["refs"].shape[0]
    page = torch.arange(pages, device=DEV)
    used = refs > 0
    total = used.sum()
    # pages that move, lowest first, into the free ones below, lowest first
    source = torch.nonzero(used & (page >= total)).flatten()
    hole = torch.nonzero(~used & (page < total)).flatten()
    count = source.shape[0]
    st["moves"][:count] = torch.stack([source, hole], dim=1).to(torch.int32)
    st["num_moves"].fill_(count)
    remap = page.clone()
    remap[source] = hole
    entries = remap[st["table"].long()].to(torch.int32)
    st["new_table"].copy_(torch.where(held(st, st["blocks"]), entries, st["new_table"]))
    st["new_refs"].copy_(torch.where(used & (page < total), refs, 0))
    st["new_refs"][hole] = refs[source]
    copy_pages(st["pools"], st["moves"], st["num_moves"])
    return compact_outputs(st)


def compact_outputs(st):
    names = ["new_table", "new_refs", "moves", "num_moves"]
    return {**{n: st[n] for n in names}, **st["pools"]}


def run(st):
    if own:
        return run_own(st)
    return {"attend": plain_attend, "fork": plain_fork,
            "compact": plain_compact}[st["case"]["op"]](st)


# ---- the framework's calls --------------------------------------------------------------
def handles(st):
    """The structs and the workspace that a program keeps beside its buffers."""
    if "handles" in st:
        return st["handles"]
    import block_sparse_long_quest_gb300 as kt
    c = st["case"]
    h = {"kt": kt}
    if c["op"] == "attend":
        p = kt.sparse_params(c["q"], 0, 1, 1, kt.KT_REP_QUEST, kt.KT_HEAD_SHARED)
        if c["cache"] == "f16":
            h["kv"] = kt.paged_kv(st["k"], st["v"], st["table"], st["lens"])
            h["ws"] = kt.workspace(kt.KT_OP_PREFIX_ATTN, h["kv"], p)
        else:
            h["kv"] = kt.paged_kv_f8(st["k"], st["k_scale"], st["v"], st["v_scale"], st["table"],
                                     st["lens"])
            h["ws"] = kt.workspace_f8(kt.KT_OP_PREFIX_ATTN, h["kv"], p)
        h["groups"] = kt.prefix_groups(st["cu"], st["prefix"])
    else:
        h["map"] = kt.page_map(st["table"], st["lens"], st["blocks"], st["refs"])
        h["ws"] = kt.page_workspace(h["map"])
        h["pools"] = kt.page_pools(list(st["pools"].values()))
    st["handles"] = h
    return h


def run_own(st):
    c, h = st["case"], handles(st)
    kt = h["kt"]
    if c["op"] == "attend":
        call = kt.kt_prefix_decode_attn if c["cache"] == "f16" else kt.kt_prefix_decode_attn_f8
        call(st["q"], h["kv"], h["groups"], c["q"], D ** -0.5, st["out"], h["ws"])
        return st["out"]
    if c["op"] == "fork":
        kt.kt_free_seqs(h["map"], st["dst"], h["ws"])
        kt.kt_fork_seqs(h["map"], st["src"], st["dst"], st["moves"], st["num_moves"], h["ws"])
        kt.kt_reserve_pages(h["map"], h["ws"])
        kt.kt_copy_pages(h["pools"], st["moves"], st["num_moves"], h["ws"])
        return fork_outputs(st)
    kt.kt_compact_pages(h["map"], st["moves"], st["num_moves"], h["ws"], new_table=st["new_table"],
                        new_refs=st["new_refs"])
    kt.kt_copy_pages(h["pools"], st["moves"], st["num_moves"], h["ws"])
    return compact_outputs(st)


# ---- work -------------------------------------------------------------------------------
def page_bytes(c):
    """A page in all pools of all layers."""
    one = 2 * BS * D * 2 if c["cache"] == "f16" else 2 * (BS * D + 4)
    return c["layers"] * c["kv"] * (one + 2 * D * 2)


def work(case):
    c = case
    if c["op"] == "attend":
        members, prefix, tails = group_shape(c)
        tokens = BS * sum(prefix) + sum(tails)
        pairs = BS * sum(m * p for m, p in zip(members, prefix)) + sum(tails)
        size = 2 if c["cache"] == "f16" else 1
        return {"bytes": tokens * c["kv"] * 2 * D * size + len(tails) * c["q"] * D * 6,
                "flops": pairs * c["q"] * D * 4}
    if c["op"] == "fork":
        n = c["parents"] * c["children"]
        entries = n * 0.75 * c["most"] / BS
        pages = c["parents"] * c["most"] / BS + 2 * n + c["spare"]
        return {"bytes": 2 * n * page_bytes(c) + 4 * (3 * entries + pages), "flops": 0}
    used = c["batch"] * 0.75 * c["most"] / BS
    pages = c["batch"] * c["most"] / BS + c["spare"]
    moves = used * (pages - used) / pages  # the used ones of the last pages, as many as are free
    return {"bytes": 2 * moves * page_bytes(c) + 4 * (2 * used + 2 * pages), "flops": 0}


# ---- the operators in 64 bits, written apart --------------------------------------------
def exact_attend(c, st):
    _, prefix, _ = group_shape(c)
    table, lens = st["table"].tolist(), st["lens"].tolist()
    group = c["q"] // c["kv"]

    def tokens(side, ids, h):
        x = st[side][torch.tensor(ids, device=DEV), h] if c["cache"] == "f16" else \
            st[side].view(torch.uint8)[torch.tensor(ids, device=DEV), h].view(F8)
        x = x.double()
        if c["cache"] == "f8":
            x = x * st[side + "_scale"][torch.tensor(ids, device=DEV), h].double()[:, None, None]
        return x.reshape(-1, D)

    out = torch.zeros(len(lens), c["q"], D, dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        ids = table[b][: -(-n // BS)]
        for h in range(c["kv"]):
            rows = slice(h * group, (h + 1) * group)
            s = st["q"][b, rows].double() @ tokens("k", ids, h)[:n].T / math.sqrt(D)
            out[b, rows] = torch.softmax(s, dim=-1) @ tokens("v", ids, h)[:n]
    return out


def _move_exact(st, moves):
    """The pools after the moves (from, to): values are moved as they are, so in their own types."""
    pools = {}
    for name, x in st["pools"].items():
        y = x.clone()
        a, b = y.view(torch.uint8).flatten(1), x.view(torch.uint8).flatten(1)
        for source, to in moves:
            a[to] = b[source]
        pools[name] = y
    return pools


def exact_fork(c, st):
    table, lens = st["table"].tolist(), st["lens"].tolist()
    blocks, refs = st["blocks"].tolist(), st["refs"].tolist()
    src, dst = st["src"].tolist(), st["dst"].tolist()
    for b in dst:
        for p in table[b][: blocks[b]]:
            refs[p] -= 1
        blocks[b] = lens[b] = 0
    free = iter([p for p, r in enumerate(refs) if r == 0])
    moves = []
    for a, b in zip(src, dst):
        lens[b], blocks[b] = lens[a], -(-lens[a] // BS)
        for j in range(blocks[b]):
            p = table[a][j]
            if (j + 1) * BS > lens[a]:
                p = next(free)
                moves.append((table[a][j], p))
            table[b][j] = p
            refs[p] += 1
    for b, n in enumerate(lens):
        if blocks[b] * BS < n + 1:
            p = next(free)
            table[b][blocks[b]] = p
            blocks[b] += 1
            refs[p] += 1
    whole = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    listed_moves = moves + [(0, 0)] * (len(dst) - len(moves))
    return {"table": whole(table), "lens": whole(lens), "blocks": whole(blocks),
            "refs": whole(refs), "moves": whole(listed_moves), "num_moves": whole([len(moves)]),
            **_move_exact(st, moves)}


def exact_compact(c, st):
    table, blocks, refs = st["table"].tolist(), st["blocks"].tolist(), st["refs"].tolist()
    total = sum(r > 0 for r in refs)
    holes = [p for p in range(total) if refs[p] == 0]
    moves = list(zip([p for p in range(total, len(refs)) if refs[p] > 0], holes))
    to = dict(moves)
    new_refs, new_table = list(refs), [[0] * len(row) for row in table]
    for a, b in moves:
        new_refs[b], new_refs[a] = refs[a], 0
    for row, n, old in zip(new_table, blocks, table):
        row[:n] = [to.get(p, p) for p in old[:n]]
    whole = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    listed_moves = moves + [(0, 0)] * (len(refs) // 2 - len(moves))
    return {"new_table": whole(new_table), "new_refs": whole(new_refs),
            "moves": whole(listed_moves).reshape(-1, 2), "num_moves": whole([len(moves)]),
            **_move_exact(st, moves)}


def exact(case, seed):
    st = prepare(case, seed)
    return {"attend": exact_attend, "fork": exact_fork,
            "compact": exact_compact}[case["op"]](dict(case), st)
