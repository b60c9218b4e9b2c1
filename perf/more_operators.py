"""Page maps, ragged appends and the 8-bit paged cache: cases, their plain form,
and what they compute in 64 bits.

Five operators over the block table that the library's decode already reads:

  map     give rows pages for their new tokens from a free list, enter them in
          the block table, and list every new token's slot and position;
  slots   copy packed K and V of new tokens to their slots in the fp16 pages;
  append  quantise a ragged run of new K/V tokens per row (or one token per row)
          into the pages of an 8-bit cache, then read the blocks they touched
          back as fp16;
  read    read whole rows of the 8-bit cache back into packed fp16 K and V;
  decode  attention of one query token per row straight over the 8-bit cache,
          over the whole row or over a sliding window with sinks.

The map.  Row i has N tokens in ceil(N / P) pages and gets n more; the pages it
lacks are taken in row order from the top (the end) of the free list.  A row is
served when it needs no page or the rows up to and including it need no more
than there are free; one that is not gets -1 in place of its pages and slots,
and keeps its length.  slot = page * P + position % P; entries behind the last
token have slot -1, and a token without a slot position 0.

The 8-bit format.  SB = min(P, 16) neighbouring tokens of one head and side (K
or V) share a scale 2^e, kept as fp32; a code c stands for c * 2^e, where c is an
int8 ("int8": Q = 127, e in -24 .. 9) or a float of 1 + 4 + 3 bits ("e4m3":
Q = 448, e in -15 .. 7).  Values beyond Q * 2^(greatest e) are taken as it.  e is
the least in its range with max |x| <= Q * 2^e, c the code nearest to x / 2^e
(ties to even).  A block that holds earlier tokens keeps its e unless the new
ones need a greater one: then the earlier codes c * 2^e are rounded alike.

A cache is uint8 [num_pages][Hkv][bytes]; a page of one head holds blocks of
TB = min(P, 64) tokens, each of three parts:
  K codes  [token][dim]; with d = 128 the two 64-byte halves of tokens 2, 3 of every four swapped
  V codes  [token / SB][dim / 4][token % SB / 4][dim % 4][token % 4]
  scales   [token / SB][K | V] fp32, padded to a multiple of 16 bytes
"""
import math
import random

import torch

own = False

TOKEN_BUDGET = 1 << 21  # tokens of the largest cases' pools
LEAST = {"int8": -24, "e4m3": -15}
MOST = {"int8": 9, "e4m3": 7}
Q = {"int8": 127.0, "e4m3": 448.0}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a serving step: every running row gets a place for the token it produces
        dict(name="map_step_b64", op="map", B=64, P=16, lo=128, hi=65536, new_lo=1, new_hi=1, spare=64, pad=0, lens_seed=1),
        # prompts of all lengths enter beside running rows, in a batch padded to a captured size
        dict(name="map_prompts_b256", op="map", B=256, P=16, lo=0, hi=2048, new_lo=1, new_hi=8192, spare=1000, pad=4096,
             lens_seed=2),
        # a step of one token per row into the fp16 pages
        dict(name="slots_step_b64", op="slots", B=64, Hkv=8, d=128, P=16, lo=128, hi=8192, new_lo=1, new_hi=1, stray=0,
             pad=0, lens_seed=3),
        # a batch of prompts into the fp16 pages, K and V slices of one fused projection
        dict(name="slots_prompts_b8", op="slots", B=8, Hkv=8, d=128, P=16, lo=0, hi=999, new_lo=512, new_hi=8192, stray=512,
             pad=4096, lens_seed=4),
        # a serving step: every running row stores the token it just produced in 8 bits
        dict(name="append_step_b64_int8", op="append", fmt="int8", B=64, Hq=64, Hkv=8, d=128, P=16, lens="uniform", lo=128,
             hi=4096, new_lo=1, new_hi=1, pad=0, lens_seed=5),
        # a batch of prompts behind what the rows already hold
        dict(name="append_prompts_b8_e4m3", op="append", fmt="e4m3", B=8, Hq=32, Hkv=8, d=128, P=16, lens="uniform", lo=0,
             hi=999, new_lo=512, new_hi=8192, pad=4096, lens_seed=6),
        # one short conversation read back, as a prefix that another model path reuses
        dict(name="read_b1_1k_e4m3", op="read", fmt="e4m3", B=1, Hq=8, Hkv=2, d=128, P=16, lens="uniform", lo=1024, hi=1024,
             lens_seed=7),
        # a mixed batch of short and long rows read back whole
        dict(name="read_b8_bimodal_int8", op="read", fmt="int8", B=8, Hq=32, Hkv=8, d=128, P=16, lens="bimodal", lo=512,
             hi=32768, lens_seed=8),
        # the smallest decode step: one short row
        dict(name="decode_b1_1k_int8", op="decode", fmt="int8", B=1, Hq=8, Hkv=2, d=128, P=16, lens="uniform", lo=1024,
             hi=1024, window=-1, sinks=0, lens_seed=9),
        # short chats beside long documents in one batch
        dict(name="decode_b8_bimodal_e4m3", op="decode", fmt="e4m3", B=8, Hq=32, Hkv=8, d=128, P=16, lens="bimodal", lo=512,
             hi=32768, window=-1, sinks=0, lens_seed=10),
        # a large mixed batch at long context, eight query heads per KV head
        dict(name="decode_b64_uniform_int8", op="decode", fmt="int8", B=64, Hq=64, Hkv=8, d=128, P=16, lens="uniform",
             lo=128, hi=65536, window=-1, sinks=0, lens_seed=11),
        # odd sizes in a window: five heads per KV head, d = 64, an empty row among the rest
        dict(name="decode_window_b5_odd_e4m3", op="decode", fmt="e4m3", B=5, Hq=15, Hkv=3, d=64, P=32, lens="uniform", lo=0,
             hi=20000, window=4097, sinks=5, lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["map", "slots", "append", "append", "read", "decode", "decode"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    P = rng.choice([8, 16, 32, 64, 128, 256])
    seed = rng.randrange(1 << 30)
    if op == "map":
        B = _log_int(rng, 1, 4096)
        one = rng.random() < 0.4
        new_hi = 1 if one else _log_int(rng, 1, max(1, min(32768, (1 << 20) // B)))
        return dict(op=op, B=B, P=P, lo=rng.choice([0, 0, 1, 100]), hi=_log_int(rng, 100, 8192),
                    new_lo=1 if one else rng.choice([0, 1, new_hi // 2]), new_hi=new_hi,
                    spare=rng.choice([0, 1, 100, -1]), pad=rng.choice([0, 0, 7, 1000]), lens_seed=seed)
    B = _log_int(rng, 1, 64)
    # tokens a row may have so that the batch stays below the largest case
    cap = min(65536, (TOKEN_BUDGET // 8) // B)
    hi = _log_int(rng, 1, cap)
    lo = min(rng.choice([0, 1, hi, hi // 2, hi // 16]), hi)
    if op == "read" or op == "decode":
        c = dict(op=op, fmt=rng.choice(["int8", "e4m3"]), B=B, Hq=Hkv * G, Hkv=Hkv, d=d, P=P, lens="uniform", lo=lo, hi=hi,
                 lens_seed=seed)
        if op == "decode":
            whole = rng.random() < 0.6
            c.update(window=-1 if whole else _log_int(rng, 1, 16384),
                     sinks=0 if whole else rng.choice([0, 1, 4, 5, 16, 64, 200]))
        return c
    new_hi = _log_int(rng, 1, max(1, min(cap, 65536 // B)))
    one = rng.random() < 0.3
    hi = min(hi, 4096)
    c = dict(op=op, B=B, Hkv=Hkv, d=d, P=P, lo=min(lo, hi), hi=hi, new_lo=1 if one else rng.choice([0, 1, new_hi // 2]),
             new_hi=1 if one else new_hi, pad=8 * rng.choice([0, 0, 1, 37, 512]), lens_seed=seed)
    if op == "slots":
        c.update(stray=rng.choice([0, 0, 3, 100]))
    else:
        c.update(fmt=rng.choice(["int8", "e4m3"]), Hq=Hkv * G, lens="uniform")
    return c


def _lengths(case):
    """The rows' lengths, and the new tokens of each row."""
    rng = random.Random(case["lens_seed"])
    B = case["B"]
    if case.get("lens") == "bimodal":
        lens = [rng.randint(512, 2048) if i % 2 else rng.randint(24576, 32768) for i in range(B)]
    else:
        lens = [rng.randint(case["lo"], case["hi"]) for _ in range(B)]
        if B > 2 and case["lo"] == 0:
            lens[B // 2] = 0
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(B)] if "new_hi" in case else [0] * B
    return lens, new


def _visible(n, case):
    w = case.get("window", -1)
    if w < 0:
        return n
    return min(n, w + case["sinks"])


def _first(case, n):
    """The first token of the block that a row's next token belongs to."""
    sb = min(case["P"], 16)
    return n // sb * sb


def work(case):
    lens, new = _lengths(case)
    B, P, op = case["B"], case["P"], case["op"]
    if op == "map":  # lengths in and out, free pages in, table entries out, a slot and a position per token
        pages = sum(-(-(a + b) // P) - -(-a // P) for a, b in zip(lens, new))
        return {"bytes": 16.0 * B + 8 * pages + 12 * (sum(new) + case["pad"]), "flops": 0.0}
    per = case["Hkv"] * case["d"]
    if op == "slots":
        return {"bytes": sum(new) * (8.0 * per + 8), "flops": 0.0}
    side = 2 + 8 / (min(P, 16) * case["d"])  # of K and V together: codes and scales, bytes per dim
    if op == "append":  # fp16 K and V in, 8-bit codes stored, fp16 K and V of the touched blocks out
        out = sum(a + b - _first(case, a) for a, b in zip(lens, new))
        return {"bytes": per * (sum(new) * (4 + side) + out * 4) + 8 * B, "flops": 0.0}
    if op == "read":
        return {"bytes": sum(lens) * per * (side + 4) + 8 * B, "flops": 0.0}
    vis = sum(_visible(n, case) for n in lens)
    return {"bytes": vis * per * side + B * case["Hq"] * (4 * case["d"] + 4), "flops": 4.0 * vis * case["Hq"] * case["d"]}


# ------------------------------------------------------------------ inputs

def _table(pages, num_pages, gen, stride):
    """A block table whose rows have `pages[i]` pages of their own, and the pages that are left."""
    order = torch.randperm(num_pages, generator=gen, device="cuda")
    B, used = len(pages), sum(pages)
    per = torch.tensor(pages, device="cuda")
    row = torch.repeat_interleave(torch.arange(B, device="cuda"), per, output_size=used)
    first = per.cumsum(0) - per
    # what is behind a row's pages names some page, and is never read
    table = order[torch.arange(B * stride, device="cuda") % num_pages].view(B, stride)
    table[row, torch.arange(used, device="cuda") - first[row]] = order[:used]
    return table.to(torch.int32).contiguous(), order[used:].to(torch.int32).contiguous()


def _offsets(count):
    off = [0]
    for n in count:
        off.append(off[-1] + n)
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def _tokens(gen, shape):
    """Keys or values [T, Hkv, d]: channels of unequal size, tokens of unequal size."""
    T, Hkv, d = shape
    gain = torch.exp(0.5 * torch.randn((Hkv, d), generator=gen, device="cuda"))
    gain /= gain.square().mean().sqrt()
    size = torch.exp(0.3 * torch.randn((T, 1, 1), generator=gen, device="cuda")).half()
    return torch.randn((T, Hkv, d), generator=gen, device="cuda", dtype=torch.float16).mul_(gain.half()).mul_(size)


def _page_bytes(P, d):
    tb, sb = min(P, 64), min(P, 16)
    return P // tb * (2 * tb * d + max(16, tb // sb * 8))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, P, op = case["B"], case["P"], case["op"]
    lens, new = _lengths(case)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    st = dict(case=case, lens=ints(lens))
    if op == "map":
        have = [-(-n // P) for n in lens]
        want = [-(-(a + b) // P) for a, b in zip(lens, new)]
        need = sum(want) - sum(have)
        stride = max(1, max(want))
        free = need + case["spare"] if case["spare"] >= 0 else need * 3 // 4
        num_pages = sum(have) + max(free, 1)
        st["table"], st["free"] = _table(have, num_pages, gen, stride)
        T = sum(new) + case["pad"]
        st.update(T=T, new=ints(new), free_count=ints([free]), num_pages=num_pages, free_out=ints([0]),
                  lens_out=torch.empty_like(st["lens"]), offsets=torch.empty(B + 1, dtype=torch.int32, device="cuda"),
                  slots=torch.empty(T, dtype=torch.int64, device="cuda"),
                  positions=torch.empty(T, dtype=torch.int32, device="cuda"))
        if own:
            from paged_kv_gqa_09_gb300 import api
            st["shape"] = api.Shape(B, 1, 1, 128, P, num_pages, stride, 1.0)
            st["ws"] = torch.zeros(api.pkv_attn_workspace_size(st["shape"]), dtype=torch.uint8, device="cuda")
        return st
    Hkv, d = case["Hkv"], case["d"]
    pages = [-(-(a + b) // P) for a, b in zip(lens, new)]
    stride = max(1, max(pages))
    num_pages = max(1, sum(pages)) + 3
    st["table"], _ = _table(pages, num_pages, gen, stride)
    if "new_hi" in case:  # K and V of the new tokens, slices of one fused projection
        T = sum(new) + case.get("stray", 0)
        buf = torch.empty((T, 2 * Hkv * d + case["pad"]), dtype=torch.float16, device="cuda")
        st["k_new"] = buf[:, :Hkv * d].unflatten(1, (Hkv, d))
        st["v_new"] = buf[:, Hkv * d:2 * Hkv * d].unflatten(1, (Hkv, d))
        st["k_new"].copy_(_tokens(gen, (T, Hkv, d)))
        st["v_new"].copy_(_tokens(gen, (T, Hkv, d)))
    if op == "slots":
        st["k"] = torch.randn((num_pages, P, Hkv, d), generator=gen, device="cuda", dtype=torch.float16)
        st["v"] = torch.randn((num_pages, P, Hkv, d), generator=gen, device="cuda", dtype=torch.float16)
        off = _offsets(new).long()
        row = torch.repeat_interleave(torch.arange(B, device="cuda"), off[1:] - off[:-1], output_size=sum(new))
        pos = st["lens"].long()[row] + torch.arange(sum(new), device="cuda") - off[row]
        st["slots"] = torch.full((T,), -1, dtype=torch.int64, device="cuda")  # those behind the last row's have none
        st["slots"][:sum(new)] = st["table"].long()[row, pos // P] * P + pos % P
        if own:
            from paged_kv_gqa_09_gb300 import api
            st["shape"] = api.Shape(B, Hkv, Hkv, d, P, num_pages, stride, 1.0)
            st["ws"] = torch.zeros(api.pkv_attn_workspace_size(st["shape"]), dtype=torch.uint8, device="cuda")
        return st
    # pages of quantised tokens, dealt out over the pool
    bank = min(num_pages * Hkv, max(16, (1 << 22) // (P * d)))
    full = torch.zeros((bank, 1, _page_bytes(P, d)), dtype=torch.uint8, device="cuda")
    at = torch.arange(bank * P // min(P, 16), device="cuda")
    sb = min(P, 16)
    tok = at.unsqueeze(1) * sb + torch.arange(sb, device="cuda")
    _store(full, case["fmt"], P, d, at // (P // sb), at % (P // sb), tok, torch.zeros_like(tok, dtype=torch.bool),
           _tokens(gen, (bank * P, 1, d)), _tokens(gen, (bank * P, 1, d)))
    pick = torch.randint(0, bank, (num_pages * Hkv,), generator=gen, device="cuda")
    st["cache"] = full.view(bank, -1)[pick].view(num_pages, Hkv, -1)
    if op == "decode":
        st["q"] = torch.randn((B, case["Hq"], d), generator=gen, device="cuda", dtype=torch.float16)
        st["o"] = torch.empty((B, case["Hq"], d), dtype=torch.float16, device="cuda")
        st["lse"] = torch.empty((B, case["Hq"]), dtype=torch.float32, device="cuda")
        st["scale"] = 1.0 / math.sqrt(d)
    else:
        first = [_first(case, n) if op == "append" else 0 for n in lens]
        count = [a + b - f for a, b, f in zip(lens, new, first)]
        st.update(first=ints(first), out_offsets=_offsets(count), T_out=sum(count))
        st["k_out"] = torch.empty((sum(count), Hkv, d), dtype=torch.float16, device="cuda")
        st["v_out"] = torch.empty((sum(count), Hkv, d), dtype=torch.float16, device="cuda")
        if op == "append":
            st.update(offsets=_offsets(new), lens_out=torch.empty_like(st["lens"]), one=case["new_lo"] == case["new_hi"] == 1)
    if own:
        from paged_kv_gqa_09_gb300 import api
        st["fmt"] = {"int8": api.PKV_BYTE_INT8, "e4m3": api.PKV_BYTE_E4M3}[case["fmt"]]
        st["shape"] = api.make_byte_shape(case["Hq"], d, st["cache"], st["table"])
        st["ws"] = torch.zeros(api.pkv_attn_workspace_size(st["shape"]), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ a pass

def run(st):
    op = st["case"]["op"]
    if own:
        return _run_own(st, op)
    return {"map": _plain_map, "slots": _plain_slots, "append": _plain_append, "read": _plain_read,
            "decode": _plain_decode}[op](st)


def _run_own(st, op):
    from paged_kv_gqa_09_gb300 import api
    c = st["case"]
    if op == "map":
        api.pkv_map_pages(st["shape"], st["ws"], st["lens"], st["new"], st["table"], st["free"], st["free_count"],
                          st["slots"], st["offsets"], seq_lens_out=st["lens_out"], free_count_out=st["free_out"],
                          positions=st["positions"])
        return {k: st[k] for k in ("table", "slots", "positions", "offsets", "lens_out", "free_out")}
    if op == "slots":
        api.pkv_append_slots(st["shape"], st["ws"], st["k_new"], st["v_new"], st["slots"], st["k"], st["v"])
        return {"k": st["k"], "v": st["v"]}
    if op == "append":
        api.pkv_byte_append(st["shape"], st["ws"], st["fmt"], st["k_new"], st["v_new"], st["table"], st["lens"], st["cache"],
                          new_offsets=None if st["one"] else st["offsets"], seq_lens_out=st["lens_out"])
        api.pkv_byte_read(st["shape"], st["ws"], st["fmt"], st["cache"], st["table"], st["lens_out"], st["out_offsets"],
                        st["k_out"], st["v_out"], first=st["first"])
        return {"lens": st["lens_out"], "k": st["k_out"], "v": st["v_out"]}
    if op == "read":
        api.pkv_byte_read(st["shape"], st["ws"], st["fmt"], st["cache"], st["table"], st["lens"], st["out_offsets"],
                        st["k_out"], st["v_out"])
        return {"k": st["k_out"], "v": st["v_out"]}
    if c["window"] < 0:
        api.pkv_byte_decode(st["shape"], st["ws"], st["fmt"], st["q"], st["cache"], st["table"], st["lens"], st["o"], st["lse"])
    else:
        api.pkv_byte_decode(st["shape"], st["ws"], st["fmt"], st["q"], st["cache"], st["table"], st["lens"], st["o"], st["lse"],
                          window=c["window"], sinks=c["sinks"])
    return {"o": st["o"], "lse": st["lse"]}


# ------------------------------------------------------------------ the plain form

def _power(e):
    """2^e in 32 bits, for whole e."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _spread(off, total):
    """Row and place within its row of every packed token."""
    off = off.long()
    row = torch.repeat_interleave(torch.arange(off.numel() - 1, device=off.device), off[1:] - off[:-1], output_size=total)
    return row, torch.arange(total, device=off.device) - off[row]


def _plain_map(st):
    P, T = st["case"]["P"], st["T"]
    N, n, free = st["lens"].long(), st["new"].long(), st["free_count"].long()
    have = (N + P - 1) // P
    need = (N + n + P - 1) // P - have
    upto = need.cumsum(0)
    served = (need == 0) | (upto <= free)
    taken = torch.where(upto <= free, upto, 0).amax().view(1)
    table = st["table"]
    top = st["free"].numel()
    # a row of the table per needed page
    most = int(st["T"]) // P + n.numel()
    which = torch.arange(most, device=N.device)
    row = torch.searchsorted(upto, which, right=True).clamp(max=n.numel() - 1)
    there = which < upto[-1]
    block = torch.where(there, have[row] + which - (upto[row] - need[row]), 0)
    page = st["free"][(free - 1 - which).clamp(0, top - 1)]
    page = torch.where(served[row], page, -1).to(torch.int32)
    flat = torch.where(there, row * table.shape[1] + block, table.numel())
    grown = torch.cat([table.view(-1), table.new_zeros(1)]).index_put((flat,), page)
    table.copy_(grown[:-1].view_as(table))
    off = torch.cat([n.new_zeros(1), n.cumsum(0)])
    x = torch.arange(T, device=N.device)
    row = torch.searchsorted(off[1:], x, right=True).clamp(max=n.numel() - 1)
    live = (x < off[-1]) & served[row]
    pos = torch.where(live, N[row] + x - off[row], 0)
    slots = torch.where(live, table[row, pos // P].long() * P + pos % P, -1)
    return {"table": table, "slots": slots, "positions": pos.to(torch.int32), "offsets": off.to(torch.int32),
            "lens_out": torch.where(served, N + n, N).to(torch.int32), "free_out": (free - taken).to(torch.int32)}


def _plain_slots(st):
    at = st["slots"]
    live = (at >= 0).nonzero().squeeze(1)
    at = at[live]
    st["k"].flatten(0, 1)[at] = st["k_new"][live]
    st["v"].flatten(0, 1)[at] = st["v_new"][live]
    return {"k": st["k"], "v": st["v"]}


def _parts(cache, P, d):
    """K codes [page, head, block, token, d], V codes [page, head, block, SB block, d / 4, SB / 4, 4, 4] and scales
    [page, head, block, SB block, 2], views of the cache (see the layout above)."""
    tb, sb = min(P, 64), min(P, 16)
    size = _page_bytes(P, d) // (P // tb)
    blocks = cache.unflatten(2, (P // tb, size))
    k = blocks[..., :tb * d].unflatten(3, (tb, d))
    v = blocks[..., tb * d:2 * tb * d].unflatten(3, (tb // sb, d // 4, sb // 4, 4, 4))
    f = cache.view(torch.float32).unflatten(2, (P // tb, size // 4))[..., tb * d // 2:tb * d // 2 + tb // sb * 2]
    return k, v, f.unflatten(3, (tb // sb, 2))


def _turned(k, token):
    """K codes [.., d] of tokens [..] with the halves of two in four swapped, back or forth."""
    if k.shape[-1] < 128:
        return k
    swapped = (token % 4 >= 2).view(token.shape + (1,) * (k.dim() - token.dim()))
    return torch.where(swapped, k.roll(64, -1), k)


def _decoded(c, fmt):
    """Codes to the numbers they are, in 32 bits."""
    return c.view(torch.int8).float() if fmt == "int8" else c.view(torch.float8_e4m3fn).float()


def _coded(y, fmt):
    """The codes nearest to y."""
    return (y.round().to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)).view(torch.uint8)


def _store(cache, fmt, P, d, page, block, tok, keep, k, v):
    """Block x is SB tokens at `block[x]` of page `page[x]`: token tok[x, u] of k and v [T, Hkv, d] where that is not
    negative, what is there already where keep[x, u]."""
    sb, tb = min(P, 16), min(P, 64)
    kc, vc, sc = _parts(cache, P, d)
    blk, sub = block * sb // tb, block * sb % tb // sb
    slot = sub.unsqueeze(1) * sb + torch.arange(sb, device=cache.device)
    mine, keeps = (tok >= 0)[..., None, None], keep[..., None, None]
    for side, x in enumerate((k, v)):
        x = torch.where(mine, x[tok.clamp(min=0)].float(), 0).clamp(-Q[fmt] * 2.0 ** MOST[fmt], Q[fmt] * 2.0 ** MOST[fmt])
        # [blocks, SB, Hkv, d] of what the blocks hold
        if side == 0:
            raw = kc[page.unsqueeze(1), :, blk.unsqueeze(1), slot]
            old = _decoded(_turned(raw, slot).contiguous(), fmt)
        else:
            raw = vc[page, :, blk, sub].permute(0, 3, 5, 1, 2, 4).flatten(1, 2).flatten(3, 4)
            old = _decoded(raw.contiguous(), fmt)
        scale = sc[page, :, blk, sub, side]  # [blocks, Hkv]
        top = x.abs().amax((1, 3))
        e = torch.frexp(top / Q[fmt])[1]  # 2^e beyond top / Q
        e = torch.where(top > 0, e, LEAST[fmt]).clamp(LEAST[fmt], MOST[fmt] + 1)
        s = _power(torch.where(top <= Q[fmt] * _power(e - 1), e - 1, e).clamp(LEAST[fmt], MOST[fmt]))
        s = torch.where(keep.any(1).unsqueeze(1), torch.maximum(s, scale), s)
        wide = s[:, None, :, None]
        y = torch.where(mine, x / wide, torch.where(keeps, old * (scale / s)[:, None, :, None], 0))
        c = _coded(y, fmt)
        if side == 0:
            c = torch.where(mine | keeps, _turned(c, slot), raw)
            kc[page.unsqueeze(1), :, blk.unsqueeze(1), slot] = c
        else:
            c = torch.where(mine | keeps, c, raw)
            vc[page, :, blk, sub] = c.unflatten(3, (d // 4, 4)).unflatten(1, (sb // 4, 4)).permute(0, 3, 4, 1, 5, 2)
        sc[page, :, blk, sub, side] = s


def _load(cache, fmt, page, slot, P, d):
    """K and V of tokens [..] as [.., Hkv, d] in 32 bits."""
    tb, sb = min(P, 64), min(P, 16)
    kc, vc, sc = _parts(cache, P, d)
    blk, sub, u = slot // tb, slot % tb // sb, slot % sb
    scale = sc[page, :, blk, sub]  # [.., Hkv, 2]
    k = _decoded(_turned(kc[page, :, blk, slot % tb], slot).contiguous(), fmt) * scale[..., 0:1]
    v = _decoded(vc[page, :, blk, sub, :, u // 4, :, u % 4].flatten(-2).contiguous(), fmt) * scale[..., 1:2]
    return k, v


def _plain_append(st):
    c, table = st["case"], st["table"].long()
    P, d, sb = c["P"], c["d"], min(c["P"], 16)
    N, off = st["lens"].long(), st["offsets"].long()
    n = off[1:] - off[:-1]
    count = torch.where(n > 0, (N + n + sb - 1) // sb - N // sb, 0)  # blocks the rows write to
    ends = count.cumsum(0)
    most = st["k_new"].shape[0] // sb + 2 * N.numel()
    x = torch.arange(most, device=N.device)
    x = x[x < ends[-1]]
    row = torch.searchsorted(ends, x, right=True)
    block = (N // sb)[row] + x - (ends - count)[row]
    pos = block.unsqueeze(1) * sb + torch.arange(sb, device=N.device)
    place = pos - N[row].unsqueeze(1)
    tok = torch.where((place >= 0) & (place < n[row].unsqueeze(1)), off[row].unsqueeze(1) + place, -1)
    _store(st["cache"], c["fmt"], P, d, table[row, block * sb // P], block * sb % P // sb, tok, place < 0, st["k_new"],
           st["v_new"])
    return {"lens": st["lens"] + n.to(torch.int32), **_plain_read(st)}


def _plain_read(st):
    c, table = st["case"], st["table"].long()
    row, at = _spread(st["out_offsets"], st["T_out"])
    pos = st["first"].long()[row] + at
    k, v = _load(st["cache"], c["fmt"], table[row, pos // c["P"]], pos % c["P"], c["P"], c["d"])
    return {"k": k.half(), "v": v.half()}


def _seen(st):
    """Positions [B, X] that the queries see, and which of them are there."""
    c, n = st["case"], st["lens"].long().unsqueeze(1)
    most = max(_lengths(c)[0])
    sinks = c["sinks"] if c["window"] >= 0 else 0
    w = c["window"] if c["window"] >= 0 else most
    x = torch.arange(max(1, min(most, w + sinks)), device=n.device).unsqueeze(0)
    head = n.clamp(max=sinks)
    pos = torch.where(x < head, x, x - head + torch.maximum(head, n - w))
    return pos, pos < n


def _plain_decode(st):
    c, q = st["case"], st["q"]
    P, d = c["P"], c["d"]
    pos, there = _seen(st)
    pos = torch.where(there, pos, 0)
    k, v = _load(st["cache"], c["fmt"], st["table"].long().gather(1, pos // P), pos % P, P, d)
    B, Hq, _ = q.shape
    Hkv = k.shape[2]
    s = torch.matmul(q.float().view(B, Hkv, Hq // Hkv, d), k.permute(0, 2, 3, 1)) * st["scale"]
    s = s.masked_fill(~there.view(B, 1, 1, -1), -math.inf)
    top = s.amax(-1, keepdim=True)
    base = torch.where(torch.isfinite(top), top, 0)
    p = (s - base).exp()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, 1)
    return {"o": o.view(B, Hq, d).half(), "lse": (base + total.log()).view(B, Hq)}


# ------------------------------------------------------------------ in 64 bits

def _exact_bytes(cache, pages, n, P, d):
    """Codes of K and V [n, Hkv, d] (uint8) and their scales [n, Hkv, 1] of the first n tokens in `pages`, by each
    value's place in the cache."""
    tb, sb = min(P, 64), min(P, 16)
    size = 2 * tb * d + max(16, 8 * (tb // sb))
    held = cache[pages]
    tok = torch.arange(n, device=cache.device).view(n, 1, 1)
    dim = torch.arange(d, device=cache.device).view(1, 1, d)
    head = torch.arange(cache.shape[1], device=cache.device).view(1, -1, 1)
    page, slot = tok // P, tok % P
    base, r = slot // tb * size, slot % tb
    half = r % 4 // 2 * 64 if d == 128 else 0
    u = r % sb
    k = held[page, head, base + r * d + torch.bitwise_xor(dim, torch.as_tensor(half, device=cache.device))]
    v = held[page, head, base + tb * d + r // sb * sb * d + (dim // 4 * (sb // 4) + u // 4) * 16 + dim % 4 * 4 + u % 4]
    real = held.view(torch.float32)
    at = base // 4 + tb * d // 2 + r // sb * 2
    return k, v, real[page, head, at].double(), real[page, head, at + 1].double()


def _exact_number(c, fmt):
    """Codes to the numbers they are, in 64 bits."""
    b = c.long()
    if fmt == "int8":
        return torch.where(b < 128, b, b - 256).double()
    exponent, mantissa = b // 8 % 16, b % 8
    power = (torch.clamp(exponent, min=1) + (1023 - 10) << 52).view(torch.float64)
    size = (torch.where(exponent > 0, 8 + mantissa, mantissa)).double() * power
    return torch.where(b < 128, size, -size)


def _exact_round(y, fmt):
    """The numbers nearest to y that have a code, ties to even."""
    if fmt == "int8":
        return y.round()
    exponent = (torch.frexp(y)[1] - 1).clamp(min=-6)
    step = (exponent.long() + (1023 - 3) << 52).view(torch.float64)
    return (y / step).round() * step


def _exact_append(st, side, i, n, new):
    """What the blocks that row i's `new` tokens touch hold afterwards [tokens, Hkv, d], side 0 K, 1 V."""
    c = st["case"]
    P, d, fmt, sb = c["P"], c["d"], c["fmt"], min(c["P"], 16)
    first = _first(c, n)
    off = int(st["offsets"][i])
    x = (st["k_new"], st["v_new"])[side][off:off + new].double()
    bound = Q[fmt] * 2.0 ** MOST[fmt]
    x = torch.minimum(torch.maximum(x, torch.full_like(x, -bound)), torch.full_like(x, bound))
    held = _exact_bytes(st["cache"], st["table"][i, :-(-n // P)].long(), n, P, d) if n > first else None
    out = []
    for a in range(first, n + new, 1 << 14):  # whole blocks at a time
        b = min(a + (1 << 14), n + new)
        y = torch.zeros((-(-(b - a) // sb) * sb, c["Hkv"], d), dtype=torch.float64, device="cuda")
        old = max(0, n - a)
        if old:
            was = held[2 + side][a:n, :, 0][:1]  # one block's: [1, Hkv]
            y[:old] = _exact_number(held[side][a:n], fmt) * was.unsqueeze(-1)
        y[old:b - a] = x[a + old - n:b - n]
        fresh = y.clone()
        fresh[:old] = 0
        top = fresh.abs().view(-1, sb, c["Hkv"], d).amax((1, 3))
        scale = torch.full_like(top, 2.0 ** LEAST[fmt])
        for e in range(LEAST[fmt], MOST[fmt]):
            scale = torch.where(top > Q[fmt] * 2.0 ** e, 2.0 ** (e + 1), scale)
        if old:
            scale[0] = torch.maximum(scale[0], was[0])
        scale = scale.repeat_interleave(sb, 0).unsqueeze(-1)
        out.append((_exact_round(y / scale, fmt) * scale)[:b - a])
    return torch.cat(out) if out else torch.zeros((0, c["Hkv"], d), dtype=torch.float64, device="cuda")


def _exact_slots(st, side, lens, new):
    """The pages [num_pages, P, Hkv, d] of one side after every row's new tokens, a page at a time."""
    P, pages, packed = st["case"]["P"], st[side].double(), st[side + "_new"].double()
    table, off = st["table"].tolist(), 0
    for row, n, m in zip(table, lens, new):
        for a in range(n // P * P, n + m, P):
            b, e = max(a, n), min(a + P, n + m)
            pages[row[a // P], b - a:e - a] = packed[off + b - n:off + e - n]
        off += m
    return pages


def exact(case, seed):
    op = case["op"]
    if op == "map":  # whole numbers
        return None
    st = prepare(case, seed)
    lens, new = _lengths(case)
    if op == "slots":
        return {side: _exact_slots(st, side, lens, new) for side in ("k", "v")}
    P, d, B, Hkv, fmt = case["P"], case["d"], case["B"], case["Hkv"], case["fmt"]
    if op == "append":
        # a row without new tokens keeps its last block
        sides = [[], []]
        for i, (n, m) in enumerate(zip(lens, new)):
            if m:
                for side in (0, 1):
                    sides[side].append(_exact_append(st, side, i, n, m))
            elif n > _first(case, n):
                held = _exact_bytes(st["cache"], st["table"][i, :-(-n // P)].long(), n, P, d)
                for side in (0, 1):
                    sides[side].append((_exact_number(held[side], fmt) * held[2 + side])[_first(case, n):])
        empty = torch.zeros((0, Hkv, d), dtype=torch.float64, device="cuda")
        return {"lens": None, "k": torch.cat([empty] + sides[0]), "v": torch.cat([empty] + sides[1])}
    o = torch.zeros((B, case["Hq"], d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, case["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    G = case["Hq"] // Hkv
    rows = []
    for i, n in enumerate(lens):
        if not n:
            continue
        ck, cv, sk, sv = _exact_bytes(st["cache"], st["table"][i, :-(-n // P)].long(), n, P, d)
        k, v = _exact_number(ck, fmt) * sk, _exact_number(cv, fmt) * sv
        if op == "read":
            rows.append((k, v))
            continue
        keep = torch.arange(n, device="cuda")
        if case["window"] >= 0:
            keep = keep[(keep < case["sinks"]) | (keep >= n - case["window"])]
        if not keep.numel():
            continue
        for h in range(Hkv):
            s = st["q"][i, h * G:(h + 1) * G].double() @ k[keep, h].T / math.sqrt(d)
            lse[i, h * G:(h + 1) * G] = torch.logsumexp(s, 1)
            o[i, h * G:(h + 1) * G] = torch.softmax(s, 1) @ v[keep, h]
    if op == "read":
        empty = torch.zeros((0, Hkv, d), dtype=torch.float64, device="cuda")
        return {"k": torch.cat([empty] + [r[0] for r in rows]), "v": torch.cat([empty] + [r[1] for r in rows])}
    return {"o": o, "lse": lse}
