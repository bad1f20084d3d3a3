"""The decode-side operators over the paged K/V store: what is measured, and their plain forms.

Four families, as one beam-search decode step uses them: rotary positions (with the store write),
attention of one new token over the paged store, the selection over beams and vocabulary, and the
pages of the store (fork, reserve with copy-on-write, compaction).
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 32 sequences: q, k, v straight from the fused projection, k and v to store slots
        dict(name="rotary decode 32", op="rotary", tokens=32, hq=32, hkv=8, dh=128, rd=128, inter=False, f32=False,
             scaling="none", inverse=False, store=16),
        # a prompt chunk in f32, interleaved pairs over a quarter of an 80-wide head, far positions, scaled by parts
        dict(name="rotary prompt part", op="rotary", tokens=2001, hq=16, hkv=4, dh=80, rd=20, inter=True, f32=True,
             scaling="parts", inverse=False, store=0),
        # the gradient of a training batch's rotation: 8 sequences of 4096 tokens
        dict(name="rotary gradient", op="rotary", tokens=32768, hq=32, hkv=8, dh=128, rd=128, inter=False, f32=False,
             scaling="linear", inverse=True, store=0),
        # one short sequence of the 0.6B-shaped layer: latency
        dict(name="decode one", op="decode", reqs=1, hq=16, hkv=8, dh=128, lo=700, hi=700, page=16, window=0, f32=False),
        # one long sequence alone: only the split over its length fills the GPU
        dict(name="decode one long", op="decode", reqs=1, hq=32, hkv=8, dh=128, lo=32000, hi=32000, page=16, window=0,
             f32=False),
        # a window layer, f32 output, 64-row pages
        dict(name="decode window f32", op="decode", reqs=16, hq=32, hkv=8, dh=128, lo=9000, hi=16384, page=64, window=4096,
             f32=True),
        # a ragged serving batch, 1K to 32K
        dict(name="decode ragged 64", op="decode", reqs=64, hq=32, hkv=8, dh=128, lo=1024, hi=32768, page=16, window=0,
             f32=False),
        # four beams of one request
        dict(name="beams 1x4", op="beam", reqs=1, beams=4, out=4, vocab=151936, f32=False, finished=False),
        # f32 logits of an odd vocabulary, some beams finished, some tokens masked
        dict(name="beams 17x5 f32", op="beam", reqs=17, beams=5, out=5, vocab=32003, f32=True, finished=True),
        # 64 requests of 8 beams
        dict(name="beams 64x8", op="beam", reqs=64, beams=8, out=8, vocab=151936, f32=False, finished=True),
        # the pages' side of a beam step: 32 requests of 8 beams fork, then make room for one row each
        dict(name="pages beam step", op="step", reqs=32, beams=8, lo=256, hi=8192, page=16, hkv=8, dh=128),
        # a store of 16384 pages, 60% in use, moved together
        dict(name="pages compact", op="compact", pages=16384, used=0.6, rows=128, page=16, hkv=8, dh=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "decode", "decode", "decode", "beam", "beam", "step", "compact"])
    if op == "rotary":
        dh = rng.choice([64, 80, 96, 128, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 5, 8])
        rd = rng.choice([dh, dh, dh // 2, 2 * rng.randint(1, dh // 2)])
        f32 = rng.random() < 0.3
        most = max(1, 32768 * 40 * 128 // ((hq + 2 * hkv) * dh * (2 if f32 else 1)))
        inverse = rng.random() < 0.3
        return dict(op=op, tokens=_log(rng, 1, most), hq=hq, hkv=hkv, dh=dh, rd=rd, inter=rng.random() < 0.5, f32=f32,
                    scaling=rng.choice(["none", "linear", "base", "parts"]), inverse=inverse,
                    store=0 if inverse else rng.choice([0, 0, 16, 5]))
    if op == "decode":
        reqs = _log(rng, 1, 256)
        hkv = rng.choice([1, 2, 4, 8])
        g = rng.choice([1, 2, 4, 4, 6, 8, 16, 32])
        dh = rng.choice([64, 128, 128])
        hi = _log(rng, 1, max(1, min(60000, 64 * 9000 * 1024 // (reqs * hkv * dh * (4 if g > 16 else 1)))))
        lo = max(1, min(hi, int(hi * rng.choice([0.05, 0.5, 1.0]))))
        return dict(op=op, reqs=reqs, hq=hkv * g, hkv=hkv, dh=dh, lo=lo, hi=hi, page=rng.choice([16, 16, 24, 32, 64, 128]),
                    window=rng.choice([0, 0, 0, _log(rng, 1, 8192)]), f32=rng.random() < 0.3)
    if op == "beam":
        f32 = rng.random() < 0.3
        beams = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
        vocab = _log(rng, 50, 152000)
        reqs = _log(rng, 1, max(1, min(256, 64 * 8 * 151936 // (beams * vocab * (2 if f32 else 1)))))
        return dict(op=op, reqs=reqs, beams=beams, out=min(beams * vocab, rng.choice([beams, beams, 1, 4, 16, 32])), vocab=vocab,
                    f32=f32, finished=rng.random() < 0.5)
    page, hkv, dh = rng.choice([16, 16, 24, 32, 64]), rng.choice([2, 4, 8]), rng.choice([64, 128])
    if op == "step":
        lo = _log(rng, 1, 2048)
        return dict(op=op, reqs=_log(rng, 1, 32), beams=rng.choice([1, 2, 4, 5, 8]), lo=lo, hi=min(8192, lo * rng.choice([1, 2, 4])),
                    page=page, hkv=hkv, dh=dh)
    most = 16384 * 16 * 1024 // (page * hkv * dh)
    return dict(op=op, pages=_log(rng, 64, min(most, 40000)), used=rng.choice([0.1, 0.5, 0.6, 0.9]), rows=_log(rng, 1, 256), page=page,
                hkv=hkv, dh=dh)


# ------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _dt(case):
    return torch.float32 if case["f32"] else torch.bfloat16


def _frequencies(rd, scaling, theta=1e6, factor=4.0, original=8192):
    """The pairs' angles per position (64 bits, on the host) and the amplitude: plain, positions
    divided by the factor, a stretched base, or blended by parts."""
    i = np.arange(rd // 2, dtype=np.float64)
    amp = 1.0
    if scaling == "base":
        theta = theta * factor ** (rd / (rd - 2.0)) if rd > 2 else theta
    f = theta ** (-2.0 * i / rd)
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        lo = max(0, math.floor(rd * math.log(original / (32.0 * 2 * math.pi)) / (2 * math.log(theta))))
        hi = min(rd - 1, math.ceil(rd * math.log(original / (1.0 * 2 * math.pi)) / (2 * math.log(theta))))
        part = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        f = f * (1 - part) + f / factor * part
        amp = 0.1 * math.log(factor) + 1.0
    return f, amp


def _lens(case, rng):
    lo, hi = case["lo"], case["hi"]
    n = np.exp(rng.uniform(math.log(lo), math.log(hi + 0.999), case["reqs"])).astype(np.int64).clip(lo, hi)
    n[0] = hi
    return n


def prepare(case, seed):
    g, rng = _gen(seed), np.random.default_rng(int(seed))
    op = case["op"]
    s = dict(case=case)
    if op == "rotary":
        t, hq, hkv, dh = case["tokens"], case["hq"], case["hkv"], case["dh"]
        x = torch.randn(t, hq + 2 * hkv, dh, device="cuda", generator=g).to(_dt(case))
        s.update(q=x[:, :hq], k=x[:, hq:hq + hkv], v=x[:, hq + hkv:])
        s["pos"] = torch.randint(0, 131072 if case["scaling"] != "none" else 32768, (t,), device="cuda", generator=g, dtype=torch.int32)
        s["freq"], s["amp"] = _frequencies(case["rd"], case["scaling"])
        if case["store"]:
            rows = (t + 7) // case["store"] * case["store"] + 2 * case["store"]
            s["k_store"] = torch.zeros(rows, hkv, dh, device="cuda", dtype=_dt(case))
            s["v_store"] = torch.zeros_like(s["k_store"])
            s["slot"] = torch.randperm(rows, device="cuda", generator=g)[:t].to(torch.int32)
            if t > 8:
                s["slot"][t - 3:] = -1  # padding rows of the batch
        return s
    if op == "decode":
        n, ps, hkv, dh = case["reqs"], case["page"], case["hkv"], case["dh"]
        lens = _lens(case, rng)
        per = -(-lens // ps)
        pages, width = int(per.sum()) + 3, int(per.max()) + 1
        table = np.full((n, width), -1, np.int32)
        table[np.arange(width)[None] < per[:, None]] = rng.permutation(pages)[:int(per.sum())]
        s["table"] = torch.from_numpy(table).cuda()
        s["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
        s["k"] = torch.randn(pages, ps, hkv, dh, device="cuda", generator=g, dtype=torch.bfloat16)
        s["v"] = torch.randn(pages, ps, hkv, dh, device="cuda", generator=g, dtype=torch.bfloat16)
        s["q"] = (1.5 * torch.randn(n, case["hq"], dh, device="cuda", generator=g)).to(torch.bfloat16)
        s["longest"] = int(lens.max())
        return s
    if op == "beam":
        n, w, vocab = case["reqs"], case["beams"], case["vocab"]
        s["logits"] = torch.randn(n, w, vocab, device="cuda", generator=g, dtype=_dt(case)).mul_(2.5)
        for r in range(n):  # tokens that the request may not take, one in a hundred; never the end token 7
            ban = torch.randint(8, vocab, (vocab // 100,), device="cuda", generator=g)
            s["logits"][r, :, ban] = -math.inf
        s["scores"] = -10.0 * torch.rand(n, w, device="cuda", generator=g)
        s["finished"] = torch.rand(n, w, device="cuda", generator=g) < 0.15 if case["finished"] else None
        return s
    ps, hkv, dh = case["page"], case["hkv"], case["dh"]
    if op == "step":
        n, w = case["reqs"], case["beams"]
        lens = np.repeat(_lens(case, rng), w)
        rows = n * w
        per, kept = -(-lens // ps), np.repeat(rng.integers(0, 4, n), w)  # the last 0 to 3 pages are each beam's own
        width = int(per.max()) + 2
        first = np.maximum(per - 1 - kept, 0)  # pages that the request's beams share
        at = np.arange(width)[None]
        base = np.arange(rows)[:, None] // w * w
        key = np.where(at < first[:, None], base, np.arange(rows)[:, None]) * width + at
        live = at < per[:, None]
        names, back = np.unique(key[live], return_inverse=True)
        pages = n * -(-case["hi"] // ps) + 5 * rows + 8  # whatever the lengths drawn
        ids = rng.permutation(pages)[:len(names)].astype(np.int32)
        table = np.full((rows, width), -1, np.int32)
        table[live] = ids[back]
        s["table0"] = torch.from_numpy(table).cuda()
        s["refs0"] = torch.from_numpy(np.bincount(table[live], minlength=pages).astype(np.int32)).cuda()
        s["lens0"] = torch.from_numpy(lens.astype(np.int32)).cuda()
        s["parent"] = torch.from_numpy((np.arange(rows) // w * w + rng.integers(0, w, rows)).astype(np.int32)).cuda()
        s["starts"] = torch.arange(rows + 1, dtype=torch.int32, device="cuda")  # one new row each
        for k in ("table", "refs", "lens"):
            s[k] = s[k + "0"].clone()
    else:
        pages, rows = case["pages"], case["rows"]
        used = max(1, int(pages * case["used"]))
        ids = rng.permutation(pages)[:used].astype(np.int32)
        width = -(-used // rows) + 3
        table = np.full((rows, width), -1, np.int32)
        cut = np.array_split(ids, rows)
        for r in range(rows):
            table[r, :len(cut[r])] = cut[r]
        if rows > 1:
            share = min(len(cut[0]), len(cut[1])) // 2  # some pages in two rows' tables
            table[rows - 1, :share] = table[0, :share]
        s["table0"] = torch.from_numpy(table).cuda()
        refs = np.bincount(table[table >= 0], minlength=pages).astype(np.int32)
        s["refs0"] = torch.from_numpy(refs).cuda()
        for k in ("table", "refs"):
            s[k] = s[k + "0"].clone()
    s["k"] = torch.randn(pages, ps, hkv, dh, device="cuda", generator=g, dtype=torch.bfloat16)
    s["v"] = torch.randn(pages, ps, hkv, dh, device="cuda", generator=g, dtype=torch.bfloat16)
    return s


# ------------------------------------------------------------------------------------- plain forms
def _rotated(x, cos, sin, c):
    rd = c["rd"]
    x = x.float()
    a, b = (x[..., 0:rd:2], x[..., 1:rd:2]) if c["inter"] else (x[..., :rd // 2], x[..., rd // 2:rd])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, v), -1).flatten(-2) if c["inter"] else torch.cat((u, v), -1)
    return torch.cat((turned, x[..., rd:]), -1).to(_dt(c))


def _rotary(s):
    c = s["case"]
    f = torch.from_numpy(s["freq"]).cuda()
    angle = s["pos"].double()[:, None] * f  # 64 bits: far positions
    cos = (s["amp"] * angle.cos()).float()[:, None]
    sin = (s["amp"] * angle.sin()).float()[:, None]
    if c["inverse"]:
        sin = -sin
    q, k = _rotated(s["q"], cos, sin, c), _rotated(s["k"], cos, sin, c)
    if not c["store"]:
        return dict(q=q, k=k)
    keep = s["slot"] >= 0
    at = s["slot"][keep].long()
    s["k_store"][at] = k[keep]
    s["v_store"][at] = s["v"][keep]
    return dict(q=q, k=s["k_store"], v=s["v_store"])


def _decode(s):
    c = s["case"]
    n, ps, hkv, dh, longest = c["reqs"], c["page"], c["hkv"], c["dh"], s["longest"]
    lens = s["lens"].long()
    first = (lens - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(lens)
    span = min(longest, c["window"] or longest)
    j = first[:, None] + torch.arange(span, device="cuda")[None]
    seen = j < lens[:, None]
    j = j.clamp(max=longest - 1)
    page = s["table"].gather(1, j // ps).long().clamp(min=0)
    k, v = s["k"][page, j % ps].float(), s["v"][page, j % ps].float()
    q = s["q"].float().view(n, hkv, c["hq"] // hkv, dh)
    score = torch.einsum("nhgd,nlhd->nhgl", q, k) / math.sqrt(dh)
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("nhgl,nlhd->nhgd", p / total, v.masked_fill(~seen[:, :, None, None], 0.0))
    return dict(out=out.reshape(n, c["hq"], dh).to(_dt(c)), lse=(top + total.log()).reshape(n, c["hq"]))


def _beam(s):
    c = s["case"]
    n, w, vocab = c["reqs"], c["beams"], c["vocab"]
    x = s["logits"].double()  # 64 bits: candidates next to the border
    top = x.amax(-1, keepdim=True)
    cand = s["scores"].double()[..., None] + x - (top + (x - top).exp().sum(-1, keepdim=True).log())
    if s["finished"] is not None:
        ended = torch.full((vocab,), -math.inf, device="cuda", dtype=torch.float64)
        ended[7] = 0.0
        cand = torch.where(s["finished"][..., None], s["scores"].double()[..., None] + ended, cand)
    score, at = cand.view(n, w * vocab).sort(dim=-1, descending=True, stable=True)  # ties: the lowest first
    score, at = score[:, :c["out"]], at[:, :c["out"]]
    none = score == -math.inf
    token = torch.where(none, -1, at % vocab).int()
    parent = torch.where(none, -1, at // vocab + w * torch.arange(n, device="cuda")[:, None]).int()
    done = (token == 7) & ~none
    if s["finished"] is not None:
        done |= s["finished"].view(-1)[parent.clamp(min=0).long()] & ~none
    return dict(scores=score.float(), tokens=token, parents=parent, finished=done)


def _page_step(s):
    c, ps, pages = s["case"], s["case"]["page"], s["k"].shape[0]
    # fork: row i continues its parent's
    parent = s["parent"].long()
    table = s["table0"][parent]
    lens = s["lens0"].long()[parent]
    ids = torch.where(table < 0, pages, table).long()
    refs = torch.zeros(pages + 1, dtype=torch.int32, device="cuda").scatter_add_(0, ids.view(-1), torch.ones_like(ids.view(-1), dtype=torch.int32))[:pages]
    # reserve: pages for the new rows, the lowest free ones in row order; a shared page is left for an own copy
    starts = s["starts"].long()
    new = starts[1:] - starts[:-1]
    idx = torch.arange(table.shape[1], device="cuda")[None]
    touched = (idx >= (lens // ps)[:, None]) & (idx < (-(-(lens + new) // ps))[:, None]) & (new > 0)[:, None]
    shared = (table >= 0) & (refs[table.clamp(min=0).long()] > 1)
    need = touched & ((table < 0) | shared)
    count = need.sum(1)
    before = count.cumsum(0) - count
    free = refs == 0
    served = need & (before + count <= free.sum())[:, None]
    order = free.logical_not().to(torch.int8).sort(stable=True).indices  # free pages first, ascending
    fresh = order[(before[:, None] + need.cumsum(1) - 1).clamp(0, pages - 1)].int()
    row, col = (served & shared & (idx == (lens // ps)[:, None]) & (lens % ps > 0)[:, None]).nonzero(as_tuple=True)
    src, dst, live = table[row, col].long(), fresh[row, col].long(), (lens % ps)[row]
    mine = torch.arange(ps, device="cuda")[None] < live[:, None]
    at, r = mine.nonzero(as_tuple=True)
    s["k"][dst[at], r] = s["k"][src[at], r]
    s["v"][dst[at], r] = s["v"][src[at], r]
    left = table[served & shared].long()
    refs.scatter_add_(0, left, torch.full_like(left, -1, dtype=torch.int32))
    refs[fresh[served].long()] = 1
    table = torch.where(served, fresh, table)
    # where the new rows go
    ok = before + count <= free.sum()
    t = torch.arange(c["reqs"] * c["beams"], device="cuda")
    r = torch.searchsorted(starts[1:], t, right=True)
    p = lens[r] + t - starts[r]
    slot = table[r, p // ps].long() * ps + p % ps
    slot = torch.where(ok[r], slot, -1).int()
    position = torch.where(ok[r], p, 0).int()
    lens = torch.where(ok, lens + new, lens).int()
    s["table"].copy_(table)
    s["refs"].copy_(refs)
    s["lens"].copy_(lens)
    return dict(table=s["table"], refs=s["refs"], lens=s["lens"], slot=slot, position=position, k=s["k"].view(torch.int16),
                v=s["v"].view(torch.int16))


def _compact(s):
    refs, table = s["refs0"], s["table0"]
    pages = refs.shape[0]
    used = refs > 0
    count = used.sum()
    i = torch.arange(pages, device="cuda")
    src, dst = (used & (i >= count)).nonzero()[:, 0], (~used & (i < count)).nonzero()[:, 0]
    s["k"][dst] = s["k"][src]
    s["v"][dst] = s["v"][src]
    to = i.int()
    to[src] = dst.int()
    s["table"].copy_(torch.where(table < 0, table, to[table.clamp(min=0).long()]))
    s["refs"].copy_(refs)
    s["refs"][dst] = refs[src]
    s["refs"][src] = 0
    return dict(table=s["table"], refs=s["refs"], used=count.int().view(1), k=s["k"].view(torch.int16), v=s["v"].view(torch.int16))


# ------------------------------------------------------------------------------------- the framework's calls
def _own(s):
    import speculative_decoding_draft_rmsnorm_gb300 as lib
    c, op = s["case"], s["case"]["op"]
    if op == "rotary":
        how = dict(interleaved=c["inter"], inverse=c["inverse"], amplitude=s["amp"])
        if not c["store"]:
            q, k = lib.rotary(s["q"], s["pos"], s["freq"], k=s["k"], **how)
            return dict(q=q, k=k)
        q, _ = lib.rotary(s["q"], s["pos"], s["freq"], k=s["k"], k_out=s["k_store"], v=s["v"], v_out=s["v_store"], slot=s["slot"],
                          **how)
        return dict(q=q, k=s["k_store"], v=s["v_store"])
    if op == "decode":
        if "workspace" not in s:  # kept by a serving loop too: its size goes by the bounds alone
            s["workspace"] = lib.alloc_workspace(lib.decode_workspace_size(c["reqs"], c["hq"], c["hkv"], c["dh"], s["longest"], c["window"]))
        out, lse = lib.decode_attention_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], max_ctx_len=s["longest"],
                                              window=c["window"], out_dtype=lib.OUT_F32 if c["f32"] else lib.OUT_BF16,
                                              return_lse=True, workspace=s["workspace"])
        return dict(out=out, lse=lse)
    if op == "beam":
        return lib.beam_select(s["logits"], s["scores"], beams_out=c["out"], finished=s["finished"], eos=7)
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    pools = [s["k"], s["v"]]
    if op == "step":
        s["lens"].copy_(s["lens0"])
        lib.fork_pages(s["parent"], s["lens"], s["table"], s["refs"])
        slot, position = lib.reserve_pages(s["starts"], s["lens"], s["table"], s["refs"], pools, num_new=c["reqs"] * c["beams"],
                                           advance=True)
        return dict(table=s["table"], refs=s["refs"], lens=s["lens"], slot=slot, position=position, k=s["k"].view(torch.int16),
                    v=s["v"].view(torch.int16))
    used = lib.compact_pages(s["table"], s["refs"], pools)
    return dict(table=s["table"], refs=s["refs"], used=used, k=s["k"].view(torch.int16), v=s["v"].view(torch.int16))


def run(state):
    if own:
        return _own(state)
    return dict(rotary=_rotary, decode=_decode, beam=_beam, step=_page_step, compact=_compact)[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    c, op = case, case["op"]
    if op == "rotary":
        heads = c["hq"] + (2 if c["store"] else 1) * c["hkv"]
        return dict(bytes=2 * c["tokens"] * heads * c["dh"] * (4 if c["f32"] else 2) + 4 * c["tokens"] * (2 if c["store"] else 1),
                    flops=3 * c["tokens"] * (c["hq"] + c["hkv"]) * c["rd"])
    if op == "decode":
        lo, hi, w = c["lo"], c["hi"], c["window"]
        # the mean of the lengths that _lens draws; below the window the whole length is read
        mean = (hi - lo) / math.log(hi / lo) if hi > lo else hi
        rows = hi + (c["reqs"] - 1) * mean
        if w:
            if lo >= w:
                rows = c["reqs"] * w
            elif hi > w:
                short = math.log(w / lo) / math.log(hi / lo)
                rows = w + (c["reqs"] - 1) * (short * (w - lo) / math.log(w / lo) + (1 - short) * w)
        out = c["reqs"] * c["hq"] * c["dh"]
        return dict(bytes=4 * rows * c["hkv"] * c["dh"] + 4 * rows / c["page"] + out * (6 if c["f32"] else 4) + 4 * out / c["dh"],
                    flops=4 * rows * c["hq"] * c["dh"])
    if op == "beam":
        n = c["reqs"] * c["beams"] * c["vocab"]
        return dict(bytes=n * (4 if c["f32"] else 2) + 16 * c["reqs"] * c["out"], flops=4 * n)
    row = 2 * 2 * c["hkv"] * c["dh"]  # K and V of one row
    if op == "step":
        rows = c["reqs"] * c["beams"]
        width = -(-c["hi"] // c["page"]) + 2
        shared = 1 - (1 - 1 / c["beams"]) ** (c["beams"] - 1)  # a row whose parent another row continues too
        mean = (c["hi"] - c["lo"]) / math.log(c["hi"] / c["lo"]) if c["hi"] > c["lo"] else c["hi"]
        pages = c["reqs"] * mean / c["page"] + rows * 2.5
        # tables read and written, counts read, live rows of the shared last pages copied
        return dict(bytes=8 * rows * width + 4 * pages + 2 * row * rows * shared * (c["page"] - 1) / 2, flops=rows * width)
    moved = c["pages"] * c["used"] * (1 - c["used"])
    return dict(bytes=8 * c["pages"] * c["used"] + 8 * c["pages"] + 2 * moved * c["page"] * row, flops=c["pages"])


# ------------------------------------------------------------------------------------- 64-bit values
def exact(case, seed):
    op = case["op"]
    if op in ("step", "compact"):
        return None  # counts, tables and copied bits: nothing is computed in floating point
    s = prepare(case, seed)
    if op == "rotary":
        rd, t = case["rd"], case["tokens"]
        f = torch.tensor(list(s["freq"]), dtype=torch.float64, device="cuda")
        turn = torch.polar(torch.full((t, 1, rd // 2), float(s["amp"]), dtype=torch.float64, device="cuda"),
                           (s["pos"].double().view(t, 1, 1) * f) * (-1.0 if case["inverse"] else 1.0))

        def turned(x):
            y = x.double()
            z = y[..., :rd].unflatten(-1, (rd // 2, 2) if case["inter"] else (2, rd // 2))
            re, im = (z[..., 0], z[..., 1]) if case["inter"] else (z[..., 0, :], z[..., 1, :])
            z = torch.complex(re, im) * turn
            z = torch.stack((z.real, z.imag), dim=-1 if case["inter"] else -2).flatten(-2)
            y = y.clone()
            y[..., :rd] = z
            return y

        q, k = turned(s["q"]), turned(s["k"])
        if not case["store"]:
            return dict(q=q, k=k)
        ks, vs = s["k_store"].double(), s["v_store"].double()
        slot = s["slot"].tolist()
        rows = [i for i, x in enumerate(slot) if x >= 0]
        to = [slot[i] for i in rows]
        ks[to], vs[to] = k[rows], s["v"][rows].double()
        return dict(q=q, k=ks, v=vs)
    if op == "decode":
        out = torch.empty(case["reqs"], case["hq"], case["dh"], dtype=torch.float64, device="cuda")
        lse = torch.empty(case["reqs"], case["hq"], dtype=torch.float64, device="cuda")
        for r, n in enumerate(s["lens"].tolist()):
            at = torch.arange(max(0, n - case["window"]) if case["window"] else 0, n, device="cuda")
            page, off = s["table"][r][at // case["page"]].long(), at % case["page"]
            for h in range(case["hkv"]):
                k, v = s["k"][page, off, h].double(), s["v"][page, off, h].double()
                g = case["hq"] // case["hkv"]
                a = s["q"][r, h * g:(h + 1) * g].double() @ k.T * case["dh"] ** -0.5
                out[r, h * g:(h + 1) * g] = torch.softmax(a, -1) @ v
                lse[r, h * g:(h + 1) * g] = torch.logsumexp(a, -1)
        return dict(out=out, lse=lse)
    best = []
    for r in range(case["reqs"]):
        x = s["logits"][r].double()
        x = torch.log_softmax(x, -1)
        if s["finished"] is not None:
            for b, f in enumerate(s["finished"][r].tolist()):
                if f:
                    x[b] = -math.inf
                    x[b, 7] = 0.0
        best.append(torch.topk((x + s["scores"][r].double()[:, None]).view(-1), case["out"]).values)
    return dict(scores=torch.stack(best), tokens=None, parents=None, finished=None)
