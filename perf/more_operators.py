"""A layer's step for sequences that share a prompt: what is measured, and the plain forms.

Four operators: attention of one new token per sequence in which the rows that a group of sequences
shares are read once for all, the extent of that sharing from the page tables, rotary positions over
several axes, and the RMS norm with the residual's addition and an output in 8 bits.
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # four beams of one request of the 0.6B-shaped layer, just past its prompt: latency
        dict(name="shared 1x4", op="shared", groups=1, per=4, hq=16, hkv=8, dh=128, lo=700, hi=700, mine=20, page=16, window=0, f32=False),
        # a beam search: 32 requests of 8 beams, prompts of 512 to 8192 rows
        dict(name="shared 32x8", op="shared", groups=32, per=8, hq=32, hkv=8, dh=128, lo=512, hi=8192, mine=64, page=16, window=0,
             f32=False),
        # one long prompt with 64 samples drawn from it
        dict(name="shared 1x64 long", op="shared", groups=1, per=64, hq=32, hkv=8, dh=128, lo=32000, hi=32000, mine=1000, page=16,
             window=0, f32=False),
        # a window layer, f32 output, 64-row pages, groups of 5
        dict(name="shared window f32", op="shared", groups=16, per=5, hq=32, hkv=8, dh=128, lo=9000, hi=16384, mine=300, page=64,
             window=4096, f32=True),
        # 256 sequences on one prompt: the products bound it, not the reads
        dict(name="shared 1x256", op="shared", groups=1, per=256, hq=32, hkv=8, dh=128, lo=16384, hi=16384, mine=200, page=16, window=0,
             f32=False),
        # how far the beams of 32 requests still share their pages
        dict(name="prefixes 32x8", op="prefixes", groups=32, per=8, lo=512, hi=8192, mine=64, page=16),
        # 256 sequences on one prompt of 8000 to 32000 rows
        dict(name="prefixes 1x256", op="prefixes", groups=1, per=256, lo=8000, hi=32000, mine=200, page=16),
        # one decode step of 32 sequences: q, k, v from the fused projection, k and v to store slots
        dict(name="axes decode 32", op="axes", tokens=32, hq=32, hkv=8, dh=128, sections="16,24,24", mixed=False, inter=False,
             f32=False, inverse=False, store=16),
        # the gradient over 16384 tokens of pictures and text, axes dealt out pair by pair
        dict(name="axes gradient", op="axes", tokens=16384, hq=32, hkv=8, dh=128, sections="24,20,20", mixed=True, inter=False,
             f32=False, inverse=True, store=0),
        # one token of the 4B-shaped layer: latency
        dict(name="norm 1", op="norm", rows=1, cols=2560, f32=False, residual=True, eight=True, group=0),
        # an odd width in f32, 8 bits for every 128 columns
        dict(name="norm odd f32", op="norm", rows=333, cols=5003, f32=True, residual=True, eight=True, group=128),
        # a prompt chunk
        dict(name="norm 16384", op="norm", rows=16384, cols=5120, f32=False, residual=True, eight=True, group=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "shared", "prefixes", "axes", "axes", "norm", "norm"])
    if op == "shared":
        hkv = rng.choice([1, 2, 4, 8])
        g = rng.choice([1, 2, 4, 4, 5, 8, 16])
        dh = rng.choice([64, 128, 128])
        f32 = rng.random() < 0.3
        groups = _log(rng, 1, 64)
        per = _log(rng, 1, 256 // groups)
        heavy = (4 if g > 4 else 1) * (2 if f32 else 1)
        hi = _log(rng, 1, max(1, min(40000, 256 * 13000 * 1024 // (groups * per * hkv * dh * heavy), 8 * 16384 * 1024 // (groups * hkv * dh))))
        mine = _log(rng, 1, max(1, min(1000, hi // 4, 256 * 300 * 1024 // (groups * per * hkv * dh))))
        return dict(op=op, groups=groups, per=per, hq=hkv * g, hkv=hkv, dh=dh, lo=max(1, int(hi * rng.choice([0.05, 0.5, 1.0]))), hi=hi,
                    mine=mine, page=rng.choice([16, 16, 24, 32, 64]), window=rng.choice([0, 0, 0, _log(rng, 1, 8192)]), f32=f32)
    if op == "prefixes":
        groups = _log(rng, 1, 256)
        hi = _log(rng, 2000, 40000)
        per = _log(rng, 1, max(1, min(256, 1024 // groups, 256 * 32000 // (groups * hi))))
        return dict(op=op, groups=groups, per=per, lo=max(1, int(hi * rng.choice([0.05, 0.5]))), hi=hi,
                    mine=_log(rng, 1, 1000), page=rng.choice([16, 16, 24, 32, 64]))
    if op == "axes":
        dh = rng.choice([64, 80, 96, 128, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 5, 8])
        n = rng.choice([2, 3, 3, 4])
        pairs = rng.choice([dh // 2, dh // 2, dh // 4])
        cut = sorted(rng.sample(range(1, pairs), n - 1))
        f32 = rng.random() < 0.3
        inverse = rng.random() < 0.3
        most = max(1, 16384 * 40 * 128 // ((hq + 2 * hkv) * dh * (2 if f32 else 1)))
        sections = ",".join(str(b - a) for a, b in zip([0] + cut, cut + [pairs]))
        return dict(op=op, tokens=_log(rng, 1, most), hq=hq, hkv=hkv, dh=dh, sections=sections, mixed=rng.random() < 0.5, inter=rng.random() < 0.5, f32=f32, inverse=inverse,
                    store=0 if inverse else rng.choice([0, 0, 16, 5]))
    cols = rng.choice([1024, 2560, 4096, 5120, 8192, _log(rng, 16, 16384), _log(rng, 16, 16384)])
    f32 = rng.random() < 0.3
    eight = rng.random() < 0.7
    return dict(op=op, rows=_log(rng, 1, max(1, 16384 * 5120 // (cols * (2 if f32 else 1)))), cols=cols, f32=f32,
                residual=rng.random() < 0.7, eight=eight, group=rng.choice([0, 0, 128, 64]) if eight else 0)


# ------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _dt(case):
    return torch.float32 if case["f32"] else torch.bfloat16


def _sequences(case, rng):
    """Lengths, page table, group bounds and prefixes of sequences that share their group's prompt.

    The sequences of a group hold the prompt's full pages together and the rest each for itself, as
    fork and reserve leave them; all have `mine` rows of their own to within a few."""
    n, per, ps = case["groups"], case["per"], case["page"]
    prompt = np.exp(rng.uniform(math.log(case["lo"]), math.log(case["hi"] + 0.999), n)).astype(np.int64).clip(case["lo"], case["hi"])
    if case["op"] == "shared":
        prompt[0] = case["hi"]
    grown = 1 + rng.integers(case["mine"] // 2, case["mine"] + 1, (n, per))
    full = prompt // ps if per > 1 else -(-(prompt + grown[:, 0]) // ps)  # pages of the whole group
    lens = prompt[:, None] + grown
    held = -(-lens // ps)
    width = -(-(case["hi"] + case["mine"] + 1) // ps) + 1
    pages = int(n * -(-(case["hi"] + case["mine"] + 1) // ps) + n * per * (-(-(case["mine"] + 1) // ps) + 2)) + 3  # whatever was drawn
    ids = rng.permutation(pages).astype(np.int32)
    table, at = np.full((n, per, width), -1, np.int32), 0
    for g in range(n):
        table[g, :, :full[g]] = ids[at:at + full[g]]
        at += int(full[g])
        for i in range(per):
            more = max(0, int(held[g, i] - full[g]))
            table[g, i, full[g]:full[g] + more] = ids[at:at + more]
            at += more
    shared = np.minimum(full * ps, lens.min(1))
    return lens.reshape(-1), table.reshape(n * per, width), shared, pages


def _sections(case):
    return [int(n) for n in case["sections"].split(",")]


def _axes_of(case):
    """The axis of every pair: sections one after the other, or dealt out in turn."""
    left = _sections(case)
    if not case["mixed"]:
        return np.repeat(np.arange(len(left)), left)
    out, pairs = [], sum(left)
    while len(out) < pairs:
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return np.array(out)


def prepare(case, seed):
    g, rng = _gen(seed), np.random.default_rng(int(seed))
    op = case["op"]
    s = dict(case=case)
    if op == "norm":
        n, d = case["rows"], case["cols"]
        s["x"] = torch.randn(n, d, device="cuda", generator=g).to(_dt(case))
        # the residual stream is larger than what a layer adds, and a few of its columns are far larger
        stream = 4 * torch.randn(n, d, device="cuda", generator=g)
        stream[:, torch.randint(0, d, (max(1, d // 500),), device="cuda", generator=g)] *= 30
        s["residual"] = stream.to(_dt(case)) if case["residual"] else None
        s["weight"] = (1 + 0.3 * torch.randn(d, device="cuda", generator=g)).to(torch.bfloat16)
        return s
    if op == "axes":
        t, hq, hkv, dh = case["tokens"], case["hq"], case["hkv"], case["dh"]
        x = torch.randn(t, hq + 2 * hkv, dh, device="cuda", generator=g).to(_dt(case))
        s.update(q=x[:, :hq], k=x[:, hq:hq + hkv], v=x[:, hq + hkv:])
        # text counts all axes up together; a picture keeps the first and runs its grid through the others
        pos, at, now = np.zeros((len(_sections(case)), t), np.int64), 0, int(rng.integers(0, 30000))
        while at < t:
            text = int(rng.integers(1, 200))
            n = min(text, t - at)
            pos[:, at:at + n] = now + np.arange(n)
            at, now = at + n, now + n
            high, wide = (int(v) for v in rng.integers(4, 48, 2))
            n = min(high * wide, t - at)
            cell = np.arange(n)
            pos[:, at:at + n] = now
            if len(pos) > 1:
                pos[-1, at:at + n] += cell % wide
            if len(pos) > 2:
                pos[-2, at:at + n] += cell // wide
            at, now = at + n, now + max(high, wide)
        s["pos"] = torch.from_numpy(pos.astype(np.int32)).cuda()
        s["axes"] = _axes_of(case)
        pairs = sum(_sections(case))
        s["freq"] = 1e6 ** (-np.arange(pairs, dtype=np.float64) / pairs)
        if case["store"]:
            rows = (t + 7) // case["store"] * case["store"] + 2 * case["store"]
            s["k_store"] = torch.zeros(rows, hkv, dh, device="cuda", dtype=_dt(case))
            s["v_store"] = torch.zeros_like(s["k_store"])
            s["slot"] = torch.randperm(rows, device="cuda", generator=g)[:t].to(torch.int32)
            if t > 8:
                s["slot"][t - 3:] = -1  # padding rows of the batch
        return s
    lens, table, shared, pages = _sequences(case, rng)
    s["table"] = torch.from_numpy(table).cuda()
    s["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    s["starts"] = torch.arange(0, len(lens) + 1, case["per"], dtype=torch.int32, device="cuda")
    if op == "prefixes":
        return s
    s["prefix"] = torch.from_numpy(shared.astype(np.int32)).cuda()
    ps, hkv, dh = case["page"], case["hkv"], case["dh"]
    s["k"] = torch.randn(pages, ps, hkv, dh, device="cuda", generator=g, dtype=torch.bfloat16)
    s["v"] = torch.randn(pages, ps, hkv, dh, device="cuda", generator=g, dtype=torch.bfloat16)
    s["q"] = (1.5 * torch.randn(len(lens), case["hq"], dh, device="cuda", generator=g)).to(torch.bfloat16)
    s["longest"] = int(lens.max())
    return s


# ------------------------------------------------------------------------------------- plain forms
def _norm(s):
    c = s["case"]
    h = s["x"].float()
    if s["residual"] is not None:
        h = (h + s["residual"].float()).to(_dt(c)).float()  # the stream as it is stored
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * s["weight"].float()
    residual = h.to(_dt(c)) if s["residual"] is not None else None
    if not c["eight"]:
        return dict(out=y.to(_dt(c)), residual=residual) if residual is not None else dict(out=y.to(_dt(c)))
    n, d = y.shape
    each = c["group"] or d
    parts = -(-d // each)
    padded = torch.zeros(n, parts * each, device="cuda")
    padded[:, :d] = y
    scale = (padded.view(n, parts, each).abs().amax(-1) / 448).clamp(min=2.0 ** -126)
    out = (y / scale.repeat_interleave(each, 1)[:, :d]).to(torch.float8_e4m3fn)
    return dict(out=out, scale=scale, residual=residual) if residual is not None else dict(out=out, scale=scale)


def _rotated(x, cos, sin, c):
    rd = 2 * sum(_sections(c))
    x = x.float()
    a, b = (x[..., 0:rd:2], x[..., 1:rd:2]) if c["inter"] else (x[..., :rd // 2], x[..., rd // 2:rd])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, v), -1).flatten(-2) if c["inter"] else torch.cat((u, v), -1)
    return torch.cat((turned, x[..., rd:]), -1).to(_dt(c))


def _axes(s):
    c = s["case"]
    at = torch.from_numpy(s["axes"]).cuda()
    angle = s["pos"][at].double().T * torch.from_numpy(s["freq"]).cuda()  # 64 bits: far positions
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
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


def _prefixes(s):
    c = s["case"]
    table, lens, starts = s["table"], s["lens"].long(), s["starts"].long()
    n = starts.shape[0] - 1
    group = torch.searchsorted(starts[1:], torch.arange(table.shape[0], device="cuda"), right=True)
    first = starts[:-1][group]
    same = (table == table[first]) & (table >= 0)
    rows = torch.minimum(lens, same.int().cumprod(1).sum(1) * c["page"])
    out = torch.full((n,), 2 ** 31 - 1, device="cuda").scatter_reduce_(0, group, rows, "amin")
    return dict(prefix=out.int())


def _shared(s):
    c = s["case"]
    ps, hkv, dh, longest = c["page"], c["hkv"], c["dh"], s["longest"]
    total = c["groups"] * c["per"]
    span = min(longest, c["window"] or longest)
    each = max(1, min(total, 2 ** 28 // (span * hkv * max(dh, c["hq"] // hkv))))  # sequences at once: a few GB
    outs, sums = [], []
    for at in range(0, total, each):
        lens = s["lens"][at:at + each].long()
        n = lens.shape[0]
        first = (lens - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(lens)
        j = first[:, None] + torch.arange(span, device="cuda")[None]
        seen = j < lens[:, None]
        j = j.clamp(max=longest - 1)
        page = s["table"][at:at + each].gather(1, j // ps).long().clamp(min=0)
        k, v = s["k"][page, j % ps].float(), s["v"][page, j % ps].float()
        q = s["q"][at:at + each].float().view(n, hkv, c["hq"] // hkv, dh)
        score = torch.einsum("nhgd,nlhd->nhgl", q, k) / math.sqrt(dh)
        score = score.masked_fill(~seen[:, None, None], -math.inf)
        top = score.amax(-1, keepdim=True)
        p = (score - top).exp()
        mass = p.sum(-1, keepdim=True)
        out = torch.einsum("nhgl,nlhd->nhgd", p / mass, v.masked_fill(~seen[:, :, None, None], 0.0))
        outs.append(out.reshape(n, c["hq"], dh).to(_dt(c)))
        sums.append((top + mass.log()).reshape(n, c["hq"]))
    return dict(out=torch.cat(outs), lse=torch.cat(sums))


# ------------------------------------------------------------------------------------- the framework's calls
def _own(s):
    import speculative_decoding_draft_rmsnorm_gb300 as lib
    c, op = s["case"], s["case"]["op"]
    if op == "norm":
        out, residual, scale = lib.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=1e-6, group_size=c["group"],
                                            out_dtype=lib.OUT_E4M3 if c["eight"] else None)
        got = dict(out=out)
        if c["eight"]:
            got["scale"] = scale
        if s["residual"] is not None:
            got["residual"] = residual
        return got
    if op == "axes":
        how = dict(interleaved=c["inter"], inverse=c["inverse"])
        if not c["store"]:
            q, k = lib.rotary_axes(s["q"], s["pos"], s["axes"], s["freq"], k=s["k"], **how)
            return dict(q=q, k=k)
        q, _ = lib.rotary_axes(s["q"], s["pos"], s["axes"], s["freq"], k=s["k"], k_out=s["k_store"], v=s["v"], v_out=s["v_store"],
                               slot=s["slot"], **how)
        return dict(q=q, k=s["k_store"], v=s["v_store"])
    if op == "prefixes":
        return dict(prefix=lib.shared_prefixes(s["table"], s["lens"], s["starts"], page_size=c["page"]))
    if "workspace" not in s:  # kept by a serving loop too: its size goes by the bounds alone
        s["workspace"] = lib.alloc_workspace(lib.shared_workspace_size(c["groups"] * c["per"], c["groups"], c["hq"], c["hkv"], c["dh"],
                                                                       s["longest"], c["window"]))
    out, lse = lib.decode_attention_shared(s["q"], s["k"], s["v"], s["table"], s["lens"], s["starts"], s["prefix"],
                                           max_ctx_len=s["longest"], window=c["window"],
                                           out_dtype=lib.OUT_F32 if c["f32"] else lib.OUT_BF16, return_lse=True,
                                           workspace=s["workspace"])
    return dict(out=out, lse=lse)


def run(state):
    if own:
        return _own(state)
    return dict(norm=_norm, axes=_axes, prefixes=_prefixes, shared=_shared)[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------- what a pass cannot do without
def _mean_prompt(c):
    lo, hi = c["lo"], c["hi"]
    mean = (hi - lo) / math.log(hi / lo) if hi > lo else hi  # of the lengths that _sequences draws
    return mean if c["op"] == "prefixes" else (hi + (c["groups"] - 1) * mean) / c["groups"]


def work(case):
    c, op = case, case["op"]
    if op == "norm":
        n, e = c["rows"] * c["cols"], 4 if c["f32"] else 2
        scales = 4 * c["rows"] * -(-c["cols"] // (c["group"] or c["cols"])) if c["eight"] else 0
        return dict(bytes=n * (e + (2 * e if c["residual"] else 0) + (1 if c["eight"] else e)) + scales + 2 * c["cols"], flops=6 * n)
    if op == "axes":
        heads = c["hq"] + (2 if c["store"] else 1) * c["hkv"]
        return dict(bytes=2 * c["tokens"] * heads * c["dh"] * (4 if c["f32"] else 2) +
                    4 * c["tokens"] * (len(_sections(c)) + (1 if c["store"] else 0)),
                    flops=6 * c["tokens"] * (c["hq"] + c["hkv"]) * sum(_sections(c)))
    n = c["groups"] * c["per"]
    prompt, grown = _mean_prompt(c), 1 + 0.75 * c["mine"]
    if op == "prefixes":
        return dict(bytes=4 * n * (prompt / c["page"] + 1) + 4 * n + 4 * c["groups"], flops=n * prompt / c["page"])
    rows = prompt + grown  # of a sequence
    seen = min(rows, c["window"]) if c["window"] else rows
    mine = min(grown, seen)
    read = n * mine + c["groups"] * (seen - mine)
    out = n * c["hq"] * c["dh"]
    return dict(bytes=4 * read * c["hkv"] * c["dh"] + 4 * read / c["page"] + out * (6 if c["f32"] else 4) + 4 * out / c["dh"],
                flops=4 * n * seen * c["hq"] * c["dh"])


# ------------------------------------------------------------------------------------- 64-bit values
def exact(case, seed):
    op = case["op"]
    if op == "prefixes":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "norm":
        h = s["x"].double()
        got = {}
        if case["residual"]:
            got["residual"] = h + s["residual"].double()
            h = got["residual"].to(s["x"].dtype).double()  # normed as stored
        y = h / torch.linalg.vector_norm(torch.cat((h / case["cols"] ** 0.5, torch.full_like(h[:, :1], 1e-3)), 1), dim=1, keepdim=True)
        y = y * s["weight"].double()
        if not case["eight"]:
            return dict(out=y, **got)
        cut = y.split(case["group"] or case["cols"], dim=1)
        scale = [(p.abs().max(1, keepdim=True).values / 448).clamp(min=2.0 ** -126) for p in cut]
        return dict(out=torch.cat([p / q for p, q in zip(cut, scale)], 1), scale=torch.cat(scale, 1), **got)
    if op == "axes":
        t, pairs = case["tokens"], sum(_sections(case))
        angle = torch.empty(t, 1, pairs, dtype=torch.float64, device="cuda")
        for i, (a, f) in enumerate(zip(s["axes"].tolist(), s["freq"].tolist())):
            angle[:, 0, i] = s["pos"][a].double() * f
        turn = torch.polar(torch.ones_like(angle), -angle if case["inverse"] else angle)

        def turned(x):
            y = x.double()
            z = y[..., :2 * pairs].unflatten(-1, (pairs, 2) if case["inter"] else (2, pairs))
            re, im = (z[..., 0], z[..., 1]) if case["inter"] else (z[..., 0, :], z[..., 1, :])
            z = torch.complex(re, im) * turn
            z = torch.stack((z.real, z.imag), dim=-1 if case["inter"] else -2).flatten(-2)
            y = y.clone()
            y[..., :2 * pairs] = z
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
    n, g = case["groups"] * case["per"], case["hq"] // case["hkv"]
    out = torch.empty(n, case["hq"], case["dh"], dtype=torch.float64, device="cuda")
    lse = torch.empty(n, case["hq"], dtype=torch.float64, device="cuda")
    for r, length in enumerate(s["lens"].tolist()):
        at = torch.arange(max(0, length - case["window"]) if case["window"] else 0, length, device="cuda")
        page, off = s["table"][r][at // case["page"]].long(), at % case["page"]
        k, v = s["k"][page, off].double().transpose(0, 1), s["v"][page, off].double().transpose(0, 1)
        a = torch.matmul(s["q"][r].double().view(case["hkv"], g, case["dh"]), k.transpose(1, 2)) * case["dh"] ** -0.5
        out[r] = torch.matmul(torch.softmax(a, -1), v).view(case["hq"], case["dh"])
        lse[r] = torch.logsumexp(a, -1).view(case["hq"])
    return dict(out=out, lse=lse)
