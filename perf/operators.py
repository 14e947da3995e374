"""Sliding-window attention with sinks, and the paged cache it is served from:
the cases that are measured, in plain torch and through the library.

A query at position t sees key j iff j <= t and (j > t - window or j < sinks).

kind "prompt": the forward of dense sequences (output and log-sum-exp).
kind "train":  the forward and the backward (also dq, dk, dv).
kind "append": rotary positions on the queries and keys of new tokens, and their
               K and V rows into the pages of a cache (ragged sequences).
kind "attend": the new tokens' queries over the paged cache (ragged sequences,
               from one token each to long chunks of a prompt).
"""
import random

import torch

own = False


# ------------------------------------------------------------------ the cases
def _dense(name, kind, B, T, heads, kv_heads, hd, window, sinks):
    return {"name": name, "kind": kind, "B": B, "T": T, "heads": heads, "kv_heads": kv_heads,
            "hd": hd, "window": window, "sinks": sinks}


def _paged(name, kind, seqs, chunks, chunk, longest, heads, kv_heads, hd, window, sinks, page):
    """`seqs` sequences of up to `longest` tokens in the cache; `chunks` of them
    bring up to `chunk` new tokens each and the others one."""
    return {"name": name, "kind": kind, "seqs": seqs, "chunks": chunks, "chunk": chunk,
            "longest": longest, "heads": heads, "kv_heads": kv_heads, "hd": hd,
            "window": window, "sinks": sinks, "page": page}


def listed():
    return [
        # two short sequences, odd length: latency of one call
        _dense("prompt_short", "prompt", 2, 300, 4, 2, 64, 48, 4),
        # the SmolLM2-360M layer shape at 16K tokens, its teacher window
        _dense("prompt_16k", "prompt", 1, 16384, 15, 5, 64, 4096, 4),
        # the Qwen3-0.6B layer shape at 64K tokens, its teacher window
        _dense("prompt_64k", "prompt", 1, 65536, 16, 8, 128, 8192, 4),
        # a small training step: odd length, a window that is no multiple of a tile
        _dense("train_short", "train", 2, 700, 4, 2, 64, 300, 5),
        # training at the two layer shapes
        _dense("train_16k", "train", 1, 16384, 15, 5, 64, 4096, 4),
        _dense("train_32k", "train", 1, 32768, 16, 8, 128, 8192, 16),
        # one decode step of a small batch, and prompts of several lengths at once
        _paged("append_step", "append", 8, 0, 1, 16384, 16, 8, 128, 8192, 4, 64),
        _paged("append_prompts", "append", 6, 6, 4096, 4096, 16, 8, 128, 8192, 4, 64),
        # decode of one sequence past its window, and of a batch of 64
        _paged("decode_one", "attend", 1, 0, 1, 65536, 16, 8, 128, 8192, 4, 64),
        _paged("decode_64", "attend", 64, 0, 1, 65536, 16, 8, 128, 8192, 4, 64),
        # chunks of long prompts
        _paged("chunked_prompt", "attend", 4, 4, 2048, 65536, 16, 8, 128, 8192, 4, 64),
        # a continuous batch: decode steps with two chunks among them, small pages
        _paged("mixed_batch", "attend", 26, 2, 700, 32768, 15, 5, 64, 4096, 4, 16),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["prompt", "train", "append", "attend", "attend"])
    kv = rng.choice([1, 2, 4, 5, 8])
    heads = kv * rng.choice([1, 2, 3, 4])
    hd = rng.choice([64, 128])
    sinks = rng.choice([0, 1, 4, 4, 16, 64, 128])
    window = _log(rng, 32, 8192)
    if kind in ("prompt", "train"):
        T = _log(rng, 100, 24000)
        B = 1 if T > 6000 else rng.choice([1, 2, 3])
        return {k: v for k, v in _dense("", kind, B, T, heads, kv, hd, window, sinks).items()
                if k != "name"}
    page = rng.choice([16, 32, 64, 128])
    if kind == "append":
        seqs = _log(rng, 1, 64)
        chunks = rng.randint(0, min(seqs, 6))
        c = _paged("", kind, seqs, chunks, _log(rng, 2, 2048), _log(rng, 2048, 65536), heads, kv,
                   hd, window, sinks, page)
    else:
        seqs = _log(rng, 1, 48)
        chunks = rng.choice([0, 0, 1, min(seqs, 3)])
        c = _paged("", kind, seqs, chunks, _log(rng, 2, 1500), _log(rng, 2048, 65536), heads, kv,
                   hd, window, sinks, page)
    return {k: v for k, v in c.items() if k != "name"}


def _lengths(case):
    """(new tokens, tokens in the cache with them) of each sequence of a paged
    case: drawn from the case, so that the work is known without the inputs."""
    rng = random.Random("%(seqs)d %(chunks)d %(chunk)d %(longest)d %(window)d" % case)
    new, total = [], []
    for s in range(case["seqs"]):
        n = 1 if s >= case["chunks"] else rng.randint((case["chunk"] + 1) // 2, case["chunk"])
        # half of the sequences are near the longest, the others anywhere
        least = max(n, case["longest"] // (2 if s % 2 == 0 else 64))
        new.append(n)
        total.append(rng.randint(least, max(least, case["longest"])))
    order = list(range(case["seqs"]))
    rng.shuffle(order)
    return [new[i] for i in order], [total[i] for i in order]


def _first_page(case, n, total):
    """First page of the window of a sequence's first new token."""
    return max(0, total - n - case["window"] + 1) // case["page"]


def _seen(t, window, sinks):
    """Keys that position t sees."""
    return min(t + 1, window) + min(sinks, max(0, t + 1 - window))


def _pairs(first, n, window, sinks):
    """Visible (query, key) pairs of the positions first .. first + n - 1."""
    return sum(_seen(t, window, sinks) for t in range(first, first + n))


def work(case):
    hq, hkv, hd = case["heads"], case["kv_heads"], case["hd"]
    w, sinks = case["window"], case["sinks"]
    if case["kind"] in ("prompt", "train"):
        rows = case["B"] * case["T"]
        pairs = case["B"] * _pairs(0, case["T"], w, sinks) * hq
        data = rows * (2 * hq + 2 * hkv) * hd * 2 + rows * hq * 4
        if case["kind"] == "prompt":
            return {"bytes": data, "flops": 4 * hd * pairs}
        # dO in; dq, dk, dv out
        return {"bytes": data + rows * (2 * hq + 2 * hkv) * hd * 2, "flops": 14 * hd * pairs}
    new, total = _lengths(case)
    if case["kind"] == "append":
        rows = sum(new)
        return {"bytes": 2 * rows * (hq + 2 * hkv) * hd * 2, "flops": 3 * rows * (hq + hkv) * hd}
    keys = sum(min(L, n + w - 1) + min(sinks, max(0, L - (n + w - 1))) for n, L in zip(new, total))
    pairs = sum(_pairs(L - n, n, w, sinks) for n, L in zip(new, total)) * hq
    return {"bytes": keys * 2 * hkv * hd * 2 + sum(new) * hq * (hd * 4 + 4),
            "flops": 4 * hd * pairs}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    hq, hkv, hd = case["heads"], case["kv_heads"], case["hd"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16)

    # Queries share a direction and the keys of the first tokens carry it (about
    # 6 on their scores), so that the sinks draw a part of the weight, as they do
    # in a trained model.
    lean = torch.randn(hkv, hd, generator=g, device=dev)
    lean = lean / lean.norm(dim=-1, keepdim=True) * 2.4 * hd ** 0.25
    s = dict(case)
    if case["kind"] in ("prompt", "train"):
        B, T = case["B"], case["T"]
        s["q"] = (normal(B, T, hq, hd) + lean.repeat_interleave(hq // hkv, 0)).bfloat16()
        s["k"], s["v"] = normal(B, T, hkv, hd), normal(B, T, hkv, hd)
        s["k"][:, : case["sinks"]] += lean.bfloat16()
        if case["kind"] == "train":
            s["d_o"] = normal(B, T, hq, hd)
        return s
    new, total = _lengths(case)
    page, w, sinks = case["page"], case["window"], case["sinks"]
    # pages that the call touches: the sinks' (attend only) and those from the
    # window of the first new token on; the pages between them were given back
    held = []
    for n, L in zip(new, total):
        first = (L - n) // page if case["kind"] == "append" else _first_page(case, n, L)
        kept = [] if case["kind"] == "append" else range(min(first, -(-sinks // page)))
        held.append([*kept, *range(first, -(-L // page))])
    n_pages = sum(len(h) for h in held) + 3
    at = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32).cpu()
    table = torch.full((case["seqs"], max(-(-L // page) for L in total)), -1, dtype=torch.int32)
    used = 0
    for i, h in enumerate(held):
        table[i, torch.tensor(h)] = at[used:used + len(h)]
        used += len(h)
    s["new"], s["total"] = new, total
    s["table"] = table.to(dev)
    s["q_start"] = torch.tensor([0, *torch.tensor(new).cumsum(0).tolist()], dtype=torch.int32,
                                device=dev)
    s["kv_len"] = torch.tensor(total, dtype=torch.int32, device=dev)
    s["k_pages"], s["v_pages"] = normal(n_pages, hkv, page, hd), normal(n_pages, hkv, page, hd)
    rows = sum(new)
    if case["kind"] == "append":
        s["qkv"] = normal(rows, (hq + 2 * hkv) * hd)
        s["theta"] = 10000.0
        return s
    s["q"] = (normal(rows, hq, hd) + lean.repeat_interleave(hq // hkv, 0)).bfloat16()
    if sinks:
        first = s["table"][:, 0].long()
        s["k_pages"][first[first >= 0], :, : min(sinks, page)] += lean.bfloat16()[:, None]
    return s


# ------------------------------------------------------------------ plain forms
def _scores(q, k, q_pos, k_pos, window, sinks, scale):
    """Masked scores [B, Hkv, G, m, n] of q [B, m, Hq, hd] and k [B, n, Hkv, hd],
    both in 32 bits; q_pos [B, m] and k_pos [B, n] are positions, -1 for no key."""
    B, m, hq, hd = q.shape
    hkv = k.shape[2]
    qg = q.view(B, m, hkv, hq // hkv, hd).permute(0, 2, 3, 1, 4)
    s = torch.matmul(qg, k.permute(0, 2, 3, 1)[:, :, None]) * scale
    t, j = q_pos[:, :, None], k_pos[:, None, :]
    sees = (j >= 0) & (j <= t) & ((j > t - window) | (j < sinks))
    return torch.where(sees[:, None, None], s, float("-inf"))


def _softmax(s):
    top = s.amax(-1, keepdim=True)
    e = (s - top).exp()
    total = e.sum(-1, keepdim=True)
    return e / total, (top + total.log())[..., 0]


def _rows(x):
    """[B, Hkv, G, m, hd] to [B, m, Hq, hd]."""
    B, hkv, G, m, hd = x.shape
    return x.permute(0, 3, 1, 2, 4).reshape(B, m, hkv * G, hd)


def _plain_dense(s):
    """Blocks of queries, each over the keys it can see, so that 64K tokens fit."""
    B, T, w, sinks = s["B"], s["T"], s["window"], s["sinks"]
    hq, hkv, hd = s["heads"], s["kv_heads"], s["hd"]
    G, scale = hq // hkv, hd ** -0.5
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    train = s["kind"] == "train"
    at = torch.arange(T, device=q.device)
    o, lse = torch.empty_like(q), q.new_empty(B, hq, T)
    if train:
        d_o = s["d_o"].float()
        dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for a in range(0, T, 1024):
        b, lo = min(T, a + 1024), max(0, a - w + 1)
        keys = torch.cat([at[:min(sinks, lo)], at[lo:b]])
        kk, vv = k[:, keys], v[:, keys]
        p, l = _softmax(_scores(q[:, a:b], kk, at[None, a:b], keys[None], w, sinks, scale))
        vt = vv.permute(0, 2, 1, 3)[:, :, None]
        ob = torch.matmul(p, vt)
        o[:, a:b], lse[:, :, a:b] = _rows(ob), l.reshape(B, hq, b - a)
        if train:
            g = d_o[:, a:b].view(B, b - a, hkv, G, hd).permute(0, 2, 3, 1, 4)
            qb = q[:, a:b].view(B, b - a, hkv, G, hd).permute(0, 2, 3, 1, 4)
            delta = (g * ob).sum(-1, keepdim=True)
            ds = p * (torch.matmul(g, vt.transpose(-1, -2)) - delta) * scale
            dq[:, a:b] = _rows(torch.matmul(ds, kk.permute(0, 2, 1, 3)[:, :, None]))
            dk.index_add_(1, keys, torch.matmul(ds.transpose(-1, -2), qb).sum(2).transpose(1, 2))
            dv.index_add_(1, keys, torch.matmul(p.transpose(-1, -2), g).sum(2).transpose(1, 2))
    out = (o.bfloat16(), lse)
    return (*out, dq.bfloat16(), dk.bfloat16(), dv.bfloat16()) if train else out


def _positions(s):
    return torch.cat([torch.arange(L - n, L) for n, L in zip(s["new"], s["total"])])


def _slots(s, seq, pos):
    """(page, row in the page) of positions of sequences; page -1 where none is held."""
    return s["table"][seq, pos // s["page"]].long(), pos % s["page"]


def _rotate(x, pos, theta):
    """Rotate-half rotary positions of x [n, H, hd] in 32 bits, angles in 64."""
    half = x.shape[-1] // 2
    freq = theta ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    angle = pos.double()[:, None] * freq
    c, sn = angle.cos().float()[:, None], angle.sin().float()[:, None]
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * sn, b * c + a * sn], -1)


def _plain_append(s):
    hq, hkv, hd = s["heads"], s["kv_heads"], s["hd"]
    dev = s["qkv"].device
    pos = _positions(s).to(dev)
    seq = torch.repeat_interleave(torch.arange(len(s["new"]), device=dev), torch.tensor(s["new"], device=dev))
    x = s["qkv"].float().view(-1, hq + 2 * hkv, hd)
    qk = _rotate(x[:, :hq + hkv], pos, s["theta"]).bfloat16()
    page, row = _slots(s, seq, pos)
    s["k_pages"][page, :, row] = qk[:, hq:]
    s["v_pages"][page, :, row] = s["qkv"].view(-1, hq + 2 * hkv, hd)[:, hq + hkv:]
    return qk[:, :hq].contiguous(), s["k_pages"], s["v_pages"]


def _plain_attend(s):
    """Sequences with as many new tokens as one another go together."""
    w, sinks, dev = s["window"], s["sinks"], s["q"].device
    hq, hd = s["heads"], s["hd"]
    scale = hd ** -0.5
    o, lse = torch.empty_like(s["q"]), torch.empty(hq, len(s["q"]), device=dev)
    for n in sorted(set(s["new"])):
        ids = torch.tensor([i for i, m in enumerate(s["new"]) if m == n], device=dev)
        span = min(n + w - 1, max(L for L, m in zip(s["total"], s["new"]) if m == n))
        end = s["kv_len"][ids].long()[:, None]
        # the sinks before the span, then the span that ends at the last token
        back = end - span + torch.arange(span, device=dev)
        front = torch.arange(sinks, device=dev).expand(len(ids), sinks)
        k_pos = torch.cat([torch.where(front < end - span, front, -1), back.clamp(min=-1)], 1)
        q_pos = end - n + torch.arange(n, device=dev)
        page, row = _slots(s, ids[:, None], k_pos.clamp(min=0))
        rows = s["q_start"][ids].long()[:, None] + torch.arange(n, device=dev)
        k = s["k_pages"][page, :, row].float()
        v = s["v_pages"][page, :, row].float()
        p, l = _softmax(_scores(s["q"][rows].float(), k, q_pos, k_pos, w, sinks, scale))
        o[rows] = _rows(torch.matmul(p, v.permute(0, 2, 1, 3)[:, :, None])).bfloat16()
        lse[:, rows] = l.reshape(len(ids), hq, n).transpose(0, 1)
    return o, lse


# ------------------------------------------------------------------ the calls
def run(state):
    kind = state["kind"]
    if not own:
        return {"append": _plain_append, "attend": _plain_attend}.get(kind, _plain_dense)(state)
    import dual_window_attention_b200 as ttcd
    s = state
    if kind in ("prompt", "train"):
        o, lse = ttcd.sink_window_attn(s["q"], s["k"], s["v"], s["window"], s["sinks"], lse=True)
        if kind == "prompt":
            return o, lse
        dq, dk, dv, _ = ttcd.sink_window_attn_backward(s["q"], s["k"], s["v"], o, lse, s["d_o"],
                                                       s["window"], s["sinks"])
        return o, lse, dq, dk, dv
    if kind == "append":
        q = ttcd.paged_kv_append(s["qkv"], s["k_pages"], s["v_pages"], s["table"], s["q_start"],
                                 s["kv_len"], s["heads"], rope_theta=s["theta"])
        return q, s["k_pages"], s["v_pages"]
    return ttcd.paged_window_attn(s["q"], s["k_pages"], s["v_pages"], s["table"], s["q_start"],
                                  s["kv_len"], s["window"], s["sinks"], max_q=max(s["new"]),
                                  lse=True)


# ------------------------------------------------------------------ 64 bits
def _exact_attention(q, k, v, t, j, window, sinks):
    """One head: q [m, hd] at positions t, k and v [n, hd] at positions j."""
    hidden = (j[None] > t[:, None]) | ((j[None] <= t[:, None] - window) & (j[None] >= sinks))
    s = (q @ k.T / q.shape[-1] ** 0.5).masked_fill(hidden, float("-inf"))
    return torch.softmax(s, -1) @ v, torch.logsumexp(s, -1)


def _exact_dense(s):
    B, T, w, sinks = s["B"], s["T"], s["window"], s["sinks"]
    hq, hkv = s["heads"], s["kv_heads"]
    train = s["kind"] == "train"
    q, k, v = (s[n].double().requires_grad_(train) for n in "qkv")
    o = torch.empty_like(q, requires_grad=False)
    lse = o.new_empty(B, hq, T)
    grads = [torch.zeros_like(x, requires_grad=False) for x in (q, k, v)]
    at = torch.arange(T, device=o.device)
    for b in range(B):
        for h in range(hq):
            g = h * hkv // hq
            for a in range(0, T, 2048):
                e = min(T, a + 2048)
                j = at[:e][(at[:e] > a - w) | (at[:e] < sinks)]
                x = [y.detach().requires_grad_(train) for y in (q[b, a:e, h], k[b, j, g], v[b, j, g])]
                ob, l = _exact_attention(*x, at[a:e], j, w, sinks)
                o[b, a:e, h], lse[b, h, a:e] = ob.detach(), l.detach()
                if train:
                    dq, dk, dv = torch.autograd.grad(ob, x, s["d_o"][b, a:e, h].double())
                    grads[0][b, a:e, h] = dq
                    grads[1][b, :, g].index_add_(0, j, dk)
                    grads[2][b, :, g].index_add_(0, j, dv)
    return (o, lse, *grads) if train else (o, lse)


def _exact_append(s):
    hq, hkv, hd = s["heads"], s["kv_heads"], s["hd"]
    x = s["qkv"].double().view(-1, hq + 2 * hkv, hd)
    pages = [s["k_pages"].double(), s["v_pages"].double()]
    pos = _positions(s).double().to(x.device)
    # the pair (i, i + hd/2) is a complex number turned by pos * theta^(-2i/hd)
    i = torch.arange(hd // 2, device=x.device, dtype=torch.float64)
    turn = torch.polar(torch.ones_like(i)[None].expand(len(x), -1),
                       pos[:, None] * torch.exp(-2 * i / hd * torch.tensor(s["theta"]).double().log()))
    z = torch.complex(x[..., :hd // 2], x[..., hd // 2:]) * turn[:, None]
    turned = torch.cat([z.real, z.imag], -1)
    table, row = s["table"].tolist(), 0
    for seq, (n, L) in enumerate(zip(s["new"], s["total"])):
        for p in range(L - n, L):
            page = table[seq][p // s["page"]]
            pages[0][page, :, p % s["page"]] = turned[row, hq:hq + hkv]
            pages[1][page, :, p % s["page"]] = x[row, hq + hkv:]
            row += 1
    return turned[:, :hq].contiguous(), *pages


def _exact_attend(s):
    hq, hkv, w, sinks = s["heads"], s["kv_heads"], s["window"], s["sinks"]
    o = s["q"].double()
    lse = o.new_empty(hq, len(o))
    row = 0
    for seq, (n, L) in enumerate(zip(s["new"], s["total"])):
        at = torch.arange(L, device=o.device)
        j = at[(at > L - n - w) | (at < sinks)]
        page, r = s["table"][seq, j // s["page"]].long(), j % s["page"]
        k, v = s["k_pages"][page, :, r].double(), s["v_pages"][page, :, r].double()
        for h in range(hq):
            g = h * hkv // hq
            x = _exact_attention(o[row:row + n, h].clone(), k[:, g], v[:, g], at[L - n:], j, w, sinks)
            o[row:row + n, h], lse[h, row:row + n] = x
        row += n
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    with torch.set_grad_enabled(case["kind"] == "train"):
        return {"append": _exact_append, "attend": _exact_attend}.get(case["kind"], _exact_dense)(s)
