"""Cases that measure the prompt and drafting operators around the ReplaySSM decode steps.

Four operators, each in a plain form (elementary torch operations, fp32, rounded once) and, with ``own`` set, as the
calls a user makes of ``hybrid_model_ssm_gdn_b200``:

* ``scan``   -- the Mamba-2 scan over a packed batch of prompts, from zero or from each slot's state: y and the states.
* ``conv``   -- the short causal convolution over a packed batch of prompts, split into the layer's inputs.
* ``tokens`` -- the same convolution for decoding: one token a sequence, or T drafts and the commit of a prefix.
* ``accept`` -- verification of drafted tokens against the target's probabilities, from given random numbers.

Sizes are those of the library's layers: the Mamba-2 layer of a 120B-class model (128 heads of 64, state 128, 8
groups: a convolution over 8192 + 2 * 1024 channels), the tiny layer (8 heads, one group, fp32), and GDN layers (q, k, v
of 32 heads of 128).
"""

import math

import numpy as np
import torch

own = False

N = 128  # state size of the library's layers

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}


def listed():
    layer = {"heads": 128, "headdim": 64, "groups": 8}
    tiny = {"heads": 8, "headdim": 64, "groups": 1}
    return [
        # a batch of prompts of mixed lengths entering the 120B-class layer
        {"name": "scan-bf16-packed", "op": "scan", "dtype": "bf16", "total": 16384, "nseq": 8, "resume": False, **layer},
        # one long prompt: few independent rows, a long axis
        {"name": "scan-bf16-one-long", "op": "scan", "dtype": "bf16", "total": 8191, "nseq": 1, "resume": False, **layer},
        # the next turns of many conversations: short pieces on top of a held state
        {"name": "scan-bf16-short-turns", "op": "scan", "dtype": "bf16", "total": 1500, "nseq": 48, "resume": True,
         **layer},
        # the tiny fp32 layer, two prompts
        {"name": "scan-f32-tiny", "op": "scan", "dtype": "f32", "total": 301, "nseq": 2, "resume": False, **tiny},
        # the convolution in front of the first case
        {"name": "conv-bf16-packed", "op": "conv", "dtype": "bf16", "total": 16384, "nseq": 8, "resume": False,
         "width": 4, "bias": True, "silu": True, "c0": 8192, "c1": 1024, "c2": 1024},
        # a small fp32 layer without bias, resumed, odd lengths
        {"name": "conv-f32-resumed", "op": "conv", "dtype": "f32", "total": 777, "nseq": 5, "resume": True,
         "width": 3, "bias": False, "silu": True, "c0": 512, "c1": 128, "c2": 128},
        # one decode token of one sequence: latency
        {"name": "tokens-b1-step", "op": "tokens", "dtype": "bf16", "batch": 1, "drafts": 0, "width": 4, "bias": True,
         "silu": True, "c0": 8192, "c1": 1024, "c2": 1024},
        # one decode token of the library's usual batch, GDN's q, k, v
        {"name": "tokens-b256-step", "op": "tokens", "dtype": "bf16", "batch": 256, "drafts": 0, "width": 4,
         "bias": True, "silu": True, "c0": 4096, "c1": 4096, "c2": 4096},
        # the speculative workload: 8 drafts a sequence at batch 512, then the commit
        {"name": "tokens-b512-drafts8", "op": "tokens", "dtype": "bf16", "batch": 512, "drafts": 8, "width": 4,
         "bias": True, "silu": True, "c0": 8192, "c1": 1024, "c2": 1024},
        # one sequence, a small vocabulary: latency
        {"name": "accept-b1", "op": "accept", "batch": 1, "drafts": 4, "vocab": 32000, "probs": True, "ragged": False},
        # a serving batch over a large vocabulary
        {"name": "accept-b256", "op": "accept", "batch": 256, "drafts": 4, "vocab": 131072, "probs": True,
         "ragged": False},
        # drafts without probabilities (looked up, not sampled), uneven numbers of them, an odd vocabulary
        {"name": "accept-b64-lookup", "op": "accept", "batch": 64, "drafts": 8, "vocab": 50257, "probs": False,
         "ragged": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("scan", "conv", "tokens", "accept"))
    if op == "scan":
        dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
        groups = rng.choice((1, 2, 4, 8))
        heads = groups * rng.randint(1, 16 if dtype == "bf16" else 4)
        total = _log(rng, 1, 16384 if dtype == "bf16" else 2048)
        return {"op": op, "dtype": dtype, "heads": heads, "headdim": rng.choice((8, 24, 32, 48, 64, 64, 64)),
                "groups": groups, "total": total, "nseq": _log(rng, 1, min(64, total)), "resume": rng.random() < 0.5}
    if op in ("conv", "tokens"):
        dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
        if rng.random() < 0.5:
            c0, c1 = 8 * rng.randint(1, 1024), 128 * rng.randint(1, 8)
        else:
            c0 = c1 = 128 * rng.randint(1, 26)
        case = {"op": op, "dtype": dtype, "width": rng.choice((2, 3, 4, 4)), "bias": rng.random() < 0.5,
                "silu": rng.random() < 0.8, "c0": c0, "c1": c1, "c2": c1}
        if op == "conv":
            total = _log(rng, 1, 16384 if dtype == "bf16" else 8192)
            return {**case, "total": total, "nseq": _log(rng, 1, min(64, total)), "resume": rng.random() < 0.5}
        return {**case, "batch": _log(rng, 1, 512), "drafts": rng.choice((0, 0, 1, 2, 4, 5, 8))}
    vocab = _log(rng, 2, 262144)
    drafts = rng.randint(0, 8)
    most = 256 * 131072 * 5 // (vocab * (drafts + 1))
    return {"op": op, "batch": _log(rng, 1, max(1, min(512, most))), "drafts": drafts, "vocab": vocab,
            "probs": rng.random() < 0.7, "ragged": rng.random() < 0.5}


# ------------------------------------------------------------------------------------------ inputs


def _lengths(case, seed):
    """`nseq` lengths that sum to `total`, uneven; about one in eight prompts is a single token."""
    r = np.random.default_rng([int(seed), 11])
    nseq, total = case["nseq"], case["total"]
    w = r.gamma(1.5, size=nseq)
    w[r.random(nseq) < 0.125] = 0.0
    if w.sum() == 0.0:
        w[:] = 1.0
    free = total - nseq
    lens = 1 + np.floor(w / w.sum() * free).astype(np.int64)
    lens[int(np.argmax(w))] += total - int(lens.sum())
    return [int(v) for v in lens]


def _prompts(case, seed, s):
    lens = _lengths(case, seed)
    nseq = len(lens)
    r = np.random.default_rng([int(seed), 12])
    slots = nseq + 3  # a context with more slots than prompts in this call
    s["lens"] = lens
    s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    s["slots"] = torch.tensor(r.permutation(slots)[:nseq].copy(), dtype=torch.int32, device="cuda")
    s["resume"] = torch.full((nseq,), 1, dtype=torch.uint8, device="cuda") if case["resume"] else None
    return slots


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    if case["op"] == "scan":
        dt_, H, P, G, total = _DT[case["dtype"]], case["heads"], case["headdim"], case["groups"], case["total"]
        slots = _prompts(case, seed, s)
        sd = 1.0 / math.sqrt(N)
        s["A"] = -torch.exp(torch.rand(H, generator=g, device="cuda") * math.log(16.0))
        s["D"] = normal(H)
        dt0 = torch.exp(math.log(1e-3) + torch.rand(H, generator=g, device="cuda") * math.log(100.0))
        bias = dt0 + torch.log(-torch.expm1(-dt0))
        s["x"] = normal(total, H, P, dtype=dt_)
        s["B"] = normal(total, G, N, std=sd, dtype=dt_)
        s["C"] = normal(total, G, N, std=sd, dtype=dt_)
        z = normal(total, H) + bias
        s["dt"] = torch.log1p(torch.exp(z)).clamp(1e-3, 0.1).to(dt_)
        s["S"] = normal(slots, H, P, N, std=0.05)
        return s
    if case["op"] in ("conv", "tokens"):
        dt_, K = _DT[case["dtype"]], case["width"]
        s["splits"] = (case["c0"], case["c1"], case["c2"])
        ch = sum(s["splits"])
        bound = 1.0 / math.sqrt(K)
        s["weight"] = ((torch.rand(ch, K, generator=g, device="cuda") * 2 - 1) * bound).to(dt_)
        s["bias"] = ((torch.rand(ch, generator=g, device="cuda") * 2 - 1) * bound).to(dt_) if case["bias"] else None
        if case["op"] == "conv":
            slots = _prompts(case, seed, s)
            s["x"] = normal(case["total"], ch, dtype=dt_)
            ring = K - 1
        else:
            slots, T = case["batch"], max(1, case["drafts"])
            s["x"] = normal(slots, ch, dtype=dt_) if case["drafts"] == 0 else normal(slots, T, ch, dtype=dt_)
            ring = K - 1 + T
            if case["drafts"]:
                s["accepted"] = torch.randint(0, T + 1, (slots,), generator=g, device="cuda", dtype=torch.int32)
        s["hist"] = normal(slots, ring, ch, dtype=dt_)
        s["cur"] = torch.randint(0, ring, (slots,), generator=g, device="cuda", dtype=torch.int32)
        return s
    batch, T, V = case["batch"], case["drafts"], case["vocab"]
    logits = normal(batch, T + 1, V, std=2.5)
    noise = normal(batch, T + 1, V, std=0.7)
    s["target"] = torch.softmax(logits + noise, dim=-1)
    del noise
    draft = torch.softmax(logits[:, :T], dim=-1)
    if T:  # the drafts are sampled from the draft's distribution
        e = torch.empty(batch, T, V, device="cuda").exponential_(generator=g)
        s["tokens"] = (draft / e).argmax(-1).to(torch.int32)
    else:
        s["tokens"] = torch.zeros(batch, 0, dtype=torch.int32, device="cuda")
    s["draft"] = draft if case["probs"] else None
    s["u"] = torch.rand(batch, T + 1, generator=g, device="cuda")
    s["count"] = (torch.randint(0, T + 1, (batch,), generator=g, device="cuda", dtype=torch.int32)
                  if case["ragged"] else None)
    return s


# ------------------------------------------------------------------------------------------ plain forms


def _plain_scan(s):
    """The chunked form of the recurrence, all chunks of all prompts at once; each prompt's last chunk is padded."""
    Q = 64
    x, Bm, Cm, dt, A, D, off = s["x"], s["B"], s["C"], s["dt"], s["A"], s["D"], s["offsets"].long()
    total, H, P = x.shape
    G = Bm.shape[1]
    r = H // G
    dev = x.device
    nch = [-(-n // Q) for n in s["lens"]]
    nc = sum(nch)
    nseq = len(nch)
    nch_t = (off[1:] - off[:-1] + Q - 1) // Q
    seq = torch.repeat_interleave(torch.arange(nseq, device=dev), nch_t, output_size=nc)       # chunk -> prompt
    last = torch.cumsum(nch_t, 0) - 1                                                          # prompt -> last chunk
    k = torch.arange(nc, device=dev) - (last + 1 - nch_t)[seq]                                 # chunk in its prompt
    idx = off[seq][:, None] + k[:, None] * Q + torch.arange(Q, device=dev)
    live = idx < off[seq + 1][:, None]
    idx = torch.where(live, idx, 0)
    xs = (x[idx].float() * live[:, :, None, None]).view(nc, Q, G, r, P)
    Bs = Bm[idx].float() * live[:, :, None, None]
    Cs = Cm[idx].float() * live[:, :, None, None]
    dts = dt[idx].float() * live[:, :, None]
    cum = torch.cumsum(dts, 1) * A                                                             # [nc][Q][H]
    diff = cum.transpose(1, 2)[:, :, :, None] - cum.transpose(1, 2)[:, :, None, :]             # [nc][H][j][i]
    causal = torch.ones(Q, Q, dtype=torch.bool, device=dev).tril()
    M = torch.exp(diff.masked_fill(~causal, -math.inf))
    del diff
    gram = torch.matmul(Cs.transpose(1, 2), Bs.permute(0, 2, 3, 1))                            # [nc][G][j][i]
    M = (M.view(nc, G, r, Q, Q) * gram[:, :, None]).view(nc, H, Q, Q) * dts.transpose(1, 2)[:, :, None, :]
    xh = xs.reshape(nc, Q, H, P).transpose(1, 2)                                               # [nc][H][Q][P]
    y = torch.matmul(M, xh)
    del M
    end = cum[:, -1]                                                                           # [nc][H]
    w = torch.exp(end[:, None] - cum) * dts                                                    # [nc][Q][H]
    wx = (xh * w.transpose(1, 2)[..., None]).view(nc, G, r, Q, P)
    local = torch.matmul(wx.transpose(-1, -2), Bs.transpose(1, 2)[:, :, None]).view(nc, H, P * N)
    # states at the chunks' starts: decayed sums of the earlier chunks of the same prompt (long sums in 64 bits)
    run = torch.cumsum(end.double(), 0)                                                        # [nc][H]
    start = run - end
    first = (last + 1 - nch_t)[seq]
    between = (start.T[:, :, None] - run.T[:, None, :])                                        # [H][c][k]
    same = (seq[:, None] == seq[None, :]) & torch.ones(nc, nc, dtype=torch.bool, device=dev).tril(-1)
    W = torch.exp(between.masked_fill(~same, -math.inf)).float()
    S_in = torch.matmul(W, local.transpose(0, 1)).transpose(0, 1)                              # [nc][H][P*N]
    slots = s["slots"].long()
    if s["resume"] is not None:
        S0 = s["S"][slots].view(nseq, H, P * N)
        S_in = S_in + torch.exp(start - start[first]).float()[..., None] * S0[seq]
    S_in = S_in.reshape(nc, G, r * P, N)
    carried = torch.matmul(Cs.transpose(1, 2), S_in.transpose(-1, -2)).view(nc, G, Q, r, P)     # C S^T
    carried = carried.transpose(2, 3).reshape(nc, H, Q, P)
    y = y + torch.exp(cum).transpose(1, 2)[..., None] * carried + D[:, None, None] * xh
    out = torch.empty(total, H, P, device=dev)
    out[idx[live]] = y.transpose(1, 2)[live]
    S_end = torch.exp(end[last])[..., None] * S_in.view(nc, H, P * N)[last] + local[last]
    s["S"][slots] = S_end.view(nseq, H, P, N)
    return out, s["S"]


def _act(v, silu):
    return v / (1.0 + torch.exp(-v)) if silu else v


def _filter(taps, s):
    """taps [..., K, channels] fp32 -> the split outputs in the inputs' type."""
    v = (taps * s["weight"].float().T).sum(-2)
    if s["bias"] is not None:
        v = v + s["bias"].float()
    return torch.split(_act(v, s["case"]["silu"]).to(s["x"].dtype), s["splits"], dim=-1)


def _plain_conv(s):
    x, off, hist, cur, slots = s["x"], s["offsets"].long(), s["hist"], s["cur"].long(), s["slots"].long()
    total, K = x.shape[0], s["weight"].shape[1]
    nseq, ring, dev = len(s["lens"]), hist.shape[1], x.device
    at = (cur[slots][:, None] - (K - 1) + torch.arange(K - 1, device=dev)) % ring              # ring rows, oldest first
    held = hist[slots[:, None], at]
    if s["resume"] is None:
        held = torch.zeros_like(held)
    rows = torch.cat([x, held.reshape(nseq * (K - 1), -1)])                                    # tokens, then histories
    seq = torch.repeat_interleave(torch.arange(nseq, device=dev), off[1:] - off[:-1], output_size=total)
    t = torch.arange(total, device=dev)

    def row(q, tok):  # the row that holds token `tok` of prompt q, which may lie before its start
        back = tok - off[q]
        return torch.where(back >= 0, tok, total + q * (K - 1) + (K - 1) + back)

    taps = row(seq[:, None], t[:, None] - (K - 1) + torch.arange(K, device=dev))
    out = _filter(rows[taps].float(), s)
    q = torch.arange(nseq, device=dev)
    new = row(q[:, None], off[1:, None] - (K - 1) + torch.arange(K - 1, device=dev))
    hist[slots[:, None], at] = rows[new]
    return (*out, hist, s["cur"])


def _plain_tokens(s):
    x, hist, cur, K, T = s["x"], s["hist"], s["cur"], s["weight"].shape[1], max(1, s["case"]["drafts"])
    batch, ring, dev = hist.shape[0], hist.shape[1], x.device
    b = torch.arange(batch, device=dev)[:, None]
    at = cur.long()[:, None] + torch.arange(1 - K, T, device=dev)
    hist[b, at[:, K - 1:] % ring] = x.view(batch, T, -1)
    rows = hist[b, at % ring].float()                                                          # [batch][K-1+T][ch]
    taps = rows.unfold(1, K, 1).transpose(-1, -2)                                              # [batch][T][K][ch]
    out = [v.view(*x.shape[:-1], -1) for v in _filter(taps, s)]
    moved = s["accepted"] if s["case"]["drafts"] else 1
    cur.copy_((cur + moved) % ring)
    return (*out, hist, cur)


def _plain_accept(s):
    """Masses and sums in 64 bits: the sampled token is a whole number and sits next to a border of the sums."""
    p, q, d, u = s["target"], s["draft"], s["tokens"].long(), s["u"].double()
    batch, T1, V = p.shape
    T, dev = T1 - 1, p.device
    count = torch.full((batch,), T, device=dev) if s["count"] is None else s["count"].long()
    pd = torch.gather(p[:, :T], 2, d[:, :, None])[..., 0].double()
    qd = torch.ones_like(pd) if q is None else torch.gather(q, 2, d[:, :, None])[..., 0].double()
    good = (u[:, :T] * qd < pd) & (torch.arange(T, device=dev) < count[:, None])
    n = torch.cumprod(good.long(), 1).sum(1) if T else torch.zeros_like(count)
    b = torch.arange(batch, device=dev)
    row = p[b, n].double()
    rejected = n < count
    mass = row
    if T and q is not None:
        mass = torch.where(rejected[:, None], row - q[b, n.clamp(max=T - 1)].double(), row).clamp(min=0)
    elif T:
        hot = torch.arange(V, device=dev) == d[b, n.clamp(max=T - 1)][:, None]
        mass = torch.where(rejected[:, None] & hot, 0.0, row)
    mass = torch.where(mass.sum(1, keepdim=True) > 0, mass, row)
    cdf = torch.cumsum(mass, 1)
    goal = u[:, T:] * cdf[:, -1:]
    token = torch.where(mass > 0, torch.arange(V, device=dev), -1).amax(1)                     # the last one with mass
    token = torch.minimum(token, (cdf <= goal).sum(1))
    return n.to(torch.int32), (n + 1).to(torch.int32), token.to(torch.int32)


# ------------------------------------------------------------------------------------------ one pass


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import hybrid_model_ssm_gdn_b200 as rssm
        if op == "scan":
            y = rssm.mamba2_scan(s["S"], s["x"], s["B"], s["C"], s["dt"], s["A"], s["D"], s["offsets"],
                                 slots=s["slots"], resume=s["resume"])
            return y, s["S"]
        act = "silu" if s["case"].get("silu") else None
        if op == "conv":
            out = rssm.shortconv_prefill(s["hist"], s["cur"], s["x"], s["weight"], s["bias"], s["offsets"],
                                         slots=s["slots"], resume=s["resume"], splits=s["splits"], activation=act)
            return (*out, s["hist"], s["cur"])
        if op == "tokens":
            if s["case"]["drafts"] == 0:
                out = rssm.shortconv_step(s["hist"], s["cur"], s["x"], s["weight"], s["bias"], splits=s["splits"],
                                          activation=act)
            else:
                out = rssm.shortconv_verify(s["hist"], s["cur"], s["x"], s["weight"], s["bias"], splits=s["splits"],
                                            activation=act)
                rssm.shortconv_commit(s["hist"], s["cur"], s["accepted"], width=s["case"]["width"])
            return (*out, s["hist"], s["cur"])
        return rssm.accept_drafts(s["target"], s["tokens"], s["u"], draft=s["draft"], count=s["count"])
    if op == "scan":
        return _plain_scan(s)
    if op == "conv":
        return _plain_conv(s)
    if op == "tokens":
        return _plain_tokens(s)
    return _plain_accept(s)


def work(case):
    if case["op"] == "scan":
        H, P, G, esz = case["heads"], case["headdim"], case["groups"], _BYTES[case["dtype"]]
        token = esz * (H * P + 2 * G * N + H) + 4 * H * P
        state = case["nseq"] * H * P * N * 4 * (2 if case["resume"] else 1)
        return {"bytes": case["total"] * token + state, "flops": case["total"] * H * P * (5 * N + 2)}
    if case["op"] in ("conv", "tokens"):
        ch, K, esz = case["c0"] + case["c1"] + case["c2"], case["width"], _BYTES[case["dtype"]]
        weights = ch * (K + 1) * esz
        if case["op"] == "conv":
            rows, kept = case["total"], case["nseq"] * (K - 1) * (2 if case["resume"] else 1)
        else:
            T = max(1, case["drafts"])
            rows, kept = case["batch"] * T, case["batch"] * (K - 1 + T)
        return {"bytes": (2 * rows + kept) * ch * esz + weights, "flops": rows * ch * (2 * K + 5)}
    # one row of the target's probabilities a sequence, and one of the draft's where a draft was rejected (about
    # three in four drafts are accepted with these distributions)
    T, V = case["drafts"], case["vocab"]
    rejected = (1.0 - 0.75 ** T) if case["probs"] else 0.0
    return {"bytes": int(case["batch"] * (V * 4 * (1.0 + rejected) + 16 * (T + 1))), "flops": 3 * case["batch"] * V}


# ------------------------------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    s = prepare(case, seed)

    def scan(s):
        """The recurrence token by token, all prompts side by side."""
        x, Bm, Cm, dt = (s[k].double() for k in ("x", "B", "C", "dt"))
        A, D = s["A"].double(), s["D"].double()
        H, G = x.shape[1], Bm.shape[1]
        S_all, slots = s["S"].double(), s["slots"].long()
        S = S_all[slots] if s["resume"] is not None else torch.zeros_like(S_all[slots])
        y = torch.zeros_like(x)
        lens = np.array(s["lens"])
        first = np.concatenate([[0], np.cumsum(lens)[:-1]])
        order = np.argsort(-lens, kind="stable")           # longest first: the live prompts are a prefix
        S = S[torch.from_numpy(order).cuda()]
        starts = torch.from_numpy(first[order]).cuda()
        for t in range(int(lens.max())):
            m = int((lens > t).sum())
            i = starts[:m] + t
            b = Bm[i].repeat_interleave(H // G, 1)
            c = Cm[i].repeat_interleave(H // G, 1)
            step = dt[i]
            S[:m] *= torch.exp(step * A)[:, :, None, None]
            S[:m] += (step[..., None] * x[i])[..., None] * b[:, :, None, :]
            y[i] = torch.matmul(S[:m], c[..., None])[..., 0] + D[:, None] * x[i]
        back = torch.empty_like(S)
        back[torch.from_numpy(order).cuda()] = S
        S_all[slots] = back
        return y, S_all

    def line_of(line, s):
        """One sequence of rows [K-1+n][channels] -> n outputs."""
        K, n = s["weight"].shape[1], line.shape[0] - s["weight"].shape[1] + 1
        v = torch.zeros(n, line.shape[1], dtype=torch.float64, device=line.device)
        for k in range(K):
            v += line[k:k + n] * s["weight"][:, k].double()
        if s["bias"] is not None:
            v += s["bias"].double()
        return v * torch.sigmoid(v) if s["case"]["silu"] else v

    def conv(s):
        K, ring = s["weight"].shape[1], s["hist"].shape[1]
        hist, outs = s["hist"].double(), []
        bounds = [0]
        for n in s["lens"]:
            bounds.append(bounds[-1] + n)
        for i, slot in enumerate(s["slots"].tolist()):
            c = int(s["cur"][slot])
            at = [(c - (K - 1) + k) % ring for k in range(K - 1)]
            held = hist[slot, at] if s["resume"] is not None else torch.zeros_like(hist[slot, at])
            line = torch.cat([held, s["x"][bounds[i]:bounds[i + 1]].double()])
            outs.append(line_of(line, s))
            hist[slot, at] = line[line.shape[0] - (K - 1):]
        return (*torch.split(torch.cat(outs), s["splits"], dim=-1), hist, s["cur"].clone())

    def tokens(s):
        K, ring, T = s["weight"].shape[1], s["hist"].shape[1], max(1, s["case"]["drafts"])
        hist, cur, batch = s["hist"].double(), s["cur"].clone(), s["hist"].shape[0]
        x = s["x"].view(batch, T, -1).double()
        outs = []
        for b in range(batch):
            c = int(cur[b])
            held = hist[b, [(c - (K - 1) + k) % ring for k in range(K - 1)]]
            outs.append(line_of(torch.cat([held, x[b]]), s))
            hist[b, [(c + k) % ring for k in range(T)]] = x[b]
            cur[b] = (c + (int(s["accepted"][b]) if s["case"]["drafts"] else 1)) % ring
        out = torch.stack(outs).view(*s["x"].shape)
        return (*torch.split(out, s["splits"], dim=-1), hist, cur)

    def accept(s):
        batch, T1, V = s["target"].shape
        got = []
        u, d = s["u"].double().cpu().numpy(), s["tokens"].cpu().numpy()
        for b in range(batch):
            count = T1 - 1 if s["count"] is None else int(s["count"][b])
            n = 0
            while n < count:
                pd = float(s["target"][b, n, d[b, n]])
                qd = 1.0 if s["draft"] is None else float(s["draft"][b, n, d[b, n]])
                if not u[b, n] * qd < pd:
                    break
                n += 1
            row = s["target"][b, n].cpu().numpy().astype(np.float64)
            mass = row.copy()
            if n < count and s["draft"] is not None:
                mass = np.maximum(row - s["draft"][b, n].cpu().numpy().astype(np.float64), 0.0)
            elif n < count:
                mass[d[b, n]] = 0.0
            if not mass.sum() > 0:
                mass = row
            cdf = np.cumsum(mass)
            token = int(np.searchsorted(cdf, u[b, T1 - 1] * cdf[-1], side="right"))
            got.append((n, n + 1, min(token, int(np.nonzero(mass)[0][-1]))))
        return tuple(torch.tensor([g[k] for g in got], dtype=torch.int32) for k in range(3))

    return {"scan": scan, "conv": conv, "tokens": tokens, "accept": accept}[case["op"]](s)
