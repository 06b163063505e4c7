"""Cases that measure the operators of a recurrent layer between its projections.

Four operators, each in a plain form (elementary torch operations, fp32, rounded once) and, with ``own`` set, as the
calls a user makes of ``hybrid_model_ssm_gdn_b200``:

* ``scan``   -- the gated delta rule over a packed batch of prompts, from zero or from each slot's state: y and the states.
* ``inputs`` -- what the gated delta rule takes: normalised queries and keys, decays and write strengths.
* ``norm``   -- the root-mean-square norm in front of a layer, with the residual's addition and an optional 8-bit output.
* ``gated``  -- the gated norm behind a layer, over groups of its outputs, with an optional 8-bit output.

Sizes are those of the library's layers: GDN layers (32 heads of 128; 16 query and key heads where two value heads share
one), the Mamba-2 layer (128 heads of 64 in 8 groups) and the tiny fp32 layer (8 heads).
"""

import math

import numpy as np
import torch

own = False

N = 128      # key size of the library's layers
BLOCK = 128  # columns of a block scale
EPS = 1e-6

_DT = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
_BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}
TINY = torch.finfo(torch.float32).tiny


def listed():
    return [
        # a batch of prompts of mixed lengths entering a GDN layer
        {"name": "scan-bf16-packed", "op": "scan", "dtype": "bf16", "total": 16384, "nseq": 8, "resume": False,
         "heads": 32, "qk_heads": 32, "headdim": 128},
        # one long prompt, query and key heads shared by two value heads: few independent rows, a long axis
        {"name": "scan-bf16-one-long", "op": "scan", "dtype": "bf16", "total": 8191, "nseq": 1, "resume": False,
         "heads": 32, "qk_heads": 16, "headdim": 128},
        # the next turns of many conversations: short pieces on top of a held state
        {"name": "scan-bf16-short-turns", "op": "scan", "dtype": "bf16", "total": 1500, "nseq": 48, "resume": True,
         "heads": 32, "qk_heads": 16, "headdim": 128},
        # the tiny fp32 layer, two prompts
        {"name": "scan-f32-tiny", "op": "scan", "dtype": "f32", "total": 301, "nseq": 2, "resume": False,
         "heads": 8, "qk_heads": 8, "headdim": 64},
        # in front of the long prompt's kind of layer, a batch of prompts
        {"name": "inputs-bf16-prompts", "op": "inputs", "dtype": "bf16", "rows": 16384, "heads": 32, "qk_heads": 16,
         "expand": False},
        # one decode token of one sequence, heads repeated for the decode call: latency
        {"name": "inputs-bf16-b1", "op": "inputs", "dtype": "bf16", "rows": 1, "heads": 32, "qk_heads": 16,
         "expand": True},
        # in front of a layer whose projection takes 8 bits, a batch of prompts
        {"name": "norm-bf16-e4m3-prompts", "op": "norm", "dtype": "bf16", "out": "e4m3", "block": 0, "rows": 16384,
         "columns": 4096, "residual": True},
        # one decode token of one sequence: latency
        {"name": "norm-bf16-b1", "op": "norm", "dtype": "bf16", "out": "bf16", "block": 0, "rows": 1, "columns": 8192,
         "residual": True},
        # odd sizes, fp32, no residual yet (the first layer)
        {"name": "norm-f32-odd", "op": "norm", "dtype": "f32", "out": "f32", "block": 0, "rows": 333, "columns": 1000,
         "residual": False},
        # behind a GDN layer, a batch of prompts, 8 bits with a scale for each 128 columns
        {"name": "gated-e4m3-prompts", "op": "gated", "dtype": "bf16", "out": "e4m3", "block": BLOCK, "rows": 16384,
         "groups": 32, "group": 128, "shared": True, "norm_first": True},
        # behind a Mamba-2 layer, one decode token of the library's usual batch
        {"name": "gated-bf16-b256", "op": "gated", "dtype": "bf16", "out": "bf16", "block": 0, "rows": 256, "groups": 8,
         "group": 1024, "shared": False, "norm_first": False},
        # one decode token of the tiny fp32 layer
        {"name": "gated-f32-tiny-b1", "op": "gated", "dtype": "f32", "out": "f32", "block": 0, "rows": 1, "groups": 1,
         "group": 512, "shared": False, "norm_first": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("scan", "scan", "inputs", "norm", "gated"))
    if op == "scan":
        dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
        qk = rng.choice((1, 2, 3, 4, 8, 16))
        heads = qk * rng.randint(1, min(4, 32 // qk) if dtype == "bf16" else 1)
        total = _log(rng, 1, 16384 if dtype == "bf16" else 1024)
        return {"op": op, "dtype": dtype, "total": total, "nseq": _log(rng, 1, min(64, total)),
                "resume": rng.random() < 0.5, "heads": heads, "qk_heads": qk,
                "headdim": rng.choice((8, 24, 64, 88, 128, 128, 128))}
    if op == "inputs":
        qk = _log(rng, 1, 16)
        return {"op": op, "dtype": rng.choice(("bf16", "bf16", "f32")), "rows": _log(rng, 1, 8192),
                "heads": qk * rng.randint(1, 3), "qk_heads": qk, "expand": rng.random() < 0.5}
    dtype = rng.choice(("bf16", "bf16", "f32"))
    out = rng.choice((dtype, "e4m3"))
    block = BLOCK if out == "e4m3" and rng.random() < 0.5 else 0
    rows = _log(rng, 1, 8192)
    if op == "norm":
        return {"op": op, "dtype": dtype, "out": out, "block": block, "rows": rows,
                "columns": 8 * _log(rng, 1, 1024), "residual": rng.random() < 0.7}
    group = 8 * _log(rng, 1, 128)
    return {"op": op, "dtype": dtype, "out": out, "block": block, "rows": rows, "groups": rng.randint(1, max(1, 4096 // group)),
            "group": group, "shared": rng.random() < 0.5, "norm_first": rng.random() < 0.5}


# ------------------------------------------------------------------------------------------ inputs


def _lengths(case, seed):
    """`nseq` lengths that sum to `total`, uneven; about one in eight prompts is a single token."""
    r = np.random.default_rng([int(seed), 21])
    nseq, total = case["nseq"], case["total"]
    w = r.gamma(1.5, size=nseq)
    w[r.random(nseq) < 0.125] = 0.0
    if w.sum() == 0.0:
        w[:] = 1.0
    lens = 1 + np.floor(w / w.sum() * (total - nseq)).astype(np.int64)
    lens[int(np.argmax(w))] += total - int(lens.sum())
    return [int(v) for v in lens]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    def gates(heads):  # A in 1 .. 16, steps of 1e-3 .. 1e-1 at a = 0
        dt0 = torch.exp(math.log(1e-3) + uniform(heads) * math.log(100.0))
        return torch.log(1.0 + 15.0 * uniform(heads)), dt0 + torch.log(-torch.expm1(-dt0))

    op = case["op"]
    if op == "scan":
        dt_, H, Hk, P, total = _DT[case["dtype"]], case["heads"], case["qk_heads"], case["headdim"], case["total"]
        lens = _lengths(case, seed)
        slots = len(lens) + 3  # a context with more slots than prompts in this call
        r = np.random.default_rng([int(seed), 22])
        s["lens"] = lens
        s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        s["slots"] = torch.tensor(r.permutation(slots)[:len(lens)].copy(), dtype=torch.int32, device="cuda")
        s["resume"] = torch.ones(len(lens), dtype=torch.uint8, device="cuda") if case["resume"] else None
        for name in ("q", "k"):
            t = normal(total, Hk, N)
            s[name] = (t / torch.sqrt((t * t).sum(-1, keepdim=True) + EPS)).to(dt_)
        s["v"] = normal(total, H, P, dtype=dt_)
        A_log, bias = gates(H)
        s["alpha"] = torch.exp(-torch.exp(A_log) * torch.log1p(torch.exp(normal(total, H) + bias)))
        s["beta"] = torch.sigmoid(normal(total, H))
        s["S"] = normal(slots, H, P, N, std=0.05)
        s["q_scale"] = 1.0 / math.sqrt(N)
    elif op == "inputs":
        dt_, rows, H, Hk = _DT[case["dtype"]], case["rows"], case["heads"], case["qk_heads"]
        s["q"], s["k"] = normal(rows, Hk, N, dtype=dt_), normal(rows, Hk, N, dtype=dt_)
        s["a"], s["b"] = normal(rows, H, dtype=dt_), normal(rows, H, dtype=dt_)
        s["A_log"], s["bias"] = gates(H)
    elif op == "norm":
        dt_, rows, n = _DT[case["dtype"]], case["rows"], case["columns"]
        s["x"] = normal(rows, n, dtype=dt_)
        s["residual"] = normal(rows, n, std=3.0, dtype=dt_) if case["residual"] else None
        s["weight"] = (1.0 + normal(n, std=0.1)).to(dt_)
    else:
        dt_, rows, n = _DT[case["dtype"]], case["rows"], case["groups"] * case["group"]
        s["y"] = normal(rows, n, std=0.3)  # the layers' outputs are fp32
        s["gate"] = normal(rows, n, dtype=dt_)
        s["weight"] = (1.0 + normal(case["group"] if case["shared"] else n, std=0.1)).to(dt_)
    return s


# ------------------------------------------------------------------------------------------ plain forms


def _inverse(L):
    """(I + L)^-1 of strictly lower triangular [..., Q, Q], Q a power of two: blocks of twice the size at each level."""
    Q = L.shape[-1]
    T = torch.eye(Q, device=L.device).expand(L.shape).contiguous()
    i = torch.arange(Q, device=L.device)
    half = 1
    while half < Q:
        low = (i[:, None] // (2 * half) == i[None, :] // (2 * half)) & (i[:, None] % (2 * half) >= half) & \
            (i[None, :] % (2 * half) < half)
        T = T - torch.matmul(T, torch.matmul(L * low, T))
        half *= 2
    return T


def _plain_scan(s):
    """Chunks of 64 tokens: what does not depend on the state for all chunks at once, then chunk after chunk with all
    prompts side by side; each prompt's last chunk is padded with tokens that change nothing."""
    Q = 64
    q, k, v, off = s["q"], s["k"], s["v"], s["offsets"].long()
    total, H, P = v.shape
    r = H // q.shape[1]
    dev = v.device
    most = -(-max(s["lens"]) // Q)
    nseq = len(s["lens"])
    idx = off[:-1, None, None] + torch.arange(most * Q, device=dev).view(1, most, Q)
    live = idx < off[1:, None, None]
    ids = torch.nonzero(live[:, :, 0])                                  # chunks that have tokens (sequence, chunk)
    at = torch.full((nseq, most), ids.shape[0], device=dev)             # the others: one chunk more, of nothing
    at[ids[:, 0], ids[:, 1]] = torch.arange(ids.shape[0], device=dev)
    idx, live = idx[ids[:, 0], ids[:, 1]], live[ids[:, 0], ids[:, 1]]
    idx = torch.where(live, idx, 0)

    def chunks(t, to=torch.float32):  # [total][heads][...] -> [chunk][heads][Q][...], zeros for what is not there
        t = t[idx].to(to) * live.view(*live.shape, *([1] * (t.dim() - 1)))
        t = torch.cat([t, torch.zeros_like(t[:1])])
        return t.transpose(1, 2)

    qs, ks = (chunks(s[n]).repeat_interleave(r, 1) for n in ("q", "k"))
    vs, beta = chunks(v), chunks(s["beta"])
    cum = torch.cumsum(chunks(torch.log(s["alpha"].double()), torch.float64), -1)
    tri = torch.ones(Q, Q, dtype=torch.bool, device=dev).tril()
    decay = torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(~tri, -math.inf)).float()
    T = _inverse(torch.matmul(ks, ks.transpose(-1, -2)) * decay.tril(-1) * beta[..., None]) * beta[..., None, :]
    M = torch.matmul(qs, ks.transpose(-1, -2)) * decay
    rise = torch.exp(cum).float()[..., None]
    fall = torch.exp(cum[..., -1:] - cum).float()[..., None]
    carry = torch.exp(cum[..., -1]).float()[..., None, None]
    slots = s["slots"].long()
    S = s["S"][slots] if s["resume"] is not None else torch.zeros(nseq, H, P, N, device=dev)
    ys = torch.empty(at.max() + 1, H, Q, P, device=dev)
    for c in range(most):
        i = at[:, c]
        St = S.transpose(-1, -2)
        U = torch.matmul(T[i], vs[i] - rise[i] * torch.matmul(ks[i], St))
        ys[i] = rise[i] * torch.matmul(qs[i], St) + torch.matmul(M[i], U)
        S = carry[i] * S + torch.matmul(U.transpose(-1, -2), fall[i] * ks[i])
    out = torch.empty(total, H, P, device=dev)
    out[idx[live]] = s["q_scale"] * ys[:ids.shape[0]].transpose(1, 2)[live]
    s["S"][slots] = S
    return out, s["S"]


def _plain_inputs(s):
    r = s["case"]["heads"] // s["case"]["qk_heads"] if s["case"]["expand"] else 1

    def unit(t):
        f = t.float()
        return (f / torch.sqrt((f * f).sum(-1, keepdim=True) + EPS)).to(t.dtype).repeat_interleave(r, 1)

    z = s["a"].float() + s["bias"]
    softplus = torch.clamp(z, min=0.0) + torch.log1p(torch.exp(-torch.abs(z)))
    return (unit(s["q"]), unit(s["k"]), torch.exp(-torch.exp(s["A_log"]) * softplus),
            1.0 / (1.0 + torch.exp(-s["b"].float())))


def _rounded(v, case):
    """v fp32 -> the output, with its scales where it has 8 bits: the largest magnitude of a row or block becomes 448."""
    if case["out"] != "e4m3":
        return (v.to(_DT[case["out"]]),)
    rows, n = v.shape
    size = case["block"] or n
    parts = torch.nn.functional.pad(v, (0, -n % size)).view(rows, -1, size)
    scale = torch.clamp(parts.abs().amax(-1) / 448.0, min=TINY)
    codes = (parts / scale[..., None]).clamp(-448.0, 448.0).view(rows, -1)[:, :n]
    return codes.to(torch.float8_e4m3fn), scale if case["block"] else scale[:, 0]


def _plain_norm(s):
    h, more = s["x"].float(), ()
    if s["residual"] is not None:
        h = h + s["residual"].float()
        s["residual"].copy_(h)
        more = (s["residual"],)
    v = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    return (*_rounded(v, s["case"]), *more)


def _plain_gated(s):
    case = s["case"]
    z = s["gate"].float()
    gate = z / (1.0 + torch.exp(-z))
    h = s["y"] if case["norm_first"] else s["y"] * gate
    h = h.view(h.shape[0], case["groups"], case["group"])
    w = s["weight"].float() if case["shared"] else s["weight"].float().view(case["groups"], case["group"])
    v = (h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * w).view(z.shape)
    return _rounded(v * gate if case["norm_first"] else v, case)


# ------------------------------------------------------------------------------------------ one pass


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        import hybrid_model_ssm_gdn_b200 as rssm
        if op == "scan":
            y = rssm.gdn_scan(s["S"], s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["offsets"], slots=s["slots"],
                              resume=s["resume"], q_scale=s["q_scale"])
            return y, s["S"]
        if op == "inputs":
            return rssm.gdn_inputs(s["q"], s["k"], s["a"], s["b"], s["A_log"], s["bias"], eps=EPS, expand=case["expand"])
        scale = {"e4m3": "block" if case["block"] else "row"}.get(case["out"])
        if op == "norm":
            got = rssm.add_rmsnorm(s["x"], s["weight"], residual=s["residual"], eps=EPS, scale=scale)
            more = () if s["residual"] is None else (s["residual"],)
        else:
            got = rssm.gated_rmsnorm(s["y"], s["gate"], s["weight"], group=case["group"], eps=EPS,
                                     norm_first=case["norm_first"], scale=scale)
            more = ()
        return (*got, *more) if scale else (got, *more)
    return {"scan": _plain_scan, "inputs": _plain_inputs, "norm": _plain_norm, "gated": _plain_gated}[op](s)


def work(case):
    op, esz = case["op"], _BYTES[case["dtype"]]
    if op == "scan":
        H, Hk, P = case["heads"], case["qk_heads"], case["headdim"]
        token = esz * (2 * Hk * N + H * P) + 8 * H + 4 * H * P
        state = case["nseq"] * H * P * N * 4 * (2 if case["resume"] else 1)
        return {"bytes": case["total"] * token + state, "flops": 7 * case["total"] * H * P * N}
    if op == "inputs":
        rows, H, Hk = case["rows"], case["heads"], case["qk_heads"]
        out = H if case["expand"] else Hk
        return {"bytes": rows * (2 * esz * N * (Hk + out) + H * (2 * esz + 8)) + 8 * H,
                "flops": rows * (2 * Hk * 3 * N + 20 * H)}
    rows = case["rows"]
    if op == "norm":
        n = case["columns"]
        per = esz * (3 if case["residual"] else 1) + _BYTES[case["out"]]
        return {"bytes": rows * n * per + n * esz, "flops": rows * n * 5}
    n = case["groups"] * case["group"]
    return {"bytes": rows * n * (4 + esz + _BYTES[case["out"]]) + n * esz, "flops": rows * n * 10}


# ------------------------------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    s = prepare(case, seed)

    def scan():
        """The recurrence token by token, all prompts side by side."""
        q, k, v, alpha, beta = (s[n].double() for n in ("q", "k", "v", "alpha", "beta"))
        r = v.shape[1] // q.shape[1]
        S_all, slots = s["S"].double(), s["slots"].long()
        lens = np.array(s["lens"])
        order = np.argsort(-lens, kind="stable")           # longest first: the live prompts are a prefix
        pick = torch.from_numpy(order).cuda()
        starts = torch.from_numpy((np.cumsum(lens) - lens)[order]).cuda()
        S = S_all[slots[pick]]
        if s["resume"] is None:
            S.zero_()
        y = torch.zeros_like(v)
        for t in range(int(lens.max())):
            m = int((lens > t).sum())
            i = starts[:m] + t
            kt, qt = k[i].repeat_interleave(r, 1)[..., None], q[i].repeat_interleave(r, 1)[..., None]
            S[:m] *= alpha[i][..., None, None]
            u = beta[i][..., None, None] * (v[i][..., None] - torch.matmul(S[:m], kt))
            S[:m] += u * kt.transpose(-1, -2)
            y[i] = s["q_scale"] * torch.matmul(S[:m], qt)[..., 0]
        S_all[slots[pick]] = S
        return y, S_all

    def inputs():
        r = case["heads"] // case["qk_heads"] if case["expand"] else 1
        q, k = (torch.repeat_interleave(t * ((t * t).sum(-1, keepdim=True) + EPS) ** -0.5, r, 1)
                for t in (s["q"].double(), s["k"].double()))
        z = s["a"].double() + s["bias"].double()
        rate = torch.logaddexp(z, torch.zeros_like(z)) * torch.exp(s["A_log"].double())
        return q, k, torch.exp(-rate), torch.sigmoid(s["b"].double())

    def held(v):
        """The values before their rounding, in units of their scales."""
        if case["out"] != "e4m3":
            return (v,)
        if not case["block"]:
            scale = (v.abs().max(1).values / 448.0).clamp(min=TINY)
            return v / scale[:, None], scale
        scale = torch.stack([p.abs().max(1).values for p in torch.split(v, BLOCK, 1)], 1) / 448.0
        scale = scale.clamp(min=TINY)
        return v / scale.repeat_interleave(BLOCK, 1)[:, :v.shape[1]], scale

    def norm():
        h = s["x"].double()
        if s["residual"] is not None:
            h = h + s["residual"].double()
        v = h * (h.square().sum(1, keepdim=True) / h.shape[1] + EPS) ** -0.5 * s["weight"].double()
        return (*held(v), h) if s["residual"] is not None else held(v)

    def gated():
        z, y = s["gate"].double(), s["y"].double()
        gate = z * torch.sigmoid(z)
        w = s["weight"].double()
        outs = []
        for j in range(case["groups"]):
            part = slice(j * case["group"], (j + 1) * case["group"])
            h = y[:, part] if case["norm_first"] else y[:, part] * gate[:, part]
            h = h * (h.square().sum(1, keepdim=True) / case["group"] + EPS) ** -0.5
            h = h * (w if case["shared"] else w[part])
            outs.append(h * gate[:, part] if case["norm_first"] else h)
        return held(torch.cat(outs, 1))

    return {"scan": scan, "inputs": inputs, "norm": norm, "gated": gated}[case["op"]]()
