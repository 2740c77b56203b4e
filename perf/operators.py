"""Cases of the operators around the dense head: the norm in front of it with
its 8-bit output, the 8-bit copy of E, the logits from both, and the
verification of drafted tokens against those logits.

``listed`` and ``draw`` give cases, ``prepare`` their inputs on the GPU,
``run`` one pass (in plain torch operations, or through the library where
``own`` is set), ``work`` what a pass has to move and compute, and ``exact``
the outputs in 64 bits from the definitions.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128           # columns (and rows of E) that share a scale
E4M3_MAX = 448.0
TINY = 2.0 ** -126    # smallest scale of a block
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of one sequence: the norm in front of the head
        dict(name="norm one token", op="norm", rows=1, d=2048, dtype="bf16", residual=True,
             outputs="fp8", offset=0.0),
        # drafted tokens of a few sequences, a width of nine blocks, both forms of the output
        dict(name="norm drafts both", op="norm", rows=37, d=1152, dtype="bf16", residual=True,
             outputs="both", offset=1.0),
        # the positions of long prompts, scored together
        dict(name="norm prompts", op="norm", rows=8192, d=2048, dtype="bf16", residual=True,
             outputs="fp8", offset=0.0),
        # E of a 128256-token head, once per loaded model
        dict(name="quantize large head", op="quantize", v=128256, d=2048, dtype="bf16"),
        # a small fp32 head whose last blocks are cut in both directions
        dict(name="quantize ragged f32", op="quantize", v=5003, d=1104, dtype="f32"),
        # one decode step of one sequence
        dict(name="logits one token", op="logits", rows=1, v=128256, d=2048, out="f32"),
        # eight sequences with four drafted tokens each, on the widest vocabulary
        dict(name="logits drafts", op="logits", rows=40, v=262144, d=1152, out="bf16"),
        # a middling batch on a small vocabulary, cut blocks and tiles in every direction
        dict(name="logits ragged", op="logits", rows=333, v=5003, d=1104, out="f32"),
        # every position of a prompt, as scoring a text does
        dict(name="logits prompts", op="logits", rows=2048, v=128256, d=2048, out="bf16"),
        # one sequence with four drafted tokens and the draft's probabilities: latency
        dict(name="verify one sequence", op="verify", B=1, k=4, v=128256, dtype="bf16",
             mode="sample", draft="dense", tau=0.8, masked=False),
        # a serving batch with up to seven drafted tokens a sequence
        dict(name="verify batch", op="verify", B=64, k=7, v=128256, dtype="bf16", mode="sample",
             draft="dense", tau=1.0, masked=False),
        # greedy drafts (no probabilities kept) on a small odd vocabulary with a token mask
        dict(name="verify masked odd", op="verify", B=9, k=3, v=5003, dtype="f32", mode="sample",
             draft="point", tau=0.7, masked=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "quantize", "logits", "logits", "logits", "verify", "verify",
                     "verify"])
    if op == "norm":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        d = 8 * _log(rng, 32, 768)
        rows = min(_log(rng, 1, 8192), 8192 * 2048 // d)
        if dtype == "f32":
            rows = max(1, rows // 2)
        return dict(op="norm", rows=rows, d=d, dtype=dtype, residual=rng.random() < 0.7,
                    outputs=rng.choice(["fp8", "fp8", "both", "y"]),
                    offset=rng.choice([0.0, 1.0]))
    if op == "quantize":
        d = 16 * _log(rng, 16, 256)
        v = min(_log(rng, 1000, 128256), 128256 * 1024 // d)
        return dict(op="quantize", v=v, d=d, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "logits":
        d = 16 * _log(rng, 16, 256)
        v = min(_log(rng, 1000, 262144), 128256 * 2048 // d)
        rows = min(_log(rng, 1, 2048), max(1, 2048 * 128256 * 2048 // (v * d)))
        return dict(op="logits", rows=rows, v=v, d=d, out=rng.choice(["bf16", "f32"]))
    B, k, v = _log(rng, 1, 64), rng.randint(0, 8), _log(rng, 1000, 262144)
    B = max(1, min(B, 64 * 8 * 128256 // (2 * (k + 1) * v)))
    return dict(op="verify", B=B, k=k, v=v, dtype=rng.choice(["bf16", "f32"]),
                mode=rng.choice(["sample", "sample", "greedy"]),
                draft=rng.choice(["dense", "dense", "point"]),
                tau=rng.choice([0.5, 0.7, 1.0, 1.3]), masked=rng.random() < 0.3)


def _blocks(n):
    return -(-n // BLOCK)


def _counts(case):
    """Drafted tokens of each sequence: 0 to k of them, the same for every seed."""
    B, k = case["B"], case["k"]
    return [k if s == 0 else (5 * s + 2) % (k + 1) for s in range(B)]


def work(case):
    op = case["op"]
    if op == "norm":
        n, es = case["rows"] * case["d"], 2 if case["dtype"] == "bf16" else 4
        moved = n * es * (3 if case["residual"] else 1) + case["d"] * es
        if case["outputs"] != "fp8":
            moved += n * es
        if case["outputs"] != "y":
            moved += n + 4 * case["rows"] * _blocks(case["d"])
        return {"bytes": moved, "flops": 6 * n}
    if op == "quantize":
        n, es = case["v"] * case["d"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * es + n + 4 * _blocks(case["v"]) * _blocks(case["d"]), "flops": 3 * n}
    if op == "logits":
        m, v, d = case["rows"], case["v"], case["d"]
        moved = (m + v) * d + 4 * (m + _blocks(v)) * _blocks(d)
        return {"bytes": moved + m * v * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * m * v * d}
    # every row's logits; the draft's probabilities of one row a sequence
    # (where a token is drawn from what is left of a rejected one)
    rows = case["B"] + sum(_counts(case))
    n = rows * case["v"]
    moved = n * (2 if case["dtype"] == "bf16" else 4)
    if case["draft"] == "dense" and case["mode"] == "sample" and case["k"]:
        moved += 4 * case["B"] * case["v"]
    return {"bytes": moved + 16 * case["B"] * (case["k"] + 2), "flops": 4 * n}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _padded(rows, cols, dtype):
    """An uninitialised rows x cols matrix whose rows start at multiples of 16 bytes."""
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    return torch.empty(rows, -(-cols // per) * per, dtype=dtype, device="cuda")[:, :cols]


def _block_scales(x, by):
    """max |x| / 448 of each block of by x 128 values."""
    rows, cols = x.shape
    full = torch.zeros(-(-rows // by) * by, _blocks(cols) * BLOCK, device=x.device)
    full[:rows, :cols] = x
    top = full.view(full.shape[0] // by, by, -1, BLOCK).abs().amax((1, 3))
    return (top / E4M3_MAX).clamp(min=TINY)


def _spread(scale, by, rows, cols):
    """The scale of every value of a rows x cols matrix."""
    if by > 1:
        scale = scale.repeat_interleave(by, 0)[:rows]
    return scale.repeat_interleave(BLOCK, 1)[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    s = {"case": case}
    if op == "norm":
        rows, d, t = case["rows"], case["d"], DTYPES[case["dtype"]]
        # a few columns stand out, as in the residual stream of a trained model
        gain = torch.exp(normal(d) * 0.5)
        s["x"] = (normal(rows, d) * gain).to(t)
        s["residual"] = (normal(rows, d) * gain * 4).to(t) if case["residual"] else None
        s["weight"] = (normal(d, scale=0.2) + (1.0 - case["offset"])).to(t)
        s["residual_out"] = torch.empty(rows, d, dtype=t, device="cuda") if case["residual"] else None
        s["y"] = torch.empty(rows, d, dtype=t, device="cuda") if case["outputs"] != "fp8" else None
        s["y8"] = s["y_scale"] = None
        if case["outputs"] != "y":
            s["y8"] = torch.empty(rows, d, dtype=torch.float8_e4m3fn, device="cuda")
            s["y_scale"] = torch.empty(rows, _blocks(d), device="cuda")
    elif op == "quantize":
        v, d = case["v"], case["d"]
        s["E"] = (normal(v, d, scale=0.02) * torch.exp(normal(v, 1) * 0.25)).to(DTYPES[case["dtype"]])
        s["E8"] = torch.empty(v, d, dtype=torch.float8_e4m3fn, device="cuda")
        s["E_scale"] = torch.empty(_blocks(v), _blocks(d), device="cuda")
    elif op == "logits":
        rows, v, d = case["rows"], case["v"], case["d"]
        h = normal(rows, d) * torch.exp(normal(d) * 0.5)
        s["h_scale"] = _block_scales(h, 1)
        s["h8"] = (h / _spread(s["h_scale"], 1, rows, d)).to(torch.float8_e4m3fn)
        E = normal(v, d, scale=0.02)
        s["E_scale"] = _block_scales(E, BLOCK)
        s["E8"] = (E / _spread(s["E_scale"], BLOCK, v, d)).to(torch.float8_e4m3fn)
        s["out"] = _padded(rows, v, DTYPES[case["out"]])
    else:
        B, k, v, t = case["B"], case["k"], case["v"], DTYPES[case["dtype"]]
        counts = _counts(case)
        rows, drafts = B + sum(counts), sum(counts)
        starts = np.concatenate([[0], np.cumsum([n + 1 for n in counts])])
        s["row_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        # target rows of drafted tokens, in the drafts' order
        at = [r for b in range(B) for r in range(starts[b], starts[b + 1] - 1)]
        at = torch.tensor(at, dtype=torch.long, device="cuda")
        logits = normal(rows, v, scale=2.5)
        if case["masked"]:  # tokens that a grammar forbids, the same ones at a position for the draft
            logits[torch.rand(rows, v, generator=g, device="cuda") < 0.6] = -math.inf
        s["logits"] = _padded(rows, v, t)
        s["logits"].copy_(logits)
        z = logits[at]
        z = (z + normal(drafts, v, scale=0.5)) / case["tau"]
        q = torch.exp(z - z.amax(1, keepdim=True)) if drafts else z
        if case["draft"] == "dense":
            s["draft_probs"] = _padded(drafts, v, torch.float32)
            s["draft_probs"].copy_(q / q.sum(1, keepdim=True) if drafts else q)
            race = q / torch.empty_like(q).exponential_(generator=g)
        else:
            s["draft_probs"] = None
            race = q
        s["draft_tokens"] = (race.argmax(1) if drafts else at).to(torch.int32)
        s["u_accept"] = torch.rand(drafts, generator=g, device="cuda")
        s["u_sample"] = torch.rand(B, generator=g, device="cuda")
        s["out_tokens"] = torch.empty(B, k + 1, dtype=torch.int32, device="cuda")
        s["out_accepted"] = torch.empty(B, dtype=torch.int32, device="cuda")
        s["out_logp"] = torch.empty(B, k + 1, device="cuda")
        s["workspace"] = None
        if own:
            from two_stage_retrieval_amd import binding
            s["workspace"] = torch.empty(binding.flashhead_verify_workspace_bytes(B, rows, v),
                                         dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

EPS = 1e-6


def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    from two_stage_retrieval_amd import binding as fh
    case = s["case"]
    if case["op"] == "norm":
        fh.flashhead_rmsnorm(s["x"], s["weight"], residual=s["residual"],
                             residual_out=s["residual_out"], y=s["y"], y8=s["y8"],
                             y_scale=s["y_scale"], eps=EPS, weight_offset=case["offset"])
        return {n: s[n] for n in ("residual_out", "y", "y8", "y_scale")}
    if case["op"] == "quantize":
        fh.flashhead_quantize_fp8(s["E"], s["E8"], s["E_scale"])
        return {n: s[n] for n in ("E8", "E_scale")}
    if case["op"] == "logits":
        fh.dense_logits_fp8(s["h8"], s["h_scale"], s["E8"], s["E_scale"], s["out"])
        return {"out": s["out"]}
    sample = case["mode"] == "sample"
    fh.flashhead_verify(s["logits"], s["row_start"], s["draft_tokens"], s["out_tokens"],
                        s["out_accepted"], s["workspace"],
                        mode=fh.FH_MODE_SAMPLE if sample else fh.FH_MODE_GREEDY, tau=case["tau"],
                        draft_probs=s["draft_probs"] if sample else None,
                        u_accept=s["u_accept"] if sample else None,
                        u_sample=s["u_sample"] if sample else None, out_logp=s["out_logp"])
    return {n: s[n] for n in ("out_tokens", "out_accepted", "out_logp")}


def _plain(s):
    case = s["case"]
    if case["op"] == "norm":
        return _plain_norm(s, case)
    if case["op"] == "quantize":
        E = s["E"].float()
        scale = _block_scales(E, BLOCK)
        return {"E8": (E / _spread(scale, BLOCK, *E.shape)).to(torch.float8_e4m3fn),
                "E_scale": scale}
    if case["op"] == "logits":
        h, E = s["h8"].float(), s["E8"].float()
        h = h * _spread(s["h_scale"], 1, *h.shape)
        E = E * _spread(s["E_scale"], BLOCK, *E.shape)
        return {"out": torch.matmul(h, E.t()).to(s["out"].dtype)}
    return _plain_verify(s, case)


def _plain_norm(s, case):
    t = s["x"].dtype
    x = s["x"].float()
    if case["residual"]:
        x = x + s["residual"].float()
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    y = y * (s["weight"].float() + case["offset"])
    out = {"residual_out": x.to(t) if case["residual"] else None,
           "y": y.to(t) if case["outputs"] != "fp8" else None, "y8": None, "y_scale": None}
    if case["outputs"] != "y":
        out["y_scale"] = _block_scales(y, 1)
        out["y8"] = (y / _spread(out["y_scale"], 1, *y.shape)).to(torch.float8_e4m3fn)
    return out


def _plain_verify(s, case):
    # 64 bits: a drawn token is decided by a sum over the vocabulary, and one
    # in 32 bits is off by more than the share of most tokens
    B, k = case["B"], case["k"]
    sample, tau = case["mode"] == "sample", case["tau"] if case["mode"] == "sample" else 1.0
    start = s["row_start"].long()
    first, n = start[:-1], start[1:] - start[:-1] - 1
    z = s["logits"].double()
    top = z.amax(1, keepdim=True)
    e = torch.exp((z - top) / tau)
    total = e.sum(1, keepdim=True)
    best = (z == top).to(torch.uint8).argmax(1)
    # the drafts of every sequence, padded to k columns
    j = torch.arange(k, device=z.device)
    there = j < n[:, None]
    row = torch.where(there, first[:, None] + j, 0)
    d = torch.where(there, row - torch.arange(B, device=z.device)[:, None], 0)
    x = torch.zeros(B, k, dtype=torch.long, device=z.device)
    if s["draft_tokens"].numel():
        x = s["draft_tokens"].long()[d]
        if sample:
            p = e[row, x] / total[row, 0]
            q = s["draft_probs"][d, x].double() if s["draft_probs"] is not None else 1.0
            taken = s["u_accept"][d].double() * q < p
        else:
            taken = x == best[row]
    else:
        taken = there
    a = (taken & there).long().cumprod(1).sum(1)
    at = first + a
    rejected = a < n
    if sample:
        w = e[at] / total[at]
        p = w.clone()
        if s["draft_tokens"].numel():
            of = torch.where(rejected, at - torch.arange(B, device=z.device), 0)
            if s["draft_probs"] is not None:
                less = (w - s["draft_probs"][of].double()).clamp(min=0)
            else:
                less = w.scatter(1, s["draft_tokens"].long()[of][:, None], 0.0)
            w = torch.where(rejected[:, None], less, w)
        c = w.cumsum(1)
        c = torch.where(c[:, -1:] > 0, c, p.cumsum(1))
        u = s["u_sample"].double()[:, None] * c[:, -1:]
        last = (c <= u).sum(1).clamp(max=z.shape[1] - 1)
    else:
        last = best[at]
    i = torch.arange(k + 1, device=z.device)
    x = torch.cat([x, torch.zeros_like(x[:, :1]) if k else x.new_zeros(B, 1)], 1)
    tokens = torch.where(i < a[:, None], x, torch.where(i == a[:, None], last[:, None], -1))
    row = torch.minimum(first[:, None] + i, at[:, None])
    y = tokens.clamp(min=0)
    logp = (z[row, y] - top[row, 0]) / tau - torch.log(total[row, 0])
    return {"out_tokens": tokens.int(), "out_accepted": a.int(),
            "out_logp": torch.where(tokens >= 0, logp, 0.0).float()}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        t = s["x"].double()
        if s["residual"] is not None:
            t = t + s["residual"].double()
        w = s["weight"].double() + case["offset"]
        y = t / torch.sqrt(torch.sum(t * t, 1, keepdim=True) / case["d"] + EPS) * w
        out = {"residual_out": t if s["residual"] is not None else None,
               "y": y if case["outputs"] != "fp8" else None, "y8": None, "y_scale": None}
        if case["outputs"] != "y":
            parts = [y[:, i:i + BLOCK] for i in range(0, case["d"], BLOCK)]
            tops = [torch.clamp(b.abs().max(1, keepdim=True).values / E4M3_MAX, min=TINY)
                    for b in parts]
            out["y_scale"] = torch.cat(tops, 1)
            out["y8"] = torch.cat([b / top for b, top in zip(parts, tops)], 1)
        return out
    if case["op"] == "quantize":
        E = s["E"].double()
        out, scales = torch.empty_like(E), torch.empty(s["E_scale"].shape, dtype=torch.float64)
        for j in range(0, case["d"], BLOCK):
            strip = E[:, j:j + BLOCK]
            tops = [strip[i:i + BLOCK].abs().max() for i in range(0, case["v"], BLOCK)]
            tops = torch.clamp(torch.stack(tops) / E4M3_MAX, min=TINY)
            scales[:, j // BLOCK] = tops.cpu()
            rows = torch.arange(case["v"], device=E.device) // BLOCK
            out[:, j:j + BLOCK] = strip / tops[rows][:, None]
        return {"E8": out, "E_scale": scales}
    if case["op"] == "logits":
        z = torch.zeros(case["rows"], case["v"], dtype=torch.float64, device="cuda")
        rows = torch.arange(case["v"], device="cuda") // BLOCK
        for j in range(0, case["d"], BLOCK):
            b = j // BLOCK
            part = s["h8"][:, j:j + BLOCK].double() @ s["E8"][:, j:j + BLOCK].double().t()
            z += part * s["h_scale"][:, b, None].double() * s["E_scale"][:, b].double()[rows]
        return {"out": z}
    return _exact_verify(s, case)


def _exact_verify(s, case):
    h = {n: x.cpu() if isinstance(x, torch.Tensor) else x for n, x in s.items()}
    sample, tau = case["mode"] == "sample", case["tau"] if case["mode"] == "sample" else 1.0
    B, k = case["B"], case["k"]
    start, draft = h["row_start"].tolist(), h["draft_tokens"].tolist()
    tokens, logp = np.full((B, k + 1), -1, np.int32), np.zeros((B, k + 1))
    accepted = np.zeros(B, np.int32)

    def target(r):
        z = h["logits"][r].double().numpy()
        t = (z - z.max()) / tau
        return np.exp(t) / np.exp(t).sum(), t - math.log(np.exp(t).sum()), int(z.argmax())

    for b in range(B):
        n = start[b + 1] - start[b] - 1
        for i in range(n + 1):
            p, lp, best = target(start[b] + i)
            at = start[b] + i - b
            if i < n:
                x = draft[at]
                q = None
                if sample and h["draft_probs"] is not None:
                    q = h["draft_probs"][at].double().numpy()
                    take = float(h["u_accept"][at]) * q[x] < p[x]
                elif sample:
                    take = float(h["u_accept"][at]) < p[x]
                else:
                    take = x == best
                if take:
                    tokens[b, i], logp[b, i] = x, lp[x]
                    accepted[b] += 1
                    continue
            y = best
            if sample:
                w = p.copy()
                if i < n and q is None:
                    w[x] = 0.0
                elif i < n:
                    w = np.maximum(p - q, 0.0)
                c = np.cumsum(w if w.sum() > 0 else p)
                y = min(int(np.searchsorted(c, float(h["u_sample"][b]) * c[-1], side="right")),
                        case["v"] - 1)
            tokens[b, i], logp[b, i] = y, lp[y]
            break
    return {"out_tokens": torch.from_numpy(tokens), "out_accepted": torch.from_numpy(accepted),
            "out_logp": torch.from_numpy(logp)}
