"""Workloads of the training operators beside the sparse attention: causal
attention over packed sequences with grouped heads (forward and backward),
layer norm (forward and backward) and the clipping of gradients by their
global norm.

``run`` computes a pass either in its plain form (elementary torch
operations in float32, rounded once at the end) or, where ``own`` is true,
by the library's entry points; ``exact`` gives the same outputs from the
definitions in float64.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEVICE = "cuda"


def _lengths(text):
    return [int(x) for x in text.split(",")]


def listed():
    return [
        # A handful of short byte strings in one batch: one launch's latency.
        dict(name="attn-fwd-short", op="attn_fwd", lengths="1,17,130,64,5", hq=4, hkv=4, d=64, dtype="bf16"),
        # The byte-level text workload's shape (8 heads of 64, N = 12288), two documents that fill their windows.
        dict(name="attn-fwd-text", op="attn_fwd", lengths="12288,12288", hq=8, hkv=8, d=64, dtype="bf16"),
        # Ragged documents packed into one batch, four query heads to a K/V head.
        dict(name="attn-fwd-ragged-grouped", op="attn_fwd",
             lengths="4099,1,2777,640,129,5003,33,1999,128,1575", hq=32, hkv=8, d=128, dtype="fp16"),
        # One long document, eight query heads to a K/V head.
        dict(name="attn-fwd-long", op="attn_fwd", lengths="32768", hq=16, hkv=2, d=128, dtype="bf16"),
        # The backward passes of the same kinds of batch.
        dict(name="attn-bwd-short", op="attn_bwd", lengths="97,128,45,201,16,111,1,77", hq=4, hkv=2, d=64,
             dtype="fp16"),
        dict(name="attn-bwd-text", op="attn_bwd", lengths="12288,12288", hq=8, hkv=8, d=64, dtype="bf16"),
        dict(name="attn-bwd-ragged-grouped", op="attn_bwd",
             lengths="4099,1,2777,640,129,5003,33,1999,128,1575", hq=32, hkv=8, d=128, dtype="bf16"),
        # The text block's activations: 2 x 12288 positions of width 512.
        dict(name="norm-fwd-text", op="norm_fwd", rows=24576, c=512, dtype="bf16", pad=0, bias=True),
        # A few rows of an odd width in float32: latency.
        dict(name="norm-fwd-few", op="norm_fwd", rows=3, c=1001, dtype="fp32", pad=0, bias=False),
        # The widest model that the block takes.
        dict(name="norm-bwd-wide", op="norm_bwd", rows=16384, c=6144, dtype="bf16", pad=0, bias=True),
        # The text block's eight parameter gradients in float32.
        dict(name="clip-block", op="clip", sizes="512,512,786432,262144,512,512,1048576,1048576", dtypes="fp32",
             clipped=True),
        # The gradients of seven wider blocks in bfloat16 with float32 layer norms: larger than the caches.
        dict(name="clip-model", op="clip",
             sizes=",".join(["2048,2048,12582912,4194304,2048,2048,16777216,16777216"] * 7),
             dtypes=",".join(["fp32,fp32,bf16,bf16,fp32,fp32,bf16,bf16"] * 7), clipped=True),
    ]


# No drawn case costs more than the largest listed one of its operator.
MAX_PAIRS = 32768 * 32769 // 2 * 16 * 128  # (query, key) pairs x heads x head width of attn-fwd-long


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_lengths(rng, total_max):
    total = _log_int(rng, 1, total_max)
    out = []
    while total > 0 and len(out) < 200:
        n = min(total, _log_int(rng, 1, max(1, total)) if rng.random() < 0.5 else _log_int(rng, 1, 2048))
        out.append(n)
        total -= n
    rng.shuffle(out)
    return out


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd", "norm_fwd", "norm_bwd", "clip"])
    if op.startswith("attn"):
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 3, 4, 8])
        hq = hkv * rng.choice([1, 1, 2, 3, 4, 8])
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        cap = MAX_PAIRS if op == "attn_fwd" else MAX_PAIRS * 2 // 5
        while True:
            lens = _draw_lengths(rng, 20000)
            if sum(n * (n + 1) // 2 for n in lens) * hq * d <= cap and sum(lens) * hq * d <= 1 << 27:
                break
        return dict(op=op, lengths=",".join(map(str, lens)), hq=hq, hkv=hkv, d=d, dtype=dtype)
    if op.startswith("norm"):
        c = _log_int(rng, 16, 6144)
        rows = _log_int(rng, 1, max(1, min(65536, 16384 * 6144 // c)))
        return dict(op=op, rows=rows, c=c, dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    pad=rng.choice([0, 0, 8, 24]), bias=rng.random() < 0.7)
    n = _log_int(rng, 1, 60)
    sizes = [_log_int(rng, 1, 1 << 21) for _ in range(n)]
    dtypes = [rng.choice(["fp32", "bf16", "fp16"]) for _ in range(n)]
    return dict(op="clip", sizes=",".join(map(str, sizes)), dtypes=",".join(dtypes), clipped=rng.random() < 0.7)


# ------------------------------------------------------------------- inputs
def _normal(shape, gen, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32) * scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed * 7919 + 17)
    st = dict(case)
    op = case["op"]
    if op.startswith("attn"):
        dt, hq, hkv, d = DTYPES[case["dtype"]], case["hq"], case["hkv"], case["d"]
        lens = _lengths(case["lengths"])
        T = sum(lens)
        # one projection's output holds q, k and v side by side
        qkv = _normal((T, hq + 2 * hkv, d), gen, dt)
        st.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], lens=lens)
        if op == "attn_bwd":
            st["dO"] = _normal((T, hq, d), gen, dt)
            st["o"], st["lse"] = _attn_forward(st["q"], st["k"], st["v"], lens, torch.float32, dt)
        if own:
            from factorized_block_sparse_b200 import packed_attn as pa

            st["layout"] = pa.Layout(lens)
            if op == "attn_bwd":
                st["ws"] = pa.workspace(hq, hkv, d, st["layout"], DEVICE)
    elif op.startswith("norm"):
        dt, rows, c = DTYPES[case["dtype"]], case["rows"], case["c"]
        x = _normal((rows, c + case["pad"]), gen, dt, 1.5) + 0.25
        st["x"] = x[:, :c]
        st["g"] = 1.0 + 0.1 * _normal((c,), gen, torch.float32)
        st["b"] = 0.1 * _normal((c,), gen, torch.float32) if case["bias"] else None
        if op == "norm_bwd":
            st["dy"] = _normal((rows, c + case["pad"]), gen, dt)[:, :c]
            _, st["mean"], st["rstd"] = _norm_forward(st["x"], st["g"], st["b"], torch.float32, dt)
    else:
        sizes, dts = _lengths(case["sizes"]), case["dtypes"].split(",")
        dts = dts * len(sizes) if len(dts) == 1 else dts
        scales = [10.0 ** (-1 - (i % 4)) for i in range(len(sizes))]  # gradients of unlike magnitudes
        st["grads"] = [_normal((n,), gen, DTYPES[t], s) for n, t, s in zip(sizes, dts, scales)]
        st["out"] = [torch.empty_like(g) for g in st["grads"]]
        rms = math.sqrt(sum(n * s * s for n, s in zip(sizes, scales)))
        st["max_norm"] = rms * (0.3 if case["clipped"] else 3.0)
    return st


# -------------------------------------------------------------- plain forms
EPS = 1e-5
ROWS = 4096  # query rows of a score block


def _blocks(lens):
    """(first row of the sequence, first and one-past-last query row in it)."""
    at = 0
    for n in lens:
        for i0 in range(0, n, ROWS):
            yield at, i0, min(n, i0 + ROWS)
        at += n


def _heads_first(x, a, b, w):
    """Rows [a, b) of x [T, H, D] as [H, rows, D] in the working type."""
    return x[a:b].to(w).transpose(0, 1)


def _probs(q, k, i0, scale):
    """Scores of a block of query rows [i0, i0 + rows) against keys [0, i0 + rows), grouped: q [Hkv, G, r, D]."""
    r, n = q.shape[2], k.shape[1]
    s = torch.matmul(q, k.transpose(1, 2).unsqueeze(1)) * scale
    i = torch.arange(i0, i0 + r, device=q.device).unsqueeze(1)
    j = torch.arange(n, device=q.device).unsqueeze(0)
    return s.masked_fill(j > i, -math.inf)


def _attn_forward(q, k, v, lens, w, out):
    T, hq, d = q.shape
    hkv = k.shape[1]
    scale = 1.0 / math.sqrt(d)
    o = torch.empty((T, hq, d), dtype=out, device=q.device)
    lse = torch.empty((hq, T), dtype=w, device=q.device)
    for at, a, b in _blocks(lens):
        # at most about 2^28 scores at a time: heads in groups
        per = max(1, (1 << 28) // ((b - a) * b * (hq // hkv)))
        for h in range(0, hkv, per):
            hs = slice(h, min(hkv, h + per))
            qs = slice(hs.start * (hq // hkv), hs.stop * (hq // hkv))
            kk, vv = (_heads_first(x[:, hs], at, at + b, w) for x in (k, v))
            qq = _heads_first(q[:, qs], at + a, at + b, w).reshape(kk.shape[0], hq // hkv, b - a, d)
            s = _probs(qq, kk, a, scale)
            m = s.amax(-1, keepdim=True)
            e = torch.exp(s - m)
            z = e.sum(-1, keepdim=True)
            oo = torch.matmul(e, vv.unsqueeze(1)) / z
            o[at + a:at + b, qs] = oo.reshape(-1, b - a, d).transpose(0, 1).to(out)
            lse[qs, at + a:at + b] = (m + torch.log(z)).reshape(-1, b - a)
    return o, lse


def _attn_backward(q, k, v, o, lse, dO, lens, w, out):
    T, hq, d = q.shape
    hkv = k.shape[1]
    G = hq // hkv
    scale = 1.0 / math.sqrt(d)
    dq = torch.empty((T, hq, d), dtype=w, device=q.device)
    dk = torch.zeros((T, hkv, d), dtype=w, device=q.device)
    dv = torch.zeros((T, hkv, d), dtype=w, device=q.device)
    for at, a, b in _blocks(lens):
        per = max(1, (1 << 28) // ((b - a) * b * G))
        for h in range(0, hkv, per):
            hs = slice(h, min(hkv, h + per))
            qs = slice(hs.start * G, hs.stop * G)
            kk, vv = (_heads_first(x[:, hs], at, at + b, w) for x in (k, v))
            nh = kk.shape[0]
            qq, oo, gg = (_heads_first(x[:, qs], at + a, at + b, w).reshape(nh, G, b - a, d) for x in (q, o, dO))
            ll = lse[qs, at + a:at + b].to(w).reshape(nh, G, b - a, 1)
            p = torch.exp(_probs(qq, kk, a, scale) - ll)
            delta = (gg * oo).sum(-1, keepdim=True)
            ds = p * (torch.matmul(gg, vv.transpose(1, 2).unsqueeze(1)) - delta) * scale
            dq[at + a:at + b, qs] = torch.matmul(ds, kk.unsqueeze(1)).reshape(-1, b - a, d).transpose(0, 1)
            # the gradients of a shared K/V head add up over its query heads
            pt, st = (x.reshape(nh, G * (b - a), b).transpose(1, 2) for x in (p, ds))
            dv[at:at + b, hs] += torch.matmul(pt, gg.reshape(nh, -1, d)).transpose(0, 1)
            dk[at:at + b, hs] += torch.matmul(st, qq.reshape(nh, -1, d)).transpose(0, 1)
    return dq.to(out), dk.to(out), dv.to(out)


def _norm_forward(x, g, b, w, out):
    xf = x.to(w)
    mean = xf.mean(-1)
    xc = xf - mean.unsqueeze(-1)
    rstd = 1.0 / torch.sqrt((xc * xc).mean(-1) + EPS)
    y = xc * rstd.unsqueeze(-1) * g.to(w)
    if b is not None:
        y = y + b.to(w)
    return y.to(out), mean, rstd


def _norm_backward(x, g, dy, mean, rstd, bias, w, out):
    xh = (x.to(w) - mean.to(w).unsqueeze(-1)) * rstd.to(w).unsqueeze(-1)
    d = dy.to(w)
    dxh = d * g.to(w)
    dx = rstd.to(w).unsqueeze(-1) * (dxh - dxh.mean(-1, keepdim=True) - xh * (dxh * xh).mean(-1, keepdim=True))
    return dx.to(out), (d * xh).sum(0), (d.sum(0) if bias else None)


def _clip(grads, max_norm, w):
    total = sum((g.to(w) * g.to(w)).sum() for g in grads)
    norm = torch.sqrt(total)
    c = torch.clamp(max_norm / (norm + 1e-6), max=1.0)
    return norm, [(g.to(w) * c) for g in grads]


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_plain(s):
    op = s["op"]
    w = torch.float32
    if op == "attn_fwd":
        return _attn_forward(s["q"], s["k"], s["v"], s["lens"], w, s["q"].dtype)
    if op == "attn_bwd":
        return _attn_backward(s["q"], s["k"], s["v"], s["o"], s["lse"], s["dO"], s["lens"], w, s["q"].dtype)
    if op == "norm_fwd":
        return _norm_forward(s["x"], s["g"], s["b"], w, s["x"].dtype)
    if op == "norm_bwd":
        out = _norm_backward(s["x"], s["g"], s["dy"], s["mean"], s["rstd"], s["b"] is not None, w, s["x"].dtype)
        return out if s["b"] is not None else out[:2]
    norm, clipped = _clip(s["grads"], s["max_norm"], w)
    for o, c in zip(s["out"], clipped):
        o.copy_(c)
    return [norm, *s["out"]]


def _run_own(s):
    op = s["op"]
    if op.startswith("attn"):
        from factorized_block_sparse_b200 import packed_attn as pa

        if op == "attn_fwd":
            return pa.forward(s["q"], s["k"], s["v"], s["layout"])
        return pa.backward(s["q"], s["k"], s["v"], s["o"], s["lse"], s["dO"], s["layout"], ws=s["ws"])
    from factorized_block_sparse_b200 import sparse_block as sb

    if op == "norm_fwd":
        return sb.layer_norm(s["x"], s["g"], s["b"], eps=EPS)
    if op == "norm_bwd":
        out = sb.layer_norm_backward(s["x"], s["g"], s["dy"], s["mean"], s["rstd"], bias=s["b"] is not None)
        return out if s["b"] is not None else out[:2]
    return [sb.clip_grads(s["grads"], s["max_norm"], out=s["out"]), *s["out"]]


# --------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    """The outputs of ``run`` from the definitions in float64, one (sequence, head, row block) at a time."""
    s = prepare(case, seed)
    op = case["op"]
    f = torch.float64
    if op.startswith("attn"):
        hq, hkv, d, lens = case["hq"], case["hkv"], case["d"], s["lens"]
        pairs = sum(n * (n + 1) // 2 for n in lens)
        if pairs * hq * d > MAX_PAIRS * 1.01 or len(lens) * hq > 4000:
            return None
        T = sum(lens)
        new = [torch.zeros((T, h, d), dtype=f, device=DEVICE) for h in (hq, hkv, hkv)]
        o, lse = torch.zeros((T, hq, d), dtype=f, device=DEVICE), torch.zeros((hq, T), dtype=f, device=DEVICE)
        start = np.cumsum([0] + lens)
        for a, n in zip(start.tolist(), lens):
            for h in range(hq):
                kd, vd = s["k"][a:a + n, h * hkv // hq].to(f), s["v"][a:a + n, h * hkv // hq].to(f)
                for i0 in range(0, n, 8192):
                    i1 = min(n, i0 + 8192)
                    rows = slice(a + i0, a + i1)
                    qd = s["q"][rows, h].to(f)
                    scores = (qd @ kd[:i1].T) / math.sqrt(d)
                    keep = torch.ones((i1 - i0, i1), dtype=torch.bool, device=DEVICE).tril_(i0)
                    if op == "attn_fwd":
                        scores[~keep] = -math.inf
                        lse[h, rows] = torch.logsumexp(scores, -1)
                        o[rows, h] = torch.exp(scores - lse[h, rows].unsqueeze(-1)) @ vd[:i1]
                        continue
                    p = torch.exp(scores - s["lse"][h, rows].to(f).unsqueeze(-1)) * keep
                    go, oo = s["dO"][rows, h].to(f), s["o"][rows, h].to(f)
                    grad_s = p * (go @ vd[:i1].T - (go * oo).sum(-1).unsqueeze(-1)) / math.sqrt(d)
                    new[0][rows, h] = grad_s @ kd[:i1]
                    new[1][a:a + i1, h * hkv // hq] += grad_s.T @ qd
                    new[2][a:a + i1, h * hkv // hq] += p.T @ go
        return (o, lse) if op == "attn_fwd" else tuple(new)
    if op.startswith("norm"):
        x, g = s["x"].to(f), s["g"].to(f)
        if op == "norm_fwd":
            var, mu = torch.var_mean(x, -1, correction=0, keepdim=True)
            r = (var + EPS) ** -0.5
            y = (x - mu) * r * g
            return (y if s["b"] is None else y + s["b"].to(f)), mu.squeeze(-1), r.squeeze(-1)
        mu, r, dy = s["mean"].to(f)[:, None], s["rstd"].to(f)[:, None], s["dy"].to(f)
        xh, t = (x - mu) * r, dy * g
        c = case["c"]
        dx = r * (t - t.sum(-1, keepdim=True) / c - xh * ((t * xh).sum(-1, keepdim=True) / c))
        out = (dx, (dy * xh).sum(0), dy.sum(0))
        return out if s["b"] is not None else out[:2]
    norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(g.to(f)) for g in s["grads"]]))
    c = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
    return [norm, *[g.to(f) * c for g in s["grads"]]]


# ---------------------------------------------------------- bytes and FLOPs
def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if op.startswith("attn"):
        lens = _lengths(case["lengths"])
        T, pairs = sum(lens), sum(n * (n + 1) // 2 for n in lens)
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        if op == "attn_fwd":  # q, k, v in; o, lse out
            return {"bytes": T * (2 * d * (2 * hq + 2 * hkv) + 4 * hq), "flops": 4 * d * hq * pairs}
        # q, k, v, o, dO, lse in; dq, dk, dv out
        return {"bytes": T * (2 * d * (4 * hq + 4 * hkv) + 4 * hq), "flops": 10 * d * hq * pairs}
    if op.startswith("norm"):
        rows, c, e = case["rows"], case["c"], size[case["dtype"]]
        vec = 4 * c * (2 if case["bias"] else 1)
        if op == "norm_fwd":
            return {"bytes": rows * (2 * c * e + 8) + vec, "flops": 8 * rows * c}
        return {"bytes": rows * (3 * c * e + 8) + 4 * c + vec, "flops": 14 * rows * c}
    sizes, dts = _lengths(case["sizes"]), case["dtypes"].split(",")
    dts = dts * len(sizes) if len(dts) == 1 else dts
    return {"bytes": sum(2 * n * size[t] for n, t in zip(sizes, dts)) + 4, "flops": 3 * sum(sizes)}
