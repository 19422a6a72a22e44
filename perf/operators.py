"""The two ends of a masked-diffusion model around its loss: the token embedding
and its gradient, the final norm and its gradient, and 8-bit activation
checkpoints, each in a plain form (elementary torch operations, 32 bits) and
through the library's calls (`own`).

  embed       out[i] = scale * table[ids[i]]; an id outside [0, V) gives zeros
  embed_grad  d_table[v] (+)= scale * sum of d_out[i] over ids[i] = v
  norm        y = xhat * weight + bias, layer norm or RMS norm
  norm_grad   dx, d_weight, d_bias from dy, x and the saved statistics
  norm_ckpt   a training pass of the norm that keeps x as an 8-bit checkpoint:
              the forward pass writes it, the gradients are formed from it
  ckpt        an activation stored in 8 bits and restored
"""

import math

import torch

own = False

BLOCK = 128      # entries that share a scale in an 8-bit checkpoint
TOP = 448.0      # the largest value of the 8-bit format (e4m3)
NORM_EPS = 1e-5


def listed():
    return [
        # one new token of a tiny float32 model: what a call costs by itself
        dict(name="embed-one-token-f32", op="embed", n=1, H=128, V=1024, dtype="f32",
             ids="absorb", scale=1.0, pad=0),
        # a micro-batch of 4,096 absorbing-corrupted tokens, 8B shape
        dict(name="embed-4096x4096", op="embed", n=4096, H=4096, V=126464, dtype="bf16",
             ids="absorb", scale=1.0, pad=0),
        # eight canvases of 1,024 uniformly corrupted tokens, embeddings scaled by sqrt(H)
        dict(name="embed-canvas-8192x2816", op="embed", n=8192, H=2816, V=262144, dtype="bf16",
             ids="uniform", scale=math.sqrt(2816.0), pad=0),
        # the 8B shape's table gradient: half of the tokens are the mask token
        dict(name="embed-grad-4096x4096", op="embed_grad", n=4096, H=4096, V=126464,
             dtype="bf16", ids="absorb", scale=1.0, pad=0, accumulate=False),
        # a tied head: the canvas gradient is added to the head's own
        dict(name="embed-grad-tied-8192x2816", op="embed_grad", n=8192, H=2816, V=262144,
             dtype="bf16", ids="uniform", scale=math.sqrt(2816.0), pad=0, accumulate=True),
        # odd sizes in float32, a padded tail
        dict(name="embed-grad-odd-f32", op="embed_grad", n=777, H=1001, V=5003, dtype="f32",
             ids="absorb", scale=2.5, pad=19, accumulate=False),
        # one row of the 8B shape
        dict(name="norm-one-row", op="norm", n=1, H=4096, dtype="bf16", kind="layer", bias=True),
        # a packed batch before the head, RMS norm
        dict(name="norm-rms-16384x4096", op="norm", n=16384, H=4096, dtype="bf16", kind="rms",
             bias=False),
        # the canvas batch's norm gradient
        dict(name="norm-grad-8192x2816", op="norm_grad", n=8192, H=2816, dtype="bf16",
             kind="layer", bias=True),
        # odd sizes in float32
        dict(name="norm-grad-odd-f32", op="norm_grad", n=1237, H=1001, dtype="f32", kind="layer",
             bias=True),
        # a training pass of the final norm with an 8-bit checkpoint of its input
        dict(name="norm-ckpt-16384x4096", op="norm_ckpt", n=16384, H=4096, dtype="bf16",
             kind="layer", bias=True),
        # an activation of a packed batch stored in 8 bits and restored
        dict(name="ckpt-16384x4096", op="ckpt", n=16384, H=4096, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "embed_grad", "norm", "norm_grad", "norm_ckpt",
                     "ckpt"])
    H = _log(rng, 64, 8192)
    if rng.random() < 0.6:
        H = (H + 63) // 64 * 64
    n = min(_log(rng, 1, 32768), 4096 * 16384 // H)
    c = dict(op=op, n=n, H=H, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op.startswith("embed"):
        V = min(_log(rng, 500, 262144), 500_000_000 // H)
        c.update(V=V, ids=rng.choice(["absorb", "uniform"]),
                 scale=rng.choice([1.0, math.sqrt(H)]),
                 pad=rng.choice([0, 0, n // 7]))
        if op == "embed_grad":
            c["accumulate"] = rng.random() < 0.5
    elif op != "ckpt":
        c.update(kind=rng.choice(["layer", "rms"]), bias=rng.random() < 0.5)
    return c


_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _activations(n, H, dt, gen):
    """Hidden states as a residual stream has them: a row scale that varies,
    an offset, and a few channels far larger than the rest."""
    x = torch.randn(n, H, device="cuda", generator=gen)
    x *= 0.5 + 2.0 * torch.rand(n, 1, device="cuda", generator=gen)
    ch = torch.randint(0, H, (max(1, H // 500),), device="cuda", generator=gen)
    x[:, ch] *= 25.0
    x += 0.3
    return x.to(dt)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n, H, dt = case["n"], case["H"], _DT[case["dtype"]]
    s = {"case": case}
    if case["op"].startswith("embed"):
        V = case["V"]
        ids = torch.randint(0, V, (n,), device="cuda", generator=gen, dtype=torch.int32)
        if case["ids"] == "absorb":  # about half of the tokens are the mask token
            hide = torch.rand(n, device="cuda", generator=gen) < 0.5
            ids[hide] = V - 1
        if case["pad"]:
            ids[n - case["pad"]:] = -1
        s["ids"] = ids
        if case["op"] == "embed":
            s["table"] = torch.empty(V, H, device="cuda", dtype=dt).normal_(
                0.0, 0.02, generator=gen)
            s["out"] = torch.empty(n, H, device="cuda", dtype=dt)
        else:
            s["d_out"] = (torch.randn(n, H, device="cuda", generator=gen) * 1e-3).to(dt)
            s["d_table"] = torch.empty(V, H, device="cuda")
            if case["accumulate"]:
                s["d_table"].normal_(0.0, 1e-3, generator=gen)
        return s
    s["x"] = _activations(n, H, dt, gen)
    if case["op"] in ("norm_ckpt", "ckpt"):
        s["q"] = torch.empty(n, H, device="cuda", dtype=torch.uint8)
        s["q_exp"] = torch.empty(n, -(-H // BLOCK), device="cuda", dtype=torch.uint8)
    if case["op"] == "ckpt":
        s["restored"] = torch.empty(n, H, device="cuda", dtype=dt)
        return s
    s["weight"] = (1.0 + 0.1 * torch.randn(H, device="cuda", generator=gen)).to(dt)
    s["bias"] = ((0.1 * torch.randn(H, device="cuda", generator=gen)).to(dt) if case["bias"]
                 else None)
    s["y"] = torch.empty_like(s["x"])
    s["rstd"] = torch.empty(n, device="cuda")
    s["mean"] = torch.empty(n, device="cuda") if case["kind"] == "layer" else None
    if case["op"] != "norm":
        s["dy"] = (torch.randn(n, H, device="cuda", generator=gen) * 1e-3).to(dt)
        s["dx"] = torch.empty_like(s["x"])
        s["d_weight"] = torch.empty(H, device="cuda")
        s["d_bias"] = torch.empty(H, device="cuda") if case["bias"] else None
    if case["op"] == "norm_grad":  # the forward pass left its statistics
        m, r = _stats(s["x"].float(), case["kind"])
        s["rstd"].copy_(r.squeeze(1))
        if s["mean"] is not None:
            s["mean"].copy_(m.squeeze(1))
    return s


# ---- plain forms --------------------------------------------------------


def _stats(xf, kind):
    mean = xf.mean(1, keepdim=True) if kind == "layer" else None
    d = xf if mean is None else xf - mean
    return mean, torch.rsqrt((d * d).mean(1, keepdim=True) + NORM_EPS)


def _norm(x, kind, weight, bias):
    xf = x.float()
    mean, rstd = _stats(xf, kind)
    y = (xf if mean is None else xf - mean) * rstd * weight.float()
    if bias is not None:
        y = y + bias.float()
    return y.to(x.dtype), mean, rstd


def _norm_grad(dy, xf, kind, weight, bias, mean, rstd):
    g = dy.float()
    xhat = (xf if kind == "rms" else xf - mean) * rstd
    gw = g * weight.float()
    dx = gw - xhat * (gw * xhat).mean(1, keepdim=True)
    if kind == "layer":
        dx = dx - gw.mean(1, keepdim=True)
    out = {"dx": (dx * rstd).to(dy.dtype), "d_weight": (g * xhat).sum(0)}
    if bias is not None:
        out["d_bias"] = g.sum(0)
    return out


def _store(x):
    """The checkpoint of x: e4m3 values and the power of two they stand over."""
    n, H = x.shape
    xf = torch.nn.functional.pad(x.float(), (0, -H % BLOCK)).view(n, -1, BLOCK)
    top = xf.abs().amax(2, keepdim=True)
    m, k = torch.frexp(top)  # top = m 2^k, m in [1/2, 1)
    e = torch.where(m <= TOP / 512.0, k - 9, k - 8)
    e = torch.where(top > 0, e, -127).clamp(min=-127)
    return torch.ldexp(xf, -e).to(torch.float8_e4m3fn), e


def _restore(q, e, H):
    return torch.ldexp(q.float(), e).view(q.shape[0], -1)[:, :H]


def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "embed":
        ids, table = s["ids"], s["table"]
        ok = (ids >= 0) & (ids < c["V"])
        rows = table[torch.where(ok, ids, 0).long()].float() * c["scale"]
        return torch.where(ok[:, None], rows, 0.0).to(table.dtype)
    if c["op"] == "embed_grad":
        ids, d_table = s["ids"], s["d_table"]
        ok = (ids >= 0) & (ids < c["V"])
        rows = torch.where(ok[:, None], s["d_out"].float() * c["scale"], 0.0)
        if not c["accumulate"]:
            d_table.zero_()
        return d_table.index_add_(0, torch.where(ok, ids, 0), rows)
    if c["op"] == "ckpt":
        q, e = _store(s["x"])
        return _restore(q, e, c["H"]).to(s["x"].dtype)
    if c["op"] == "norm_grad":
        mean = None if s["mean"] is None else s["mean"][:, None]
        return _norm_grad(s["dy"], s["x"].float(), c["kind"], s["weight"], s["bias"], mean,
                          s["rstd"][:, None])
    y, mean, rstd = _norm(s["x"], c["kind"], s["weight"], s["bias"])
    out = {"y": y, "rstd": rstd.squeeze(1)}
    if mean is not None:
        out["mean"] = mean.squeeze(1)
    if c["op"] == "norm_ckpt":
        q, e = _store(s["x"])
        out.update(_norm_grad(s["dy"], _restore(q, e, c["H"]), c["kind"], s["weight"], s["bias"],
                              mean, rstd))
    return out


# ---- the library's calls ------------------------------------------------


def _run_own(s, c):
    from uniform_noise_diffusion_amd import binding as B
    if c["op"] == "embed":
        B.mdlm_embed(s["ids"], s["table"], c["scale"], s["out"])
        return s["out"]
    if c["op"] == "embed_grad":
        B.mdlm_embed_grad(s["ids"], s["d_out"], c["scale"], s["d_table"], c["accumulate"])
        return s["d_table"]
    if c["op"] == "ckpt":
        B.mdlm_ckpt8_save(s["x"], s["q"], s["q_exp"])
        B.mdlm_ckpt8_load(s["q"], s["q_exp"], s["restored"])
        return s["restored"]
    kind = B.MDLM_NORM_LAYER if c["kind"] == "layer" else B.MDLM_NORM_RMS
    out = {}
    if c["op"] != "norm_grad":
        q, q_exp = s.get("q"), s.get("q_exp")
        B.mdlm_norm_fwd(s["x"], kind, s["weight"], s["bias"], NORM_EPS, s["y"], s["mean"],
                        s["rstd"], q, q_exp)
        out.update(y=s["y"], rstd=s["rstd"])
        if s["mean"] is not None:
            out["mean"] = s["mean"]
    if c["op"] == "norm_grad":
        B.mdlm_norm_bwd(s["dy"], s["x"], kind, s["weight"], s["mean"], s["rstd"], s["dx"],
                        s["d_weight"], s["d_bias"])
    elif c["op"] == "norm_ckpt":
        B.mdlm_norm_bwd_ckpt8(s["dy"], s["q"], s["q_exp"], kind, s["weight"], s["mean"],
                              s["rstd"], s["dx"], s["d_weight"], s["d_bias"])
    if c["op"] != "norm":
        out.update(dx=s["dx"], d_weight=s["d_weight"])
        if s["d_bias"] is not None:
            out["d_bias"] = s["d_bias"]
    return out


def work(case):
    n, H = case["n"], case["H"]
    b = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("embed"):
        # distinct ids expected among the drawn ones: the table rows touched
        m = n - case["pad"]
        if case["ids"] == "absorb":
            m = (m + 1) // 2
        rows = case["V"] * -math.expm1(m * math.log1p(-1.0 / case["V"]))
        if case["ids"] == "absorb" and n > 1:
            rows += 1
        if case["op"] == "embed":
            return {"bytes": 4 * n + b * H * (rows + n), "flops": n * H}
        table = 8 * rows * H if case["accumulate"] else 4 * case["V"] * H
        return {"bytes": 4 * n + b * n * H + table, "flops": 2 * n * H}
    q = H + -(-H // BLOCK)
    params = b * H * (2 if case.get("bias") else 1)
    stats = 4 * n * (2 if case.get("kind") == "layer" else 1)
    grads = 4 * H * (2 if case.get("bias") else 1)
    if case["op"] == "ckpt":  # x read, the checkpoint written and read, x written
        return {"bytes": 2 * n * (b * H + q), "flops": 4 * n * H}
    fwd = {"bytes": 2 * n * b * H + params + stats, "flops": 8 * n * H}
    bwd = {"bytes": 3 * n * b * H + params + stats + grads, "flops": 14 * n * H}
    if case["op"] == "norm":
        return fwd
    if case["op"] == "norm_grad":
        return bwd
    return {"bytes": fwd["bytes"] + bwd["bytes"] + n * (2 * q - b * H),
            "flops": fwd["flops"] + bwd["flops"] + 4 * n * H}


# ---- the definitions in 64 bits -----------------------------------------


def _held(x64):
    """What an 8-bit checkpoint of x stands for: in each block of 128, the
    least power of two 2^e >= 2^-127 with |x| <= 448 * 2^e, and x / 2^e
    rounded to the nearest e4m3 value (3 fraction bits, exponents from -6)."""
    n, H = x64.shape
    out = torch.empty_like(x64)
    for lo in range(0, H, BLOCK):
        blk = x64[:, lo:lo + BLOCK]
        top = blk.abs().max(1, keepdim=True).values
        e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -200) / TOP))
        # log2 may be off by one where top / 448 is a power of two
        e = torch.where(TOP * torch.exp2(e - 1) >= top, e - 1, e)
        e = torch.where(TOP * torch.exp2(e) < top, e + 1, e).clamp(min=-127.0)
        v = blk * torch.exp2(-e)
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)
        out[:, lo:lo + BLOCK] = torch.round(v / step) * step * torch.exp2(e)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    n, H = case["n"], case["H"]
    if case["op"].startswith("embed"):
        ids = s["ids"].long()
        keep = torch.nonzero((ids >= 0) & (ids < case["V"])).squeeze(1)
        if case["op"] == "embed":
            out = torch.zeros(n, H, device="cuda", dtype=torch.float64)
            out[keep] = s["table"].index_select(0, ids[keep]).double() * case["scale"]
            return out
        d_table = (s["d_table"].double() if case["accumulate"]
                   else torch.zeros(case["V"], H, device="cuda", dtype=torch.float64))
        order = keep[torch.argsort(ids[keep], stable=True)]
        which, count = torch.unique_consecutive(ids[order], return_counts=True)
        end = torch.cumsum(count, 0)
        # sums over runs of equal ids as differences of running sums
        run_sum = torch.cumsum(s["d_out"][order].double(), 0)[end - 1]
        run_sum[1:] -= run_sum[:-1].clone()
        d_table[which] += run_sum * case["scale"]
        return d_table
    x = s["x"].double()
    if case["op"] == "ckpt":
        return _held(x)
    w = s["weight"].double()
    mu = x.sum(1) / H if case["kind"] == "layer" else torch.zeros(n, device="cuda",
                                                                  dtype=torch.float64)
    var = ((x - mu[:, None]) ** 2).sum(1) / H
    inv = (var + NORM_EPS) ** -0.5
    out = {}
    if case["op"] != "norm_grad":
        y = (x - mu[:, None]) * inv[:, None] * w
        out["y"] = y if s["bias"] is None else y + s["bias"].double()
        out["rstd"] = inv
        if case["kind"] == "layer":
            out["mean"] = mu
    if case["op"] == "norm":
        return out
    if case["op"] == "norm_grad":  # the statistics are inputs
        inv = s["rstd"].double()
        mu = s["mean"].double() if case["kind"] == "layer" else mu
    else:
        x = _held(x)
    g = s["dy"].double()
    z = (x - mu[:, None]) * inv[:, None]
    gw = g * w
    dot = (gw * z).sum(1) / H
    avg = gw.sum(1) / H if case["kind"] == "layer" else torch.zeros_like(dot)
    out["dx"] = inv[:, None] * (gw - avg[:, None] - dot[:, None] * z)
    out["d_weight"] = (g * z).sum(0)
    if s["bias"] is not None:
        out["d_bias"] = g.sum(0)
    return out
