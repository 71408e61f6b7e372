"""Measured cases of an expert layer's other operators in a training step: the layer norm before it, the router with
its balance loss, the activations kept in 8 bits for the backward pass, and the experts' products in 8 bits.

Each case is one pass as a training or serving program makes it.  With `own` false the pass is computed in
elementary torch operations, in 32 bits, rounded once at the end; with `own` true by the library's calls.
The 8-bit format: e4m3 values in blocks of 128, each block with one power of two, 2^(code - 127), the least that
brings the block's largest magnitude to 448 or below; columns are padded with zeros to whole blocks.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 128


def listed():
    return [
        # layer norm of one decoding step of 8 sequences: launch and latency
        dict(name="norm_decode_8", op="norm", way="forward", rows=8, cols=1024, dtype="bf16"),
        # a training micro-batch before the expert layer, forward and all three gradients
        dict(name="norm_step_32k", op="norm", way="step", rows=32768, cols=1024, dtype="bf16"),
        # fp32 training with odd sizes
        dict(name="norm_step_f32_odd", op="norm", way="step", rows=2011, cols=1001, dtype="f32"),
        # routing of one token each of 16 sequences over 32 experts
        dict(name="route_decode_16", op="route", way="forward", rows=16, experts=32, top=2, dtype="f32", dead=0.0),
        # a training micro-batch: routing, balance loss, gradient of the logits
        dict(name="route_step_32k", op="route", way="step", rows=32768, experts=64, top=4, dtype="f32", dead=0.0),
        # bf16 logits (so ties), odd sizes, padded tokens that are routed nowhere
        dict(name="route_step_odd", op="route", way="step", rows=4097, experts=257, top=7, dtype="bf16", dead=0.06),
        # the gated hidden layer of the same experts: its activation, kept in 8 bits, and the backward pass from there
        dict(name="checkpoint_gated_32k", op="checkpoint", way="gated", rows=32768, cols=4096, dtype="bf16"),
        # a small fp32 layer of odd width without a gate
        dict(name="checkpoint_f32_odd", op="checkpoint", way="silu", rows=779, cols=515, dtype="f32"),
        # a layer's input kept in 8 bits and read back for the weight gradient
        dict(name="checkpoint_load_8k", op="checkpoint", way="load", rows=8192, cols=4096, dtype="bf16"),
        # one token each of 16 sequences through 32 experts of 4096 x 1024 in 8 bits: the weights are what has to be read
        dict(name="fp8_serve_16", op="fp8", rows=16, experts=32, k=1024, n=4096, dtype="bf16"),
        # a training micro-batch through the same experts
        dict(name="fp8_experts_32k", op="fp8", rows=32768, experts=32, k=1024, n=4096, dtype="bf16"),
        # one dense fp32 layer of odd sizes
        dict(name="fp8_dense_odd", op="fp8", rows=1023, experts=1, k=1111, n=2003, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], uniform in its logarithm; every other one odd, the rest multiples of 8 where that fits."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        v |= 1
    elif v >= 16:
        v -= v % 8
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["norm", "route", "checkpoint", "fp8", "fp8"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        cols = _log_int(rng, 64, 8192)
        rows = min(_log_int(rng, 1, 32768), 2 ** 25 // cols // (2 if dtype == "f32" else 1))
        return dict(op=op, way=rng.choice(["forward", "step"]), rows=rows, cols=cols, dtype=dtype)
    if op == "route":
        experts = _log_int(rng, 4, 512)
        rows = min(_log_int(rng, 1, 32768), 2 ** 21 // experts)
        return dict(op=op, way=rng.choice(["forward", "step"]), rows=rows, experts=experts, top=rng.randint(1, min(8, experts)),
                    dtype=rng.choice(["f32", "bf16"]), dead=rng.choice([0.0, 0.06]))
    if op == "checkpoint":
        way = rng.choice(["silu", "gated", "load"])
        cols = _log_int(rng, 64, 4096)
        rows = min(_log_int(rng, 1, 32768), 2 ** 26 // cols)
        return dict(op=op, way=way, rows=rows, cols=cols, dtype=dtype)
    experts, k, n = _log_int(rng, 1, 64), _log_int(rng, 128, 4096), _log_int(rng, 128, 4096)
    # no dearer than the largest listed one, in its products and in its weights
    experts = max(1, min(experts, 2 ** 27 // (k * n)))
    return dict(op=op, rows=max(1, min(_log_int(rng, 1, 32768), 2 ** 37 // (k * n))), experts=experts, k=k, n=n, dtype=dtype)


# ------------------------------------------------------------------ the 8-bit format
def _exponent(amax):
    """Least k with amax <= 448 2^k (448 = 1.75 * 2^8): amax = m 2^e with 1/2 <= m < 1."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=-126), torch.zeros_like(e))


def _power(k):
    """2^k in fp32, exactly, for -126 <= k <= 127."""
    return ((k.to(torch.int32) + 127) << 23).view(torch.float32)


def _padded(v, rows_too=False):
    pad = [0, -v.shape[-1] % BLOCK] + ([0, -v.shape[-2] % BLOCK] if rows_too else [])
    return torch.nn.functional.pad(v, pad)


def _to_8bit(v):
    """Rows of fp32 values as (e4m3 values padded to whole blocks, exponents of the blocks)."""
    v = _padded(v)
    b = v.view(v.shape[0], -1, BLOCK)
    k = _exponent(b.abs().amax(dim=2))
    q = (b * _power(-k).unsqueeze(2)).to(torch.float8_e4m3fn)
    return q.view(v.shape), k


def _from_8bit(q, k, cols):
    b = q.float().view(q.shape[0], -1, BLOCK)
    return (b * _power(k).unsqueeze(2)).reshape(q.shape)[:, :cols]


def _weights_8bit(w):
    """A matrix as (e4m3 values, columns padded to whole blocks; codes of its 128 x 128 tiles)."""
    n = w.shape[0]
    v = _padded(w, True)
    t = v.view(v.shape[0] // BLOCK, BLOCK, -1, BLOCK)
    k = _exponent(t.abs().amax(dim=3).amax(dim=1))
    q = (t * _power(-k)[:, None, :, None]).to(torch.float8_e4m3fn)
    return q.reshape(v.shape)[:n], (k + 127).to(torch.uint8)


def _groups(rows, experts, g, dev):
    """Row offsets of `experts` groups as a router makes them: uneven, some of them empty when rows are few."""
    load = torch.softmax(0.4 * torch.randn(experts, generator=g, device=dev), 0)
    which = torch.multinomial(load, rows, replacement=True, generator=g)
    counts = torch.bincount(which, minlength=experts)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=dev)
    offsets[1:] = torch.cumsum(counts, 0).to(torch.int32)
    return offsets, int(counts.max())


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dt)

    s = dict(case)
    rows = case["rows"]
    if case["op"] == "norm":
        cols = case["cols"]
        # a residual stream: rows of different sizes, a mean, a few large columns
        x = torch.randn(rows, cols, generator=g, device=dev) * (0.5 + torch.rand(rows, 1, generator=g, device=dev)) + 0.2
        x[:, :: 97] *= 8.0
        s["x"] = x.to(dt)
        s["w"] = (1.0 + 0.2 * torch.randn(cols, generator=g, device=dev)).to(dt)
        s["b"] = normal(cols, scale=0.1)
        if case["way"] == "step":
            s["dy"] = normal(rows, cols, scale=0.01)
    elif case["op"] == "route":
        experts, top = case["experts"], case["top"]
        liked = 0.5 * torch.randn(experts, generator=g, device=dev)
        s["z"] = (torch.randn(rows, experts, generator=g, device=dev) + liked).to(dt)
        s["live"] = None
        if case["dead"] > 0:  # padded ends of sequences
            s["live"] = torch.rand(rows, generator=g, device=dev) >= case["dead"]
            s["live"][0] = True
        if case["way"] == "step":
            s["dg"] = 0.01 * torch.randn(rows, top, generator=g, device=dev)
            s["up"] = torch.full((), 0.5, device=dev)
        s["balance"], s["zloss"] = 1e-2, 1e-3
    elif case["op"] == "checkpoint":
        cols = case["cols"]
        h = torch.randn(rows, (2 if case["way"] == "gated" else 1) * cols, generator=g, device=dev)
        h[:, :: 61] *= 10.0  # outliers that a block's scale has to cover
        s["h"] = h.to(dt)
        if case["way"] != "load":
            s["da"] = normal(rows, cols, scale=0.01)
    else:
        experts, k, n = case["experts"], case["k"], case["n"]
        s["offsets"], s["most"] = _groups(rows, experts, g, dev)
        s["x"] = normal(rows, k)
        kp = k + -k % BLOCK
        s["w"] = torch.empty(experts, n, kp, dtype=torch.float8_e4m3fn, device=dev)
        s["ws"] = torch.empty(experts, -(-n // BLOCK), kp // BLOCK, dtype=torch.uint8, device=dev)
        for e in range(experts):
            s["w"][e], s["ws"][e] = _weights_8bit(torch.randn(n, k, generator=g, device=dev) * k ** -0.5)
    return s


# ------------------------------------------------------------------ plain forms
def _plain_norm(s):
    x, w, dt = s["x"].float(), s["w"].float(), s["x"].dtype
    mean = x.mean(dim=1, keepdim=True)
    r = 1.0 / ((x - mean).square().mean(dim=1, keepdim=True) + 1e-5).sqrt()
    xh = (x - mean) * r
    out = dict(y=(xh * w + s["b"].float()).to(dt))
    if s["way"] == "step":
        dy = s["dy"].float()
        g = dy * w
        out["dx"] = (r * (g - g.mean(dim=1, keepdim=True) - xh * (g * xh).mean(dim=1, keepdim=True))).to(dt)
        out["dw"] = (dy * xh).sum(dim=0)
        out["db"] = dy.sum(dim=0)
    return out


def _plain_route(s):
    rows, experts, top = s["rows"], s["experts"], s["top"]
    dev = s["z"].device
    z = s["z"].float()
    live = torch.ones(rows, dtype=torch.bool, device=dev) if s["live"] is None else s["live"]
    n = live.sum()
    one = live.float().unsqueeze(1)
    ids = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :top]
    high = z.amax(dim=1, keepdim=True)
    ez = (z - high).exp()
    total = ez.sum(dim=1, keepdim=True)
    p = ez / total
    lse = (high + total.log()).squeeze(1)
    chosen = p.gather(1, ids)
    gates = chosen / chosen.sum(dim=1, keepdim=True) * one
    ids = torch.where(live.unsqueeze(1), ids, torch.full_like(ids, -1))
    key = torch.where(ids < 0, torch.full_like(ids, experts), ids).flatten()
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=dev).index_add_(0, key, torch.ones_like(key))[:experts]
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=dev)
    offsets[1:] = torch.cumsum(counts, 0)
    order = torch.sort(key, stable=True)[1]
    routed = key[order] < experts
    tokens = torch.where(routed, order // top, torch.full_like(order, -1))
    slots = torch.empty_like(order)
    slots[order] = torch.where(routed, torch.arange(rows * top, device=dev), torch.full_like(order, -1))
    share = (p * one).sum(dim=0) / n
    balance = experts / (top * n) * (counts.float() * share).sum()
    loss = s["balance"] * balance + s["zloss"] * (lse.square() * one.squeeze(1)).sum() / n
    i32 = torch.int32
    out = dict(ids=ids.to(i32), gates=gates, counts=counts.to(i32), offsets=offsets.to(i32), slots=slots.view(rows, top).to(i32),
               tokens=tokens.to(i32), loss=loss)
    if s["way"] == "step":
        up = s["up"]
        a = up * s["balance"] * experts / (top * n.float() * n.float()) * counts.float()
        dz = p * (a - (p * a).sum(dim=1, keepdim=True)) + up * s["zloss"] * 2.0 * (lse / n).unsqueeze(1) * p
        dg = gates * (s["dg"] - (gates * s["dg"]).sum(dim=1, keepdim=True))
        dz = (dz * one).scatter_add_(1, ids.clamp(min=0), dg * one)
        out["dz"] = dz.to(s["z"].dtype)
    return out


def _plain_checkpoint(s):
    h, dt, cols = s["h"].float(), s["h"].dtype, s["cols"]
    if s["way"] == "load":
        return dict(x=_from_8bit(*_to_8bit(h), cols).to(dt))
    da = s["da"].float()
    gate = h[:, :cols]
    a = gate * (1.0 / (1.0 + (-gate).exp()))
    kept = _from_8bit(*_to_8bit(gate), cols)
    sig = 1.0 / (1.0 + (-kept).exp())
    slope = sig * (1.0 + kept * (1.0 - sig))
    if s["way"] == "silu":
        return dict(a=a.to(dt), dh=(da * slope).to(dt), again=(kept * sig).to(dt))
    up = h[:, cols:]
    kept_up = _from_8bit(*_to_8bit(up), cols)
    dh = torch.cat([da * kept_up * slope, da * kept * sig], dim=1)
    return dict(a=(a * up).to(dt), dh=dh.to(dt), again=(kept * sig * kept_up).to(dt))


def _plain_fp8(s):
    dev, rows, experts, most, k = s["x"].device, s["rows"], s["experts"], s["most"], s["k"]
    t = torch.arange(rows, device=dev)
    e = torch.searchsorted(s["offsets"][1:], t, right=True)
    at = t - s["offsets"][e]
    x = torch.zeros(experts, most, k, device=dev)
    x[e, at] = _from_8bit(*_to_8bit(s["x"].float()), k)
    w = s["w"].float()
    codes = (s["ws"].int() - 127).repeat_interleave(BLOCK, dim=1)[:, :s["n"]]
    w = (w.view(experts, s["n"], -1, BLOCK) * _power(codes).unsqueeze(3)).view(w.shape)[:, :, :k]
    return dict(y=torch.bmm(x, w.transpose(1, 2))[e, at].to(s["x"].dtype))


def run(state):
    s = state
    if not own:
        return {"norm": _plain_norm, "route": _plain_route, "checkpoint": _plain_checkpoint, "fp8": _plain_fp8}[s["op"]](s)
    from preconditioned_optimizer_matrix_amd import pmx
    if s["op"] == "norm":
        y, stats = pmx.layer_norm(s["x"], s["w"], s["b"], eps=1e-5)
        out = dict(y=y)
        if s["way"] == "step":
            out["dx"], out["dw"], out["db"] = pmx.layer_norm_grad(s["dy"], s["x"], stats, s["w"])
        return out
    if s["op"] == "route":
        kw = dict(live=s["live"], balance=s["balance"], zloss=s["zloss"])
        r = pmx.route(s["z"], s["top"], **kw)
        out = dict(ids=r.ids, gates=r.gates, counts=r.counts, offsets=r.offsets, slots=r.slots, tokens=r.tokens, loss=r.loss)
        if s["way"] == "step":
            out["dz"] = pmx.route_grad(s["z"], r, s["dg"], upstream=s["up"], **kw)
        return out
    if s["op"] == "checkpoint":
        if s["way"] == "load":
            values, scales = pmx.fp8_store(s["h"])
            return dict(x=pmx.fp8_load(values, scales, s["cols"], dtype=s["h"].dtype))
        a, values, scales = pmx.silu_checkpoint(s["h"], gated=s["way"] == "gated")
        dh, again = pmx.silu_checkpoint_grad(s["da"], values, scales, gated=s["way"] == "gated")
        return dict(a=a, dh=dh, again=again)
    values, scales = pmx.fp8_store(s["x"])
    return dict(y=pmx.fp8_product(values, scales, s["w"], s["ws"], s["offsets"], out_dtype=s["x"].dtype))


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    rows = case["rows"]
    if case["op"] == "norm":
        cols = case["cols"]
        step = case["way"] == "step"
        # the step reads x in either direction, dy once, and writes y and dx
        return dict(bytes=rows * cols * size * (5 if step else 2) + cols * (2 * size + (8 if step else 0)),
                    flops=rows * cols * (18 if step else 8))
    if case["op"] == "route":
        experts, top = case["experts"], case["top"]
        step = case["way"] == "step"
        moved = rows * (experts * size * (3 if step else 1) + top * (16 + (4 if step else 0)) + (1 if case["dead"] > 0 else 0))
        return dict(bytes=moved + experts * 8, flops=rows * experts * (12 if step else 6))
    if case["op"] == "checkpoint":
        cols = case["cols"]
        wide = cols * (2 if case["way"] == "gated" else 1)
        if case["way"] == "load":
            return dict(bytes=rows * cols * (2 * size + 2), flops=rows * cols * 4)
        # h and the activation; the 8-bit values written and read; their gradients, the activation again
        return dict(bytes=rows * (wide * (2 * size + 2) + cols * 3 * size), flops=rows * wide * 20)
    experts, k, n = case["experts"], case["k"], case["n"]
    # experts that have rows: their weights are read (uniform routing; a router's is a little more uneven)
    used = experts * (1 - (1 - 1 / experts) ** rows)
    return dict(bytes=rows * (k + n) * size + used * k * n, flops=2 * rows * k * n)


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _exact_8bit(v, blocks):
    """The values that v stands for after rounding; blocks(v) gives every entry its block's largest magnitude."""
    v = v.double()
    two = torch.tensor([2.0 ** i for i in range(-126, 128)], dtype=torch.float64, device=v.device)
    amax = blocks(v.abs())
    scale = two[torch.searchsorted(448.0 * two, amax)]
    scale = torch.where(amax > 0, scale, torch.ones_like(scale))
    u = v / scale
    # e4m3: three bits after the leading one, no step below 2^-9
    lead = torch.tensor([2.0 ** i for i in range(-6, 9)], dtype=torch.float64, device=v.device)
    step = lead[(torch.searchsorted(lead, u.abs(), right=True) - 1).clamp(min=0)] / 8.0
    return torch.round(u / step) * step * scale


def _row_blocks(a):
    return torch.cat([b.amax(dim=1, keepdim=True).expand_as(b) for b in a.split(BLOCK, dim=1)], dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    rows = case["rows"]
    f64 = torch.float64
    if case["op"] == "norm":
        x, w, b = s["x"].to(f64), s["w"].to(f64), s["b"].to(f64)
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        sd = torch.sqrt(var + 1e-5)
        xh = (x - mean) / sd
        out = dict(y=w * xh + b)
        if case["way"] == "step":
            dy = s["dy"].to(f64)
            c = case["cols"]
            g = dy * w
            out["dx"] = (c * g - g.sum(1, keepdim=True) - xh * (g * xh).sum(1, keepdim=True)) / (c * sd)
            out["dw"] = torch.einsum("tc,tc->c", dy, xh)
            out["db"] = dy.sum(0)
        return out
    if case["op"] == "route":
        experts, top = case["experts"], case["top"]
        z = s["z"].to(f64)
        dev = z.device
        live = torch.nonzero(s["live"]).squeeze(1) if s["live"] is not None else torch.arange(rows, device=dev)
        n = live.numel()
        zl = z[live]
        p = torch.softmax(zl, 1)
        lse = torch.logsumexp(zl, 1)
        # the largest left, the first of equals, `top` times
        picked, rest = [], zl.clone()
        for _ in range(top):
            high = rest.amax(1, keepdim=True)
            first = torch.where(rest == high, torch.arange(experts, device=dev), experts).amin(1)
            picked.append(first)
            rest.scatter_(1, first.unsqueeze(1), -math.inf)
        chosen = torch.stack(picked, 1)
        ids = torch.full((rows, top), -1, dtype=torch.int64, device=dev)
        ids[live] = chosen
        gates = torch.zeros(rows, top, dtype=f64, device=dev)
        gl = torch.softmax(zl.gather(1, chosen), 1)
        gates[live] = gl
        counts = torch.bincount(chosen.flatten(), minlength=experts)
        offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
        # pairs by expert, then token
        pair = chosen * rows + live.unsqueeze(1)
        ordered = pair.flatten().sort()[0]
        tokens = torch.full((rows * top,), -1, dtype=torch.int64, device=dev)
        tokens[: n * top] = ordered % rows
        slots = torch.full((rows, top), -1, dtype=torch.int64, device=dev)
        slots[live] = torch.searchsorted(ordered, pair)
        c = counts.to(f64)
        loss = s["balance"] * experts / (top * n) * (c * p.mean(0)).sum() + s["zloss"] * (lse ** 2).mean()
        i32 = torch.int32
        out = dict(ids=ids.to(i32), gates=gates, counts=counts.to(i32), offsets=offsets.to(i32), slots=slots.to(i32),
                   tokens=tokens.to(i32), loss=loss)
        if case["way"] == "step":
            z2 = zl.clone().requires_grad_()
            p2 = torch.softmax(z2, 1)
            total = 0.5 * (s["balance"] * experts / (top * n) * (c * p2.mean(0)).sum()
                           + s["zloss"] * (torch.logsumexp(z2, 1) ** 2).mean())
            total = total + (torch.softmax(z2.gather(1, chosen), 1) * s["dg"][live].to(f64)).sum()
            total.backward()
            dz = torch.zeros(rows, experts, dtype=f64, device=dev)
            dz[live] = z2.grad
            out["dz"] = dz
        return out
    if case["op"] == "checkpoint":
        cols = case["cols"]
        h = s["h"].to(f64)
        if case["way"] == "load":
            return dict(x=_exact_8bit(h, _row_blocks))
        da = s["da"].to(f64)
        g = h[:, :cols]
        a = g * torch.sigmoid(g)
        kept = _exact_8bit(g, _row_blocks)
        sig = torch.sigmoid(kept)
        slope = sig + kept * sig * (1 - sig)
        if case["way"] == "silu":
            return dict(a=a, dh=da * slope, again=kept * sig)
        up = h[:, cols:]
        kept_up = _exact_8bit(up, _row_blocks)
        return dict(a=a * up, dh=torch.cat([da * kept_up * slope, da * kept * sig], 1), again=kept * sig * kept_up)
    off = s["offsets"].tolist()
    k, n = case["k"], case["n"]
    x = _exact_8bit(s["x"], _row_blocks)
    y = torch.zeros(rows, n, dtype=f64, device=x.device)
    for e in range(case["experts"]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        tile = torch.exp2(s["ws"][e].to(f64) - 127)
        up = torch.arange(n, device=x.device) // BLOCK
        across = torch.arange(k, device=x.device) // BLOCK
        w = s["w"][e].to(f64)[:, :k] * tile[up][:, across]
        y[a:b] = x[a:b] @ w.t().contiguous()
    return dict(y=y)
