"""Cases, plain forms and 64-bit definitions of the operators around the routed experts.

Five operators, each reached through :mod:`mixture_experts_routed_gate_gb300.binding`:

``norm``       ``moe_residual_norm``: out = res + alpha * gate * (w_post * y / rms(y)), the
               residual add after a block with the block's own norm, gate and scale, and
               u = w_next * out / rms(out), the norm before the next block.
``norm_bwd``   ``moe_residual_norm_backward``: its gradients.
``few``        ``moe_forward_few``: the whole routed-expert layer for 1 to 16 tokens.
``mx4_quant``  ``moe_quantize_mx4`` / ``moe_dequantize_mx4``: rows to e2m1 elements with one
               power-of-two scale per 32, and back to the values they stand for.
``mx4_gemm``   ``moe_quantize_mx4`` of the routed rows and ``moe_grouped_gemm_mx4``, the
               grouped product of 4-bit rows with 4-bit expert weights.

``own`` false: the plain forms, elementary torch operations in 32 bits, rounded once at the end.
``own`` true: the framework's kernels.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
ALPHA = 0.5


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of a decode step: launch latency is all of it
        dict(name="norm_1x2048_f16", op="norm", T=1, H=2048, dtype="f16", post=True, next=True, gate="channel"),
        # a prefill batch: four passes over a tensor of 59 MB
        dict(name="norm_4096x7168_bf16", op="norm", T=4096, H=7168, dtype="bf16", post=True, next=True, gate="channel"),
        # a ragged training batch with an odd width and a gate per token (no 16-byte rows)
        dict(name="norm_bwd_333x2047_f32", op="norm_bwd", T=333, H=2047, dtype="f32", post=True, next=True, gate="token"),
        # the backward pass at the prefill size, weight gradients summed over 4096 rows
        dict(name="norm_bwd_4096x7168_bf16", op="norm_bwd", T=4096, H=7168, dtype="bf16", post=True, next=True, gate="channel"),
        # the smallest decode step: six experts' weights, about 57 MB
        dict(name="few_1x2048_f16", op="few", T=1, d_h=2048, d_e=768, E=64, k=6, dtype="f16", bias=False),
        # eight sequences decoding together: experts shared by some of the tokens
        dict(name="few_8x2048_f16", op="few", T=8, d_h=2048, d_e=768, E=64, k=6, dtype="f16", bias=True),
        # two sequences through the large layer: 16 of 256 experts, 1.4 GB of weights
        dict(name="few_2x7168_bf16", op="few", T=2, d_h=7168, d_e=2048, E=256, k=8, dtype="bf16", bias=True),
        # a decode batch's activations
        dict(name="mx4_quant_64x2048_f16", op="mx4_quant", R=64, K=2048, dtype="f16"),
        # a prefill batch's activations (or one slab of a layer's weights)
        dict(name="mx4_quant_4096x7168_bf16", op="mx4_quant", R=4096, K=7168, dtype="bf16"),
        # a decode batch through one expert projection: small ragged groups, weights are the cost
        dict(name="mx4_gemm_64x2048x768_f16", op="mx4_gemm", T=64, k=6, E=64, K=2048, N=768, dtype="f16", out="f16"),
        # odd sizes: K one scale block past a 1024 multiple, N odd, some groups over 128 rows
        dict(name="mx4_gemm_301x1056x333_f32", op="mx4_gemm", T=301, k=3, E=5, K=1056, N=333, dtype="f32", out="f32"),
        # the large layer's up projection over a prefill batch: 32768 routed rows, 1.9 GB of 4-bit weights
        dict(name="mx4_gemm_4096x7168x2048_bf16", op="mx4_gemm", T=4096, k=8, E=256, K=7168, N=2048, dtype="bf16", out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "few", "mx4_quant", "mx4_gemm"])
    dtype = rng.choice(["f16", "bf16", "f32"])
    if op in ("norm", "norm_bwd"):
        post, nxt = rng.choice([(True, True), (True, True), (True, False), (False, True)])
        return dict(op=op, T=_log_int(rng, 1, 4096), H=_log_int(rng, 33, 7168), dtype=dtype if dtype != "f32" else rng.choice(["f32", "bf16"]),
                    post=post, next=nxt, gate=rng.choice(["none", "channel", "token", "full"]))
    if op == "few":
        while True:
            c = dict(op=op, T=rng.randint(1, 16), d_h=256 * _log_int(rng, 1, 28), d_e=64 * _log_int(rng, 1, 32), E=_log_int(rng, 2, 256),
                     k=rng.randint(1, 8), dtype=rng.choice(["f16", "bf16"]), bias=rng.random() < 0.5)
            if c["k"] <= c["E"] and c["T"] * c["k"] * c["d_h"] * c["d_e"] <= 16 * 7168 * 2048 and c["E"] * c["d_h"] * c["d_e"] <= 2 << 30:
                return c
    if op == "mx4_quant":
        return dict(op=op, R=_log_int(rng, 1, 4096), K=32 * _log_int(rng, 1, 224), dtype=dtype)
    while True:
        c = dict(op=op, T=_log_int(rng, 1, 4096), k=rng.randint(1, 8), E=_log_int(rng, 1, 256), K=32 * _log_int(rng, 1, 224), N=_log_int(rng, 8, 2048),
                 dtype=dtype, out=dtype)
        if c["k"] <= c["E"] and c["T"] * c["k"] <= 8 * c["E"] + 8192:
            return c


def work(case):
    """Each input read once, each output written once."""
    c = case
    if c["op"] in ("norm", "norm_bwd"):
        T, H, es = c["T"], c["H"], 4 if c["dtype"] == "f32" else 2
        gate = dict(none=0, channel=H, token=T, full=T * H)[c["gate"]]
        if c["op"] == "norm":  # res, y -> out, u
            wide = 3 + c["next"]
            return dict(bytes=es * (wide * T * H + gate + H * (c["post"] + c["next"])) + 4 * T * (c["post"] + c["next"]), flops=T * H * (6 * c["post"] + 4 * c["next"] + 2))
        wide = 2 + 1 + 2 * c["next"] + 1  # y, d_out, (out, d_u) -> d_res, d_y
        narrow = 4 * (H * (c["post"] + c["next"]) + (gate if c["gate"] in ("channel", "token") else 0))
        return dict(bytes=es * (wide * T * H + gate * (2 if c["gate"] == "full" else 1) + H * (c["post"] + c["next"])) + narrow + 4 * T * (c["post"] + c["next"]),
                    flops=T * H * (10 * c["post"] + 8 * c["next"] + 3))
    if c["op"] == "few":
        touched = c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])  # experts that get a token, on average
        weights = touched * 3 * c["d_e"] * c["d_h"] + c["E"] * c["d_h"]
        return dict(bytes=2 * (weights + 2 * c["T"] * c["d_h"]), flops=2 * c["T"] * (3 * c["k"] * c["d_e"] * c["d_h"] + c["E"] * c["d_h"]))
    es = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "mx4_quant":  # x -> elements and scales -> values in bf16
        n = c["R"] * c["K"]
        return dict(bytes=n * es + 2 * (n // 2 + n // 32) + 2 * n, flops=3 * n)
    rows, E, K, N = c["T"] * c["k"], c["E"], c["K"], c["N"]
    touched = E * (1 - (1 - c["k"] / E) ** c["T"])
    four = lambda r: r * (K // 2 + K // 32)  # noqa: E731
    return dict(bytes=c["T"] * K * es + four(touched * N) + rows * N * (4 if c["out"] == "f32" else 2), flops=2 * rows * K * N)


# ----------------------------------------------------------------------------- inputs

def _normal(shape, std, dtype, gen):
    t = torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=gen)
    return t if std == 1.0 else t.mul_(std)


def _tables(idx, E):
    """The dispatch tables of routing idx [T, k] (128-row blocks, one block at least for each expert)."""
    T, k = idx.shape
    flat = idx.reshape(-1)
    sizes = torch.bincount(flat, minlength=E)
    ends = sizes.cumsum(0)
    padded_sizes = (sizes + 1 + 127) // 128 * 128
    padded = padded_sizes.cumsum(0) - padded_sizes
    blocks = -(-T * k // 128) + E
    starts = torch.arange(blocks, device=idx.device) * 128
    order = torch.argsort(flat, stable=True)
    i32 = lambda t: t.to(torch.int32).contiguous()  # noqa: E731
    return dict(group_sizes=i32(sizes), group_offsets=i32(ends - sizes), group_padded_offsets=i32(padded),
                group_idx_for_bx=i32(torch.searchsorted(padded, starts, right=True) - 1)), i32(order // k)


def prepare(case, seed):
    c, dt = case, DTYPES[case["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    if c["op"] in ("norm", "norm_bwd"):
        T, H = c["T"], c["H"]
        s = dict(case=c)
        s["y"] = _normal((T, H), 2.0, dt, gen)
        s["res"] = _normal((T, H), 1.0, dt, gen)
        s["w_post"] = _normal((H,), 0.2, dt, gen).add_(1.0) if c["post"] else None
        s["w_next"] = _normal((H,), 0.2, dt, gen).add_(1.0) if c["next"] else None
        shape = dict(none=None, channel=(H,), token=(T,), full=(T, H))[c["gate"]]
        s["gate"] = None if shape is None else _normal(shape, 0.5, dt, gen).add_(0.5)
        if c["op"] == "norm_bwd":  # what the forward pass kept
            f = _plain_norm(s["y"], s["res"], s["w_post"], _gate_of(s), s["w_next"], dt)
            s.update(out=f["out"], rstd_post=f.get("rstd_post"), rstd_next=f.get("rstd_next"))
            s["d_out"] = _normal((T, H), 1.0, dt, gen)
            s["d_u"] = _normal((T, H), 1.0, dt, gen) if c["next"] else None
        return s
    if c["op"] == "few":
        T, d_h, d_e, E = c["T"], c["d_h"], c["d_e"], c["E"]
        return dict(case=c, x=_normal((T, d_h), 1.0, dt, gen), w_g=_normal((E, d_h), d_h ** -0.5, dt, gen),
                    bias=_normal((E,), 0.3, torch.float32, gen) if c["bias"] else None,
                    w_gate=_normal((E, d_e, d_h), d_h ** -0.5, dt, gen), w_up=_normal((E, d_e, d_h), d_h ** -0.5, dt, gen),
                    w_down=_normal((E, d_h, d_e), d_e ** -0.5, dt, gen))
    if c["op"] == "mx4_quant":
        x = _normal((c["R"], c["K"]), 1.0, dt, gen)
        x[:, ::97] *= 8.0  # activations have a few large channels
        if c["K"] > 32:
            x[:, 32:64] = 0.0  # and blocks of zeros
        return dict(case=c, x=x)
    T, k, E, K, N = c["T"], c["k"], c["E"], c["K"], c["N"]
    x = _normal((T, K), 1.0, dt, gen)
    liked = _normal((E,), 0.5, torch.float32, gen)
    idx = (_normal((T, E), 1.0, torch.float32, gen) + liked).topk(k, dim=1).indices
    tables, token = _tables(idx, E)
    q = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    sf = torch.empty((E, N, K // 32), dtype=torch.uint8, device="cuda")
    for e in range(E):  # 4-bit weights as they are loaded, one expert at a time
        code, scale = _mx4_codes(_normal((N, K), K ** -0.5, torch.float32, gen))
        q[e] = code[:, 0::2] | (code[:, 1::2] << 4)
        sf[e] = scale
    return dict(case=c, x=x, tables=tables, token=token, q=q, sf=sf)


# ----------------------------------------------------------------------------- plain forms

def _plain_norm(y, res, w_post, gate, w_next, dt):
    got = {}
    z = y.float()
    if w_post is not None:
        got["rstd_post"] = torch.rsqrt((z * z).mean(1) + EPS)
        z = z * got["rstd_post"][:, None] * w_post.float()
    if gate is not None:
        z = z * gate.float()
    o = res.float() + ALPHA * z
    got["out"] = o.to(dt)
    if w_next is not None:
        got["rstd_next"] = torch.rsqrt((o * o).mean(1) + EPS)
        got["u"] = (o * got["rstd_next"][:, None] * w_next.float()).to(dt)
    return got


def _plain_norm_bwd(s, dt):
    y, o, d = s["y"].float(), s["out"].float(), s["d_out"].float()
    H, got = y.shape[1], {}
    if s["w_next"] is not None:
        r, du = s["rstd_next"][:, None], s["d_u"].float()
        v = du * s["w_next"].float()
        d = d + r * v - o * (r * r * r / H) * (v * o).sum(1, keepdim=True)
        got["d_w_next"] = (du * o * r).sum(0)
    got["d_res"] = d.to(dt)
    g = 1.0 if s["gate"] is None else _gate_of(s).float()
    z = y
    if s["w_post"] is not None:
        z = y * s["rstd_post"][:, None] * s["w_post"].float()
    if s["gate"] is not None:
        dg = ALPHA * d * z
        kind = s["case"]["gate"]
        got["d_gate"] = dg.sum(0) if kind == "channel" else dg.sum(1, keepdim=True) if kind == "token" else dg.to(dt)
    dz = ALPHA * g * d
    if s["w_post"] is not None:
        r = s["rstd_post"][:, None]
        v = dz * s["w_post"].float()
        got["d_w_post"] = (dz * y * r).sum(0)
        dz = r * v - y * (r * r * r / H) * (v * y).sum(1, keepdim=True)
    got["d_y"] = dz.to(dt)
    return got


def _gate_of(s):
    """gate [H], [T, 1] or [T, H]: as the entry points take it."""
    return s["gate"][:, None] if s["case"]["gate"] == "token" else s["gate"]


def _plain_few(s, dt):
    k, x = s["case"]["k"], s["x"].float()
    T, d_h = x.shape
    logits = x @ s["w_g"].float().t()
    if s["bias"] is not None:
        logits = logits + s["bias"]
    idx = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.softmax(logits, 1).gather(1, idx)
    flat = idx.reshape(-1)
    rows = x.repeat_interleave(k, 0)[:, :, None]
    g = torch.bmm(s["w_gate"][flat].float(), rows)
    h = g * torch.sigmoid(g) * torch.bmm(s["w_up"][flat].float(), rows)
    y = torch.bmm(s["w_down"][flat].float(), h).view(T, k, d_h)
    return (w[:, :, None] * y).sum(1).to(dt)


def _pow2(n):
    """2^n in fp32 from its bits, exact for -127 <= n <= 127."""
    return torch.where(n > -127, (n + 127) << 23, torch.full_like(n, 1 << 22)).view(torch.float32)


def _mx4_codes(x):
    """x [R, K] -> the 4-bit codes [R, K] (sign, then 0 .5 1 1.5 2 3 4 6) and the scale bytes [R, K / 32] (2^(byte - 127)):
    the scale is 2^(floor(log2(largest magnitude)) - 2), elements are rounded to nearest, ties to the even code, at most 6."""
    R, K = x.shape
    b = x.float().view(R, K // 32, 32)
    top = b.abs().amax(2)
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(-127, 127)
    v = b * _pow2(-e)[:, :, None]
    a = v.abs()
    code = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    return (code | ((v < 0).to(torch.uint8) << 3)).view(R, K), (e + 127).to(torch.uint8)


def _mx4_values(code, scale):
    """The numbers (fp32, exact) that codes [..., K] with scale bytes [..., K / 32] stand for."""
    m = (code & 7).to(torch.float32)
    mag = torch.where(m < 4, m * 0.5, torch.where(m < 6, m - 2.0, 2.0 * m - 8.0))
    mag = torch.where(code > 7, -mag, mag)
    s = _pow2(scale.to(torch.int32) - 127)
    return (mag.view(*scale.shape, 32) * s[..., None]).view(code.shape)


def _plain_mx4_gemm(s):
    c, t = s["case"], s["tables"]
    code, scale = _mx4_codes(s["x"])
    a = _mx4_values(code, scale)[s["token"].long()]
    rows, K = a.shape
    sizes = t["group_sizes"].long()
    expert = torch.repeat_interleave(torch.arange(c["E"], device=a.device), sizes)
    place = torch.arange(rows, device=a.device) - t["group_offsets"].long()[expert]
    padded = torch.zeros((c["E"], int(sizes.max()), K), device=a.device)
    padded[expert, place] = a
    both = torch.stack((s["q"] & 15, s["q"] >> 4), dim=3).view(c["E"], c["N"], K)
    full = torch.bmm(padded, _mx4_values(both, s["sf"]).transpose(1, 2))
    return full[expert, place].to(DTYPES[c["out"]])


# ----------------------------------------------------------------------------- one pass

def run(state):
    s, c = state, state["case"]
    dt = DTYPES[c["dtype"]]
    if own:
        from mixture_experts_routed_gate_gb300 import binding
        if c["op"] == "norm":
            return binding.moe_residual_norm(s["y"], s["res"], s["w_post"], _gate_of(s), ALPHA, s["w_next"], EPS)
        if c["op"] == "norm_bwd":
            return binding.moe_residual_norm_backward(s["d_out"], s["d_u"], s["y"], s["out"], s["w_post"], _gate_of(s),
                                                      ALPHA, s["w_next"], s["rstd_post"], s["rstd_next"])
        if c["op"] == "few":
            return binding.moe_forward_few(s["x"], s["w_g"], s["bias"], s["w_gate"], s["w_up"], s["w_down"], c["k"])
        if c["op"] == "mx4_quant":
            return binding.moe_dequantize_mx4(*binding.moe_quantize_mx4(s["x"]), torch.bfloat16)
        q, sf = binding.moe_quantize_mx4(s["x"], s["token"])
        return binding.moe_grouped_gemm_mx4(q, sf, s["q"], s["sf"], s["tables"], DTYPES[c["out"]])
    if c["op"] == "norm":
        return _plain_norm(s["y"], s["res"], s["w_post"], _gate_of(s), s["w_next"], dt)
    if c["op"] == "norm_bwd":
        return _plain_norm_bwd(s, dt)
    if c["op"] == "few":
        return _plain_few(s, dt)
    if c["op"] == "mx4_quant":
        return _mx4_values(*_mx4_codes(s["x"])).to(torch.bfloat16)
    return _plain_mx4_gemm(s)


# ----------------------------------------------------------------------------- 64 bits

def _exact_mx4(x):
    """The values of the rows' 4-bit form, from the list of what 4 bits can hold."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    middle = (grid[1:] + grid[:-1]) / 2
    b = x.double().view(x.shape[0], -1, 32)
    top = b.abs().amax(2, keepdim=True)
    power = (top.view(torch.int64) >> 52) - 1023 - 2  # floor(log2) is in a double's exponent field
    unit = ((power.clamp(-127, 127) + 1023) << 52).view(torch.float64)
    a = (b.abs() / unit).contiguous()
    low, high = torch.searchsorted(middle, a), torch.searchsorted(middle, a, right=True)  # they differ at a tie
    at = torch.where(low % 2 == 0, low, high)
    return (torch.sign(b) * grid[at] * unit).view(x.shape)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "norm":
        y, res = s["y"].double(), s["res"].double()
        got, b = {}, y
        if s["w_post"] is not None:
            rms = (y.square().mean(1) + EPS).sqrt()
            got["rstd_post"] = 1 / rms
            b = s["w_post"].double() * y / rms[:, None]
        out = res + ALPHA * (b if s["gate"] is None else _gate_of(s).double() * b)
        got["out"] = out
        if s["w_next"] is not None:
            rms = (out.square().mean(1) + EPS).sqrt()
            got["rstd_next"] = 1 / rms
            got["u"] = s["w_next"].double() * out / rms[:, None]
        return got
    if c["op"] == "norm_bwd":
        # each norm's Jacobian-vector product from its normalised rows, which the saved statistics give
        y, out, d = s["y"].double(), s["out"].double(), s["d_out"].double()
        got = {}
        if s["w_next"] is not None:
            n = out * s["rstd_next"].double()[:, None]
            up = s["d_u"].double() * s["w_next"].double()
            got["d_w_next"] = torch.einsum("th,th->h", s["d_u"].double(), n)
            d = d + s["rstd_next"].double()[:, None] * (up - n * (up * n).mean(1, keepdim=True))
        got["d_res"] = d
        n = y if s["w_post"] is None else y * s["rstd_post"].double()[:, None]
        wp = torch.ones_like(y[0]) if s["w_post"] is None else s["w_post"].double()
        gate = torch.ones_like(y[:1]) if s["gate"] is None else _gate_of(s).double()
        if s["gate"] is not None:
            spec = dict(channel="th,th->h", token="th,th->t", full="th,th->th")[c["gate"]]
            got["d_gate"] = ALPHA * torch.einsum(spec, d, n * wp)
        db = ALPHA * d * gate
        if s["w_post"] is None:
            got["d_y"] = db
        else:
            got["d_w_post"] = torch.einsum("th,th->h", db, n)
            up = db * wp
            got["d_y"] = s["rstd_post"].double()[:, None] * (up - n * (up * n).mean(1, keepdim=True))
        return got
    if c["op"] == "few":
        x = s["x"].double()
        score = x @ s["w_g"].double().t() + (0 if s["bias"] is None else s["bias"].double())
        weight = torch.exp(score - score.logsumexp(1, keepdim=True))
        best, out = torch.sort(-score, dim=1, stable=True).indices[:, : c["k"]].tolist(), torch.zeros_like(x)
        for t, experts in enumerate(best):
            for e in experts:
                g = s["w_gate"][e].double() @ x[t]
                h = g / (1 + torch.exp(-g)) * (s["w_up"][e].double() @ x[t])
                out[t] += weight[t, e] * (s["w_down"][e].double() @ h)
        return out
    if c["op"] == "mx4_quant":
        return _exact_mx4(s["x"])
    a = _exact_mx4(s["x"])[s["token"].long()]
    held = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    first, parts = 0, []
    for e, n in enumerate(s["tables"]["group_sizes"].tolist()):
        if n:
            pair = torch.stack((held[(s["q"][e] % 16).long()], held[(s["q"][e] // 16).long()]), 2).view(c["N"], -1, 32)
            w = pair * ((s["sf"][e].long() + 896) << 52).view(torch.float64)[:, :, None]
            parts.append(a[first:first + n] @ w.view(c["N"], -1).t())
        first += n
    return torch.cat(parts)
