"""Workloads of the training and serving operators beside the FP8 collectives.

Three operators, in the form a program meets them around the all-to-all-v path and the gradient allreduce:

  product   rows held as E4M3 codes with one fp32 scale per 128 elements (what a low-precision all-to-all delivers) times
            weights held as E4M3 codes with one fp32 scale per 128 x 128 tile, for one weight or for one weight per group of
            rows; and its backward pass: the incoming gradient quantized along its rows and along its columns, the gradient
            of the rows and the gradient of the weights
  router    softmax over experts, the top k with their gates, the rows per expert and the load-balance loss; its gradient
  adamw     one AdamW step over many tensors, moments in fp32 or in E4M3 with one fp32 scale per 128 elements

`run` computes them in elementary torch operations, or with `own` set through the library.
"""
import numpy as np
import torch

own = False

BLOCK = 128
FP8_MAX = 448.0
ZIPF = 1.2
DT = {"f32": torch.float32, "bf16": torch.bfloat16}

# The largest listed product; a drawn one stays below it.
MOST_ROWS, MOST_K, MOST_N = 16384, 7168, 4096
MOST_STATE = 134_217_728


def listed():
    return [
        # one decoded token through one hidden x hidden projection: the weights are read once, latency counts
        {"name": "product_1_token", "op": "product", "rows": 1, "k": 8192, "n": 8192, "groups": 1, "dropped": 0, "out": "bf16"},
        # a decode batch of 32 tokens through the same projection
        {"name": "product_32_tokens", "op": "product", "rows": 32, "k": 8192, "n": 8192, "groups": 1, "dropped": 0, "out": "bf16"},
        # a short prompt through a small projection with an odd number of outputs (a head or an adapter)
        {"name": "product_odd", "op": "product", "rows": 777, "k": 1152, "n": 1000, "groups": 1, "dropped": 0, "out": "f32"},
        # the rows of a 16,384-token all-to-all, Zipf-distributed over 8 experts, through the experts' first projection
        {"name": "product_experts", "op": "product", "rows": 16384, "k": 7168, "n": 4096, "groups": 8, "dropped": 0, "out": "bf16"},
        # the backward pass of one dense layer over a 2,048-token micro-batch
        {"name": "backward_dense", "op": "backward", "rows": 2048, "k": 8192, "n": 2048, "groups": 1, "dropped": 0, "out": "bf16"},
        # the backward pass of the experts' projection over the whole all-to-all, some rows dropped by the router
        {"name": "backward_experts", "op": "backward", "rows": 16384, "k": 7168, "n": 2048, "groups": 8, "dropped": 100, "out": "bf16"},
        # routing one decoded token: latency alone
        {"name": "router_1_token", "op": "router", "rows": 1, "experts": 64, "topk": 6, "normalize": True, "logits": "f32", "masked": False, "train": False},
        # a training micro-batch over many experts, forward and backward
        {"name": "router_16384", "op": "router", "rows": 16384, "experts": 256, "topk": 8, "normalize": True, "logits": "f32", "masked": False, "train": True},
        # packed sequences with padding rows, bf16 logits, an expert count that is no power of two
        {"name": "router_odd_masked", "op": "router", "rows": 4099, "experts": 60, "topk": 4, "normalize": False, "logits": "bf16", "masked": True, "train": True},
        # an adapter's few small tensors: one short launch
        {"name": "adamw_small", "op": "adamw", "tensors": 12, "total": 60_001, "bits": 32, "grad": "f32", "copy": False},
        # a rank's share of a model after the gradient allreduce: bf16 gradients, fp32 master weights with bf16 copies, moments in 8 bits
        {"name": "adamw_8bit", "op": "adamw", "tensors": 219, "total": MOST_STATE, "bits": 8, "grad": "bf16", "copy": True},
        # the same step with fp32 moments and fp32 gradients over a smaller share
        {"name": "adamw_32bit", "op": "adamw", "tensors": 90, "total": 33_554_432, "bits": 32, "grad": "f32", "copy": False},
    ]


def _log(rng, low, high):
    return int(round(float(np.exp(rng.uniform(np.log(low), np.log(high))))))


def draw(rng):
    op = rng.choice(["product", "product", "backward", "router", "adamw"])
    if op in ("product", "backward"):
        rows = _log(rng, 1, MOST_ROWS)
        k = BLOCK * rng.choice([_log(rng, 1, MOST_K // BLOCK - 1) | 1, 2 ** rng.randint(0, 5)])
        n = _log(rng, 1, MOST_N) if op == "product" else BLOCK * _log(rng, 1, MOST_N // 2 // BLOCK)
        groups = rng.choice([1, 1, 2, 5, 8])
        dropped = rng.choice([0, rng.randint(0, rows // 2)])
        return {"op": op, "rows": rows, "k": k, "n": n, "groups": groups, "dropped": dropped if groups > 1 else 0,
                "out": rng.choice(["bf16", "f32"])}
    if op == "router":
        experts = _log(rng, 2, 256)
        return {"op": op, "rows": _log(rng, 1, 16384), "experts": experts, "topk": rng.randint(1, min(8, experts)),
                "normalize": rng.random() < 0.5, "logits": rng.choice(["f32", "bf16"]), "masked": rng.random() < 0.5,
                "train": rng.random() < 0.7}
    bits = rng.choice([8, 32])
    tensors = _log(rng, 1, 200)
    total = _log(rng, 5000, 8_000_000) + tensors
    return {"op": op, "tensors": tensors, "total": total, "bits": bits, "grad": rng.choice(["f32", "bf16"]),
            "copy": rng.random() < 0.5}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _divide(a, b):
    """The fp32 quotient nearest to a / b, by way of 64 bits: codes next to a border go by its last bit."""
    return (a.double() / b.double()).float()


def _quantize(blocks):
    """(E4M3 values, scales) of blocks along the last dimension: s = absmax / 448, code = E4M3(x / s), +0 where s is zero."""
    top = blocks.abs().amax(-1, keepdim=True)
    s = _divide(top, torch.full_like(top, FP8_MAX))
    q = torch.where(s > 0, _divide(blocks, torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(blocks))
    return q.clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn), s.squeeze(-1)


def _rows_fp8(x):
    q, s = _quantize(x.float().reshape(x.shape[0], -1, BLOCK))
    return q.reshape(x.shape).view(torch.uint8), s.contiguous()


def _tiles_fp8(w):
    """Codes and scales of a [G, n, k] weight by 128 x 128 tiles (the last row of tiles may be short)."""
    g, n, k = w.shape
    tall = -(-n // BLOCK) * BLOCK
    wide = torch.zeros(g, tall, k, device=w.device)
    wide[:, :n] = w
    t = wide.reshape(g, tall // BLOCK, BLOCK, k // BLOCK, BLOCK).transpose(2, 3).reshape(g, tall // BLOCK, k // BLOCK, -1)
    q, s = _quantize(t)
    q = q.view(torch.uint8).reshape(g, tall // BLOCK, k // BLOCK, BLOCK, BLOCK).transpose(2, 3).reshape(g, tall, k)
    return q[:, :n].contiguous(), s.contiguous()


def _counts(case, seed):
    """Rows per group, Zipf-distributed over the groups in an order of the seed; a group may be empty."""
    r = np.random.RandomState(seed % (1 << 31))
    g, rows = case["groups"], case["rows"] - case["dropped"]
    p = np.arange(1, g + 1, dtype=np.float64) ** -ZIPF
    return [int(c) for c in r.multinomial(rows, r.permutation(p / p.sum()))]


def _activations(gen, rows, cols, dev):
    """N(0, 1) with one element in a thousand a hundred times as large."""
    x = torch.randn(rows, cols, generator=gen, device=dev)
    return torch.where(torch.rand(rows, cols, generator=gen, device=dev) < 1e-3, x * 100, x)


def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    st = dict(case)
    if case["op"] in ("product", "backward"):
        rows, k, n, g = case["rows"], case["k"], case["n"], case["groups"]
        st["x"], st["xs"] = _rows_fp8(_activations(gen, rows, k, dev))
        w = torch.randn(g, n, k, generator=gen, device=dev) * k ** -0.5
        st["w"], st["ws"] = _tiles_fp8(w)
        st["splits"] = _counts(case, seed)
        st["counts"] = torch.tensor(st["splits"], dtype=torch.int32, device=dev) if g > 1 else None
        if case["op"] == "backward":
            # what a program keeps for its backward pass: the weight's codes with rows and columns exchanged
            st["wt"], st["wts"] = st["w"].transpose(1, 2).contiguous(), st["ws"].transpose(1, 2).contiguous()
            del st["w"], st["ws"]
            dy = torch.randn(rows, n, generator=gen, device=dev) * 1e-3
            st["dy"] = (dy * torch.exp(torch.randn(rows, 1, generator=gen, device=dev))).to(torch.bfloat16)
    elif case["op"] == "router":
        rows, e = case["rows"], case["experts"]
        st["dev"] = dev
        st["x"] = (torch.randn(rows, e, generator=gen, device=dev) * 1.5 +
                   torch.randn(1, e, generator=gen, device=dev) * 0.5).to(DT[case["logits"]])
        st["mask"] = None
        if case["masked"]:
            st["mask"] = (torch.rand(rows, generator=gen, device=dev) < 0.8).to(torch.uint8)
            # experts that a row may not use, and rows that may use none
            st["x"][torch.rand(rows, e, generator=gen, device=dev) < 0.1] = -float("inf")
            st["x"][torch.rand(rows, generator=gen, device=dev) < 0.02] = -float("inf")
        st["coef"] = 0.01
        st["dgates"] = torch.randn(rows, case["topk"], generator=gen, device=dev)
        st["dloss"] = torch.rand(1, generator=gen, device=dev) + 0.5
    else:
        # flat buffers, as the gradient allreduce takes them, with every tensor a view that starts at a multiple of 512
        r = np.random.RandomState(case["total"] % (1 << 31))  # the sizes belong to the model, not to the step
        share = np.exp(r.normal(0, 1.5, case["tensors"]))
        sizes = np.maximum(1, (share / share.sum() * (case["total"] - case["tensors"])).astype(np.int64))
        sizes[int(np.argmax(sizes))] += case["total"] - sizes.sum()
        starts = np.concatenate([[0], np.cumsum(-(-sizes // 512) * 512)])
        flat = int(starts[-1])
        inside = torch.zeros(flat + 1, dtype=torch.int32, device=dev)
        inside[torch.from_numpy(starts[:-1]).to(dev)] += 1
        inside[torch.from_numpy(starts[:-1] + sizes).to(dev)] -= 1
        inside = inside.cumsum(0)[:flat] > 0
        rand = lambda s: torch.where(inside, torch.randn(flat, generator=gen, device=dev) * s, 0.0)  # noqa: E731
        st["views"] = [(int(a), int(a + n)) for a, n in zip(starts, sizes)]
        st["p"], st["g"] = rand(0.02), rand(1e-3).to(DT[case["grad"]])
        st["copy_of_p"] = st["p"].to(torch.bfloat16) if case["copy"] else None
        m, v = rand(3e-4), torch.where(inside, rand(1e-3) ** 2 + 1e-8, 0.0)
        if case["bits"] == 8:
            st["m"], st["ms"] = _state_fp8(m, False)
            st["r"], st["rs"] = _state_fp8(v.sqrt(), True)
        else:
            st["m"], st["v"] = m, v
        st["scale"] = torch.rand(1, generator=gen, device=dev) * 0.5 + 0.5
        st.update(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, decay=0.1, step=100)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _decode_rows(codes, scales):
    v = codes.view(torch.float8_e4m3fn).float()
    return (v.reshape(v.shape[0], -1, BLOCK) * scales.reshape(v.shape[0], -1, 1)).reshape(v.shape)


def _decode_tiles(codes, scales):
    n, k = codes.shape[1], codes.shape[2]
    wide = scales.repeat_interleave(BLOCK, 1)[:, :n].repeat_interleave(BLOCK, 2)[:, :, :k]
    return codes.view(torch.float8_e4m3fn).float() * wide


def _grouped(x, w, splits):
    """Each group's rows times its own weight; rows past the last group give zeros."""
    used = sum(splits)
    out = [a @ b.t() for a, b in zip(x[:used].split(splits), w)]
    return torch.cat(out + [x.new_zeros(x.shape[0] - used, w.shape[1])])


def _along_rows(x):
    """x as E4M3 holds it, one scale per 128 rows of each column (the last block of a group may be short)."""
    t = x.t()
    pad = -t.shape[1] % BLOCK
    q, s = _quantize(torch.cat([t, t.new_zeros(t.shape[0], pad)], 1).reshape(t.shape[0], -1, BLOCK))
    return (q.float() * s.unsqueeze(-1)).reshape(t.shape[0], -1)


def _weight_gradient(dy, x, splits):
    used = sum(splits)
    return torch.stack([_along_rows(a) @ _along_rows(b).t() for a, b in zip(dy[:used].split(splits), x[:used].split(splits))])


def _router_plain(st):
    x, e, k = st["x"].float(), st["experts"], st["topk"]
    allowed = x > -float("inf")
    valid = allowed.any(1)
    if st["mask"] is not None:
        valid = valid & (st["mask"] != 0)
    allowed = allowed & valid.unsqueeze(1)
    x = torch.where(allowed, x, torch.full_like(x, -float("inf")))
    top = torch.where(valid.unsqueeze(1), x.amax(1, keepdim=True), torch.zeros(1, 1, device=x.device))
    ex = torch.where(allowed, (x - top).exp(), torch.zeros_like(x))
    total = ex.sum(1, keepdim=True)
    p = ex / torch.where(total > 0, total, torch.ones_like(total))
    order, which = torch.sort(x, dim=1, descending=True, stable=True)
    chosen = order[:, :k] > -float("inf")
    which = which[:, :k]
    gates = torch.where(chosen, p.gather(1, which), torch.zeros_like(order[:, :k]))
    picked = gates.sum(1, keepdim=True)
    picked = torch.where(picked > 0, picked, torch.ones_like(picked))
    if st["normalize"]:
        gates = gates / picked
    experts = torch.where(chosen, which, torch.full_like(which, -1)).to(torch.int32)
    counts = (experts.unsqueeze(2) == torch.arange(e, device=x.device, dtype=torch.int32)).sum((0, 1)).to(torch.int32)
    rows = valid.sum().clamp(min=1).float()
    load = p.sum(0) / rows
    share = counts.float() / (rows * k)
    loss = st["coef"] * e * (share * load).sum().reshape(1)
    slope = st["coef"] * e * share / rows  # of the loss against each row's probabilities
    out = {"experts": experts, "gates": gates, "counts": counts, "load": load, "slope": slope, "loss": loss}
    if st["train"]:
        dg = torch.where(chosen, st["dgates"], torch.zeros_like(st["dgates"]))
        up = st["dloss"] * slope.unsqueeze(0)
        if st["normalize"]:
            direct = gates * (dg - (gates * dg).sum(1, keepdim=True))
            dx = p * (up - (p * up).sum(1, keepdim=True))
            dx = dx.scatter_add(1, which, direct)
        else:
            up = up.expand_as(p).scatter_add(1, which, dg)
            dx = p * (up - (p * up).sum(1, keepdim=True))
        out["dlogits"] = torch.where(allowed, dx, torch.zeros_like(dx)).to(st["x"].dtype)
    return out


def _state_fp8(x, up):
    """Codes and scales of a moment in blocks of 128; `up`: what is positive keeps a code above zero."""
    blocks = x.reshape(-1, BLOCK)
    q, s = _quantize(blocks)
    codes = q.view(torch.uint8)
    if up:
        codes = torch.where((blocks > 0) & (s > 0).unsqueeze(1), codes.clamp(min=1), codes)
    return codes.reshape(-1), s


def _state_values(codes, scales):
    return (codes.view(torch.float8_e4m3fn).float().reshape(-1, BLOCK) * scales.unsqueeze(1)).reshape(-1)


def _adamw_plain(st):
    """Over the flat buffers at once: blocks of 128 never hold two tensors, and the zeros between tensors stay zeros."""
    b1, b2 = st["beta1"], st["beta2"]
    rate = float(np.float32(st["lr"] / (1 - b1 ** st["step"])))
    root = float(np.float32((1 - b2 ** st["step"]) ** -0.5))
    keep = float(np.float32(1 - st["lr"] * st["decay"]))
    g = st["g"].float() * st["scale"]
    m = _state_values(st["m"], st["ms"]) if st["bits"] == 8 else st["m"]
    v = _state_values(st["r"], st["rs"]) ** 2 if st["bits"] == 8 else st["v"]
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * (1 - b2)) * g
    r = v.sqrt()
    st["p"].copy_(st["p"] * keep - m * rate / (r * root + st["eps"]))
    if st["bits"] == 8:
        st["m"], st["ms"] = _state_fp8(m, False)
        st["r"], st["rs"] = _state_fp8(r, True)
    else:
        st["m"].copy_(m)
        st["v"].copy_(v)
    if st["copy_of_p"] is not None:
        st["copy_of_p"].copy_(st["p"])


def _adamw_outputs(st):
    out = {"p": st["p"], "m": st["m"]}
    if st["copy_of_p"] is not None:
        out["copy"] = st["copy_of_p"]
    if st["bits"] == 8:  # the values that the codes stand for, in units of their block's scale
        out.update(m=st["m"].view(torch.float8_e4m3fn), ms=st["ms"], r=st["r"].view(torch.float8_e4m3fn), rs=st["rs"])
    else:
        out["v"] = st["v"]
    return out


def run(state):
    if own:
        return _run_own(state)
    st = state
    if st["op"] == "product":
        return _grouped(_decode_rows(st["x"], st["xs"]), _decode_tiles(st["w"], st["ws"]), st["splits"]).to(DT[st["out"]])
    if st["op"] == "backward":
        dy = st["dy"].float()
        q, s = _quantize(dy.reshape(dy.shape[0], -1, BLOCK))
        along = (q.float() * s.unsqueeze(-1)).reshape(dy.shape)
        dx = _grouped(along, _decode_tiles(st["wt"], st["wts"]), st["splits"]).to(DT[st["out"]])
        return {"dx": dx, "dw": _weight_gradient(dy, _decode_rows(st["x"], st["xs"]), st["splits"])}
    if st["op"] == "router":
        return _router_plain(st)
    _adamw_plain(st)
    return _adamw_outputs(st)


# ---------------------------------------------------------------------------
# through the library
# ---------------------------------------------------------------------------

def _run_own(st):
    from fp8_precision_allreduce_amd import lpc

    if st["op"] == "product":
        dev = st["x"].device
        out = torch.empty(st["rows"], st["n"], dtype=DT[st["out"]], device=dev)
        lpc.lpc_gemm_fp8(st["x"], st["xs"], st["w"], st["ws"], out, counts=st["counts"])
        return out
    if st["op"] == "backward":
        dev = st["x"].device
        rows, k, n, g = st["rows"], st["k"], st["n"], st["groups"]
        tall = lpc.lpc_padded_rows(rows, g)
        codes, scales = torch.empty(rows, n, dtype=torch.uint8, device=dev), torch.empty(rows, n // BLOCK, device=dev)
        dyt, dyts = torch.empty(n, tall, dtype=torch.uint8, device=dev), torch.empty(tall // BLOCK, n, device=dev)
        xt, xts = torch.empty(k, tall, dtype=torch.uint8, device=dev), torch.empty(tall // BLOCK, k, device=dev)
        dx = torch.empty(rows, k, dtype=DT[st["out"]], device=dev)
        dw = torch.empty(g, n, k, device=dev)
        lpc.lpc_quantize_fp8_cols(st["dy"], dyt, dyts, codes=codes, scales=scales, counts=st["counts"])
        lpc.lpc_requantize_fp8_cols(st["x"], st["xs"], xt, xts, counts=st["counts"])
        lpc.lpc_gemm_fp8(codes, scales, st["wt"], st["wts"], dx, counts=st["counts"])
        lpc.lpc_gemm_fp8_wgrad(dyt, dyts, xt, xts, dw, rows, counts=st["counts"])
        return {"dx": dx, "dw": dw}
    if st["op"] == "router":
        x, e, k, dev = st["x"], st["experts"], st["topk"], st["x"].device
        experts = torch.empty(st["rows"], k, dtype=torch.int32, device=dev)
        gates = torch.empty(st["rows"], k, device=dev)
        counts = torch.empty(e, dtype=torch.int32, device=dev)
        load, slope, loss = torch.empty(e, device=dev), torch.empty(e, device=dev), torch.empty(1, device=dev)
        lpc.lpc_router_forward(x, experts, gates, counts, load, slope, loss, coef=st["coef"], normalize=st["normalize"], mask=st["mask"])
        out = {"experts": experts, "gates": gates, "counts": counts, "load": load, "slope": slope, "loss": loss}
        if st["train"]:
            out["dlogits"] = torch.empty_like(x)
            lpc.lpc_router_backward(x, experts, slope, st["dgates"], st["dloss"], out["dlogits"],
                                    normalize=st["normalize"], mask=st["mask"])
        return out
    if "plan" not in st:  # the program's optimizer object: one view per tensor, checked once
        views = lambda t, d=1: None if t is None else [t[a // d:-(-b // d)] for a, b in st["views"]]  # noqa: E731
        if st["bits"] == 8:
            st["plan"] = lpc.AdamW(views(st["p"]), views(st["g"]), views(st["m"]), views(st["r"]), views(st["ms"], BLOCK),
                                   views(st["rs"], BLOCK), copies=views(st["copy_of_p"]))
        else:
            st["plan"] = lpc.AdamW(views(st["p"]), views(st["g"]), views(st["m"]), views(st["v"]), copies=views(st["copy_of_p"]))
    st["plan"].step(st["step"], lr=st["lr"], beta1=st["beta1"], beta2=st["beta2"], eps=st["eps"], weight_decay=st["decay"],
                    grad_scale=st["scale"])
    return _adamw_outputs(st)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] in ("product", "backward"):
        rows, k, n, g = case["rows"] - case["dropped"], case["k"], case["n"], case["groups"]
        used = min(g, max(rows, 1))  # groups that can have rows
        size = 2 if case["out"] == "bf16" else 4
        x = rows * (k + k // BLOCK * 4)
        w = used * (n * k + -(-n // BLOCK) * (k // BLOCK) * 4)
        if case["op"] == "product":
            return {"bytes": x + w + case["rows"] * n * size, "flops": 2 * rows * k * n}
        return {"bytes": x + w + rows * n * 2 + case["rows"] * k * size + g * n * k * 4, "flops": 4 * rows * k * n}
    if case["op"] == "router":
        rows, e, k = case["rows"], case["experts"], case["topk"]
        size = 2 if case["logits"] == "bf16" else 4
        forward = rows * e * size + rows * k * 8 + e * 12
        backward = rows * e * size + rows * k * 4
        return {"bytes": forward + (backward if case["train"] else 0) + (rows if case["masked"] else 0),
                "flops": rows * e * (4 + (6 if case["train"] else 0))}
    n = case["total"]
    grad = 2 if case["grad"] == "bf16" else 4
    state = 2 * (4 if case["bits"] == 32 else 1 + 4 / BLOCK)
    return {"bytes": int(n * (8 + grad + 2 * state + (2 if case["copy"] else 0))), "flops": 16 * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _e4m3(q):
    """The nearest E4M3 value of each q, ties to even, no further than 448."""
    _, exponent = torch.frexp(q)
    powers = torch.tensor([2.0 ** e for e in range(-9, 6)], dtype=torch.float64, device=q.device)
    step = powers[(exponent.long() + 5).clamp(0, 14)]
    return (torch.round(q / step) * step).clamp(-FP8_MAX, FP8_MAX)


def _held(x):
    """What E4M3 with one scale per block of the last dimension holds of x: both quotients are rounded to fp32, as the
    format defines them (a 64-bit quotient of two fp32 numbers rounds to the fp32 one)."""
    top = x.abs().amax(-1, keepdim=True)
    s = (top / torch.full_like(top, FP8_MAX)).float().double()
    q = torch.where(s > 0, x / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(x)).float().double()
    return _e4m3(q), s


def _value64(codes):
    size = [(1 + c % 8 / 8) * 2.0 ** (c // 8 - 7) if c >= 8 else c * 2.0 ** -9 for c in range(128)]
    return torch.tensor(size + [-v for v in size], dtype=torch.float64, device=codes.device)[codes.int()]


def _product64(x, w, splits):
    out = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device=x.device)
    at = 0
    for g, c in enumerate(splits):
        out[at:at + c] = x[at:at + c] @ w[g].double().t()
        at += c
    return out


def _rows64(codes, scales):
    return _value64(codes) * scales.double().repeat_interleave(BLOCK, 1)


def _tiles64(codes, scales):
    n = codes.shape[1]
    return _value64(codes) * scales.double().repeat_interleave(BLOCK, 1)[:, :n].repeat_interleave(BLOCK, 2)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "product":
        return _product64(_rows64(st["x"], st["xs"]), _tiles64(st["w"], st["ws"]), st["splits"])
    if case["op"] == "backward":
        dy, x, out = st["dy"].double(), _rows64(st["x"], st["xs"]).float().double(), []
        v, s = _held(dy.reshape(dy.shape[0], -1, BLOCK))
        dx = _product64((v * s).reshape(dy.shape), _tiles64(st["wt"], st["wts"]), st["splits"])
        at = 0
        for c in st["splits"]:
            held = []
            for a in (dy[at:at + c], x[at:at + c]):
                wide = torch.zeros(-(-c // BLOCK) * BLOCK, a.shape[1], dtype=torch.float64, device=a.device)
                wide[:c] = a
                v, s = _held(wide.t().reshape(a.shape[1], -1, BLOCK)) if c else (wide.t(), 1.0)
                held.append((v * s).reshape(a.shape[1], -1))
            out.append(held[0] @ held[1].t())
            at += c
        return {"dx": dx, "dw": torch.stack(out)}
    if case["op"] == "router":
        return _router64(st)
    return _adamw64(st)


def _router64(st):
    x, e, k = st["x"].double(), st["experts"], st["topk"]
    valid = torch.isfinite(x).any(1)
    if st["mask"] is not None:
        valid &= st["mask"].bool()
    rows = max(1, int(valid.sum()))
    p = torch.zeros_like(x)
    p[valid] = torch.softmax(x[valid], 1)
    sets = x.masked_fill(~valid.unsqueeze(1), -float("inf"))
    picks = []
    for _ in range(k):  # the largest that is left, the lowest index first
        best = sets.amax(1, keepdim=True)
        at = (sets == best).to(torch.int8).argmax(1)
        at = torch.where(best.squeeze(1) > -float("inf"), at, torch.full_like(at, -1))
        picks.append(at)
        sets = sets.scatter(1, at.clamp(min=0).unsqueeze(1), -float("inf"))
    which = torch.stack(picks, 1)
    taken = which >= 0
    raw = p.gather(1, which.clamp(min=0)) * taken
    total = raw.sum(1, keepdim=True)
    total = torch.where(total > 0, total, torch.ones_like(total))
    gates = raw / total if st["normalize"] else raw
    counts = torch.bincount(which[taken], minlength=e)
    load, share = p.sum(0) / rows, counts.double() / (rows * k)
    out = {"experts": None, "gates": gates, "counts": None, "load": load, "slope": st["coef"] * e * share / rows,
           "loss": (st["coef"] * e * (load * share).sum()).reshape(1)}
    if st["train"]:
        slot = st["dgates"].double() * taken
        if st["normalize"]:  # gate_j = raw_j / total
            slot = (slot - (slot * gates).sum(1, keepdim=True)) / total
        dp = (st["dloss"].double() * st["coef"] * e / rows * share).expand_as(p).clone()
        dp.scatter_add_(1, which.clamp(min=0), slot * taken)
        out["dlogits"] = p * (dp - (dp * p).sum(1, keepdim=True))
    return out


def _adamw64(st):
    b1, b2, out = st["beta1"], st["beta2"], {}
    if st["bits"] == 8:
        m = (_value64(st["m"]).reshape(-1, BLOCK) * st["ms"].double().unsqueeze(1)).reshape(-1)
        v = (_value64(st["r"]).reshape(-1, BLOCK) * st["rs"].double().unsqueeze(1)).reshape(-1) ** 2
    else:
        m, v = st["m"].double(), st["v"].double()
    g = st["g"].double() * st["scale"].double()
    m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    step = (m / (1 - b1 ** st["step"])) / ((v / (1 - b2 ** st["step"])).sqrt() + st["eps"])
    out["p"] = st["p"].double() * (1 - st["lr"] * st["decay"]) - st["lr"] * step
    if st["copy_of_p"] is not None:
        out["copy"] = out["p"]
    if st["bits"] == 32:
        return {**out, "m": m, "v": v}
    for name, x in (("m", m), ("r", v.sqrt())):
        q, scale = _held(x.reshape(-1, BLOCK))
        q = q.reshape(-1)
        out[name] = torch.where((x > 0) & (q == 0), torch.full_like(q, 2.0 ** -9), q) if name == "r" else q
        out[name + "s"] = scale.reshape(-1)
    return out
