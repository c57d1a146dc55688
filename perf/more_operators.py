"""Workloads of the operators that follow an expert layer's weights: trained in bf16, updated as matrices, served in 4 bits.

  bf16    the matrix product of bf16 rows with one weight or with one weight per group of rows (ragged, as an all-to-all
          delivers them), and its backward pass: the gradient of the rows and the gradient of the weights
  muon    one step of the optimizer over many matrices: momentum, the update orthogonalised by five Newton-Schulz
          iterations, weight decay
  mxfp4   microscaled 4-bit floating point (E2M1 elements, one power-of-two scale per 32): quantization and its inverse, and
          the product of rows that are quantized on arrival with weights that are held in it

`run` computes them in elementary torch operations, or with `own` set through the library.
"""
import numpy as np
import torch

own = False

ZIPF = 1.2
MX = 32            # elements of a microscaled block
MX_MAX = 6.0       # the largest E2M1 value
NS_A, NS_B, NS_C = 3.4445, -4.7750, 2.0315
NS_ITERATIONS = 5
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}

# The largest listed sizes; a drawn case stays below them.
MOST_ROWS, MOST_K, MOST_N = 16384, 7168, 4096
MOST_SIDE = 2048


def listed():
    return [
        # 32 decoded tokens, routed over 8 experts: every expert's weight is read once, few rows each
        {"name": "bf16_decode", "op": "bf16", "rows": 32, "k": 7168, "n": 2048, "groups": 8, "dropped": 0, "out": "bf16", "train": False},
        # the rows of a 16,384-token all-to-all, Zipf-distributed over 8 experts, through the experts' first projection
        {"name": "bf16_experts", "op": "bf16", "rows": 16384, "k": 7168, "n": 4096, "groups": 8, "dropped": 0, "out": "bf16", "train": False},
        # a short prompt through a small layer, forward and backward, no size a power of two
        {"name": "bf16_odd_step", "op": "bf16", "rows": 777, "k": 1160, "n": 1000, "groups": 3, "dropped": 20, "out": "f32", "train": True},
        # one training step of the experts' projection over the whole all-to-all, some rows dropped by the router
        {"name": "bf16_experts_step", "op": "bf16", "rows": 16384, "k": 7168, "n": 2048, "groups": 8, "dropped": 100, "out": "bf16", "train": True},
        # an adapter's factors, 16 wide: launches count
        {"name": "muon_adapter", "op": "muon", "count": 4, "rows": 16, "cols": 1152, "mixed": False, "grad": "f32", "copy": False},
        # a layer's matrices, all of other odd sizes, both tall and wide
        {"name": "muon_mixed", "op": "muon", "count": 9, "rows": 1000, "cols": 1500, "mixed": True, "grad": "bf16", "copy": True},
        # one square projection
        {"name": "muon_square", "op": "muon", "count": 1, "rows": 2048, "cols": 2048, "mixed": False, "grad": "f32", "copy": True},
        # a rank's experts: eight matrices of one shape, bf16 gradients, bf16 copies of the weights
        {"name": "muon_experts", "op": "muon", "count": 8, "rows": 2048, "cols": 7168, "mixed": False, "grad": "bf16", "copy": True},
        # one decoded token through one hidden x hidden projection held in 4 bits
        {"name": "mxfp4_1_token", "op": "mxfp4", "rows": 1, "k": 8192, "n": 8192, "groups": 1, "dropped": 0, "in": "bf16", "out": "bf16"},
        # a short prompt through a projection with an odd number of outputs
        {"name": "mxfp4_odd", "op": "mxfp4", "rows": 777, "k": 1152, "n": 1001, "groups": 1, "dropped": 0, "in": "f32", "out": "f32"},
        # a 16,384-row prompt batch through the experts' first projection in 4 bits
        {"name": "mxfp4_experts", "op": "mxfp4", "rows": 16384, "k": 7168, "n": 4096, "groups": 8, "dropped": 0, "in": "bf16", "out": "bf16"},
        # an expert's new weights brought to 4 bits, and the weights that these stand for
        {"name": "mxfp4_weights", "op": "codec", "rows": 8192, "k": 7168, "in": "f32", "out": "bf16"},
    ]


def _log(rng, low, high):
    return int(round(float(np.exp(rng.uniform(np.log(low), np.log(high))))))


def draw(rng):
    op = rng.choice(["bf16", "bf16", "muon", "muon", "mxfp4", "mxfp4", "codec"])
    if op in ("bf16", "mxfp4"):
        rows, groups = _log(rng, 1, MOST_ROWS), rng.choice([1, 1, 2, 5, 8])
        train = op == "bf16" and rng.random() < 0.5
        step = 8 if op == "bf16" else 128
        k = step * _log(rng, 1, MOST_K // step)
        n = 8 * _log(rng, 1, MOST_N // 16) if train else _log(rng, 1, MOST_N)
        dropped = rng.choice([0, rng.randint(0, rows // 2)]) if groups > 1 else 0
        case = {"op": op, "rows": rows, "k": k, "n": n, "groups": groups, "dropped": dropped, "out": rng.choice(["bf16", "f32"])}
        return {**case, "train": train} if op == "bf16" else {**case, "in": rng.choice(["bf16", "f32"])}
    if op == "codec":
        return {"op": op, "rows": _log(rng, 1, 8192), "k": MX * _log(rng, 1, MOST_K // MX), "in": rng.choice(["bf16", "f32"]),
                "out": rng.choice(["bf16", "f32"])}
    rows, cols = _log(rng, 1, MOST_SIDE), _log(rng, 1, MOST_SIDE)
    return {"op": op, "count": _log(rng, 1, 12), "rows": rows, "cols": cols, "mixed": rng.random() < 0.5,
            "grad": rng.choice(["f32", "bf16"]), "copy": rng.random() < 0.5}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

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


def _shapes(case):
    """(rows, cols) of every matrix of an optimizer case; they belong to the model, not to the step."""
    if not case["mixed"]:
        return [(case["rows"], case["cols"])] * case["count"]
    r = np.random.RandomState(case["rows"] * 4099 + case["cols"] + case["count"])
    share = r.uniform(0.2, 1.0, (case["count"], 2))
    turned = r.rand(case["count"]) < 0.5
    sizes = np.maximum(1, (share * [case["rows"], case["cols"]]).astype(np.int64))
    return [(int(b), int(a)) if t else (int(a), int(b)) for (a, b), t in zip(sizes, turned)]


def _gradient(gen, b, rows, cols, dev):
    """What a layer's gradient is like: a few strong directions, and noise over all."""
    rank = min(8, rows, cols)
    strong = torch.randn(b, rows, rank, generator=gen, device=dev) @ torch.randn(b, rank, cols, generator=gen, device=dev)
    return (strong * 0.5 + torch.randn(b, rows, cols, generator=gen, device=dev)) * 1e-3


def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    st = dict(case)
    if case["op"] == "muon":
        shapes = _shapes(case)
        # equal matrices lie in one tensor, as a layer of experts holds them
        st["sizes"] = [(1, *s) for s in shapes] if case["mixed"] else [(case["count"], *shapes[0])]
        st["p"] = [torch.randn(b, r, c, generator=gen, device=dev) * 0.02 for b, r, c in st["sizes"]]
        st["g"] = [_gradient(gen, b, r, c, dev).to(DT[case["grad"]]) for b, r, c in st["sizes"]]
        st["m"] = [_gradient(gen, b, r, c, dev) * 0.3 for b, r, c in st["sizes"]]
        st["copies"] = [p.to(torch.bfloat16) for p in st["p"]] if case["copy"] else None
        # the step's rms as a share of the learning rate is the same for every shape
        st["scale"] = [0.2 * max(r, c) ** 0.5 for _, r, c in st["sizes"]]
        st.update(lr=3e-4, beta=0.95, decay=0.1)
        return st
    rows, k = case["rows"], case["k"]
    if case["op"] == "codec":
        w = torch.randn(rows, k, generator=gen, device=dev) * k ** -0.5
        st["x"] = (w * torch.exp(torch.randn(rows, 1, generator=gen, device=dev))).to(DT[case["in"]])
        return st
    n, g = case["n"], case["groups"]
    st["splits"] = _counts(case, seed)
    st["counts"] = torch.tensor(st["splits"], dtype=torch.int32, device=dev) if g > 1 else None
    x, w = _activations(gen, rows, k, dev), torch.randn(g, n, k, generator=gen, device=dev) * k ** -0.5
    if case["op"] == "bf16":
        st["x"], st["w"] = x.to(torch.bfloat16), w.to(torch.bfloat16)
        if case["train"]:
            dy = torch.randn(rows, n, generator=gen, device=dev) * 1e-3
            st["dy"] = (dy * torch.exp(torch.randn(rows, 1, generator=gen, device=dev))).to(torch.bfloat16)
    else:
        st["x"] = x.to(DT[case["in"]])
        st["w"], st["ws"] = _pack(*_mx(w.reshape(g * n, k)))  # quantized once, when the model is loaded
        st["w"], st["ws"] = st["w"].reshape(g, n, k // 2), st["ws"].reshape(g, n, k // MX)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _mx(x):
    """E2M1 values [rows, k] of x in units of its blocks' scales, and the scales' exponent bytes [rows, k/32]: the scale is the
    power of two two binades below the block's largest magnitude (which E2M1 holds up to 6), no less than 2^-127; values are
    rounded to nearest, ties to even, and no further than 6."""
    b = x.float().reshape(x.shape[0], -1, MX)
    top = b.abs().amax(-1, keepdim=True)
    byte = torch.where(top > 0, torch.frexp(top)[1] - 3 + 127, torch.zeros_like(top, dtype=torch.int32)).clamp(min=0)
    q = (b * _power(254 - byte)).abs()  # over the scale: exact
    step = torch.where(q < 2, 0.5, torch.where(q < 4, 1.0, 2.0))
    v = torch.copysign((torch.round(q / step) * step).clamp(max=MX_MAX), b)
    return v.reshape(x.shape), byte.squeeze(-1).to(torch.uint8)


def _pack(v, byte):
    """The codes of E2M1 values, two to a byte, the first one in the low bits."""
    a = v.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code + torch.signbit(v).to(torch.uint8) * 8
    return code[:, 0::2] + code[:, 1::2] * 16, byte


def _unpack(codes):
    """The E2M1 values that bytes of two codes stand for."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    both = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    return table[both.int()]


def _power(byte):
    """2^(byte - 127) as fp32, exactly, for bytes 0 to 254."""
    return torch.where(byte > 0, byte.int() << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _scaled(v, byte):
    return (v.reshape(*byte.shape, MX) * _power(byte).unsqueeze(-1)).reshape(v.shape)


def _grouped(x, w, splits):
    """Each group's rows times its own weight; rows past the last group give zeros."""
    used = sum(splits)
    out = [a @ b.t() for a, b in zip(x[:used].split(splits), w)]
    return torch.cat(out + [x.new_zeros(x.shape[0] - used, w.shape[1])])


def _orthogonal(u):
    """Newton-Schulz on matrices [b, m, n], m <= n, from the update over its norm (zero for an update of zeros)."""
    norm = u.double().square().sum((1, 2), keepdim=True).sqrt()
    x = torch.where(norm > 0, u.double() / torch.where(norm > 0, norm, torch.ones_like(norm)), torch.zeros_like(norm)).float()
    for _ in range(NS_ITERATIONS):
        a = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = NS_A * x + torch.bmm(NS_B * a + NS_C * torch.bmm(a, a), x)
    return x


def _muon_plain(st):
    beta, lr = st["beta"], st["lr"]
    for i, (p, g, m) in enumerate(zip(st["p"], st["g"], st["m"])):
        m.copy_(m * beta + g.float() * (1 - beta))
        u = g.float() * (1 - beta) + m * beta
        tall = u.shape[1] > u.shape[2]
        o = _orthogonal(u.transpose(1, 2).contiguous() if tall else u)
        p.copy_(p * (1 - lr * st["decay"]) - (o.transpose(1, 2) if tall else o) * (lr * st["scale"][i]))
        if st["copies"] is not None:
            st["copies"][i].copy_(p)


def _muon_outputs(st):
    out = {"p": st["p"], "m": st["m"]}
    if st["copies"] is not None:
        out["copies"] = st["copies"]
    return out


def run(state):
    if own:
        return _run_own(state)
    st = state
    if st["op"] == "muon":
        _muon_plain(st)
        return _muon_outputs(st)
    if st["op"] == "codec":
        v, byte = _mx(st["x"])
        return {"values": _scaled(v, byte).to(DT[st["out"]]), "scales": byte}
    if st["op"] == "mxfp4":
        return _grouped(_scaled(*_mx(st["x"])), _scaled(_unpack(st["w"]), st["ws"]), st["splits"]).to(DT[st["out"]])
    x, w = st["x"].float(), st["w"].float()
    out = {"out": _grouped(x, w, st["splits"]).to(DT[st["out"]])}
    if st["train"]:
        dy, used = st["dy"].float(), sum(st["splits"])
        out["dx"] = _grouped(dy, w.transpose(1, 2), st["splits"]).to(DT[st["out"]])
        out["dw"] = torch.stack([a.t() @ b for a, b in zip(dy[:used].split(st["splits"]), x[:used].split(st["splits"]))])
    return out


# ---------------------------------------------------------------------------
# through the library
# ---------------------------------------------------------------------------

def _run_own(st):
    from fp8_precision_allreduce_amd import lpc

    if st["op"] == "muon":
        if "plan" not in st:  # the program's optimizer object: every tensor checked once
            st["plan"] = lpc.Muon(st["p"], st["g"], st["m"], scales=st["scale"], copies=st["copies"])
        st["plan"].step(lr=st["lr"], beta=st["beta"], weight_decay=st["decay"], iterations=NS_ITERATIONS)
        return _muon_outputs(st)
    rows, k, dev = st["rows"], st["k"], st["x"].device
    new = lambda *s, dtype=torch.uint8: torch.empty(*s, dtype=dtype, device=dev)  # noqa: E731
    if st["op"] == "bf16":
        n, g, dt = st["n"], st["groups"], DT[st["out"]]
        out = {"out": new(rows, n, dtype=dt)}
        lpc.lpc_gemm_bf16(st["x"], st["w"], out["out"], counts=st["counts"])
        if st["train"]:
            out["dx"], out["dw"] = new(rows, k, dtype=dt), new(g, n, k, dtype=torch.float32)
            lpc.lpc_gemm_bf16_dgrad(st["dy"], st["w"], out["dx"], counts=st["counts"])
            lpc.lpc_gemm_bf16_wgrad(st["dy"], st["x"], out["dw"], counts=st["counts"])
        return out
    codes, scales = new(rows, k // 2), new(rows, k // MX)
    lpc.lpc_quantize_mxfp4(st["x"], codes, scales)
    if st["op"] == "codec":
        values = new(rows, k, dtype=DT[st["out"]])
        lpc.lpc_dequantize_mxfp4(codes, scales, values)
        return {"values": values, "scales": scales}
    out = new(rows, st["n"], dtype=DT[st["out"]])
    lpc.lpc_gemm_mxfp4(codes, scales, st["w"], st["ws"], out, counts=st["counts"])
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "muon":
        n = products = 0
        for r, c in _shapes(case):
            small, large = min(r, c), max(r, c)
            n += r * c
            products += 3 * small * small * large + small ** 3  # two of the three products are symmetric
        state = 16 + SIZE[case["grad"]] + (2 if case["copy"] else 0)
        return {"bytes": n * state, "flops": NS_ITERATIONS * products + 8 * n}
    rows, k = case["rows"], case["k"]
    if case["op"] == "codec":
        # codes and scales are written and read again by the inverse
        return {"bytes": rows * k * (SIZE[case["in"]] + SIZE[case["out"]]) + rows * (k + k // 16), "flops": 4 * rows * k}
    n, g = case["n"], case["groups"]
    used = rows - case["dropped"]
    weights = min(g, max(used, 1))  # groups that can have rows
    if case["op"] == "mxfp4":
        return {"bytes": used * k * SIZE[case["in"]] + weights * n * (k // 2 + k // MX) + rows * n * SIZE[case["out"]],
                "flops": 2 * used * k * n}
    forward = used * k * 2 + weights * n * k * 2 + rows * n * SIZE[case["out"]]
    backward = used * n * 2 + rows * k * SIZE[case["out"]] + g * n * k * 4 if case["train"] else 0
    return {"bytes": forward + backward, "flops": (6 if case["train"] else 2) * used * k * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _held(x):
    """What microscaled 4-bit floats hold of x: of the eight magnitudes the nearest, between two as near the one of even index."""
    b = x.double().reshape(x.shape[0], -1, MX)
    top = b.abs().amax(-1, keepdim=True)
    powers = torch.tensor([2.0 ** e for e in range(-149, 129)], dtype=torch.float64, device=x.device)
    binade = torch.bucketize(top, powers, right=True) - 1 - 149          # the largest power of two not above the top
    scale = 2.0 ** (binade - 2).clamp(min=-127).double()
    q = b.abs() / scale
    index = torch.zeros_like(q)
    for i in range(7):
        half = (E2M1[i] + E2M1[i + 1]) / 2
        index += (q >= half) if i % 2 else (q > half)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    return (torch.sign(b) * grid[index.long()] * scale).reshape(x.shape)


def _held_codes(codes, byte):
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=codes.device)
    v = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=codes.device)
    v[..., 0::2], v[..., 1::2] = grid[(codes % 16).long()], grid[(codes // 16).long()]
    return v * (2.0 ** (byte.double() - 127)).repeat_interleave(MX, -1)


def _products64(x, w, splits):
    """x's rows of each group times w[g], w [g, k, n]."""
    out = torch.zeros(x.shape[0], w.shape[2], dtype=torch.float64, device=x.device)
    at = 0
    for g, c in enumerate(splits):
        out[at:at + c] = x[at:at + c] @ w[g].double()
        at += c
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "codec":
        return {"values": _held(st["x"]), "scales": None}
    if case["op"] == "mxfp4":
        w = _held_codes(st["w"], st["ws"])
        return _products64(_held(st["x"]), w.transpose(1, 2), st["splits"])
    if case["op"] == "bf16":
        x, at = st["x"].double(), 0
        out = {"out": _products64(x, st["w"].transpose(1, 2), st["splits"])}
        if case["train"]:
            dy = st["dy"].double()
            out["dx"] = _products64(dy, st["w"], st["splits"])
            out["dw"] = torch.zeros(st["w"].shape, dtype=torch.float64, device=x.device)
            for g, c in enumerate(st["splits"]):
                out["dw"][g] = dy[at:at + c].t() @ x[at:at + c]
                at += c
        return out
    out = {"p": [], "m": []}
    for p, g, m, scale in zip(st["p"], st["g"], st["m"], st["scale"]):
        new_p, new_m = [], []
        for q, h, v in zip(p.double(), g.double(), m.double()):
            v = st["beta"] * v + (1 - st["beta"]) * h
            o = st["beta"] * v + (1 - st["beta"]) * h
            if o.norm() > 0:
                o = o / o.norm()
            for _ in range(NS_ITERATIONS):  # odd polynomial of the singular values: the same from either side
                s = o @ o.t() if o.shape[0] <= o.shape[1] else o.t() @ o
                t = NS_B * s + NS_C * (s @ s)
                o = NS_A * o + (t @ o if o.shape[0] <= o.shape[1] else o @ t)
            new_p.append(q - st["lr"] * (st["decay"] * q + scale * o))
            new_m.append(v)
        out["p"].append(torch.stack(new_p))
        out["m"].append(torch.stack(new_m))
    if st["copies"] is not None:
        out["copies"] = out["p"]
    return out
