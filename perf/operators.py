"""Cases of the 8-bit floating point product and of the expert layer around it: what is measured,
the operators' plain forms, and their definitions in 64 bits.

Kinds of cases:

* ``weights``  quantisation of a weight matrix to e4m3 with one scale per 128 x 128 block
* ``rows``     quantisation of activations to e4m3 with one scale per 1 x 128 block
* ``linear``   one quantised layer: activations in, quantised on the way, product, output
* ``product``  the experts' products: rows sorted by expert, each expert's rows with its weights
* ``dispatch`` tokens sorted by expert and laid out so, as they are or quantised on the way
* ``combine``  the experts' outputs back in token order, weighted; with ``train`` its gradients too
"""

import numpy as np
import torch

own = False

BLOCK = 128          # elements of a scale's block
E4M3_MAX = 448.0     # the largest finite e4m3 value
TINY = 2.0 ** -100   # blocks below this absolute maximum take its scale
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def up(a, b):
    return -(-a // b)


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a gate/up weight quantised once, after training
        {"name": "weights_17408x5120", "kind": "weights", "E": 1, "N": 17408, "K": 5120, "dtype": "bf16"},
        # activations of a layer whose width fills no whole block, in 32 bits
        {"name": "rows_777x5121_f32", "kind": "rows", "M": 777, "K": 5121, "dtype": "f32"},
        # one token of one sequence through the attention projection
        {"name": "linear_1x5120x5120", "kind": "linear", "M": 1, "N": 5120, "K": 5120, "dtype": "bf16", "out": "bf16"},
        # a serving step of 24 sequences through the gate/up projection
        {"name": "linear_24x17408x5120", "kind": "linear", "M": 24, "N": 17408, "K": 5120, "dtype": "bf16", "out": "bf16"},
        # no size a multiple of a tile, results in 32 bits
        {"name": "linear_1000x1100x1000_f32", "kind": "linear", "M": 1000, "N": 1100, "K": 1000, "dtype": "f32", "out": "f32"},
        # a prompt chunk, or a chunk of calibration tokens, through the gate/up projection
        {"name": "linear_8192x17408x5120", "kind": "linear", "M": 8192, "N": 17408, "K": 5120, "dtype": "bf16", "out": "bf16"},
        # a serving step: 64 tokens, 8 of 48 experts each, about 11 rows an expert
        {"name": "product_64x8_e48", "kind": "product", "T": 64, "top": 8, "E": 48, "N": 2560, "K": 5120, "out": "bf16"},
        # calibration tokens through the experts: long and ragged runs of rows
        {"name": "product_8192x8_e64", "kind": "product", "T": 8192, "top": 8, "E": 64, "N": 5120, "K": 2048, "out": "bf16"},
        # a serving step: sort and quantise 64 tokens on the way to the experts
        {"name": "dispatch_64x8_fp8", "kind": "dispatch", "T": 64, "top": 8, "E": 48, "K": 5120, "dtype": "bf16", "fp8": True},
        # a calibration chunk laid out by expert for the experts' Hessians
        {"name": "dispatch_16384x8", "kind": "dispatch", "T": 16384, "top": 8, "E": 64, "K": 5120, "dtype": "bf16", "fp8": False},
        # a serving step's outputs back in token order
        {"name": "combine_64x8", "kind": "combine", "T": 64, "top": 8, "E": 48, "K": 5120, "dtype": "bf16", "train": False},
        # outputs, and the gradients of rows, weights and tokens
        {"name": "combine_8192x8_train", "kind": "combine", "T": 8192, "top": 8, "E": 64, "K": 5120, "dtype": "bf16", "train": True},
    ]


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, even over its logarithm; two in three end in anything, one is a multiple of 128."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    if rng.random() < 1 / 3 and v > 2 * BLOCK:
        v -= v % BLOCK
    return min(hi, max(lo, v))


def draw(rng):
    most = {c["kind"]: work(c) for c in listed()}
    while True:
        kind = rng.choice(["weights", "rows", "linear", "linear", "product", "dispatch", "combine"])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if kind == "weights":
            c = {"kind": kind, "E": rng.choice([1, 1, 3]), "N": _spread(rng, 64, 17408), "K": _spread(rng, 64, 17408), "dtype": dtype}
        elif kind == "rows":
            c = {"kind": kind, "M": _spread(rng, 1, 8192), "K": _spread(rng, 64, 17408), "dtype": dtype}
        elif kind == "linear":
            c = {"kind": kind, "M": _spread(rng, 1, 8192), "N": _spread(rng, 64, 17408), "K": _spread(rng, 64, 17408),
                 "dtype": dtype, "out": dtype}
        elif kind == "product":
            c = {"kind": kind, "T": _spread(rng, 1, 8192), "top": rng.randint(1, 8), "E": _spread(rng, 8, 128),
                 "N": _spread(rng, 64, 5120), "K": _spread(rng, 64, 5120), "out": dtype}
        elif kind == "dispatch":
            c = {"kind": kind, "T": _spread(rng, 1, 16384), "top": rng.randint(1, 8), "E": _spread(rng, 8, 256),
                 "K": _spread(rng, 64, 5120), "dtype": dtype, "fp8": rng.random() < 0.5}
        else:
            c = {"kind": kind, "T": _spread(rng, 1, 8192), "top": rng.randint(1, 8), "E": _spread(rng, 8, 256),
                 "K": _spread(rng, 64, 5120), "dtype": dtype, "train": rng.random() < 0.5}
        w, top = work(c), most.get(kind)
        limit = work(listed()[0]) if kind in ("weights", "rows") else top
        if w["bytes"] <= limit["bytes"] and w["flops"] <= limit["flops"]:
            return c


def work(case):
    c = case
    if c["kind"] == "weights":
        n = c["E"] * c["N"] * c["K"]
        return {"bytes": n * (SIZE[c["dtype"]] + 1) + 4 * c["E"] * up(c["N"], BLOCK) * up(c["K"], BLOCK), "flops": 2 * n}
    if c["kind"] == "rows":
        n = c["M"] * c["K"]
        return {"bytes": n * (SIZE[c["dtype"]] + 1) + 4 * c["M"] * up(c["K"], BLOCK), "flops": 2 * n}
    if c["kind"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": M * K * SIZE[c["dtype"]] + N * K + 4 * up(N, BLOCK) * up(K, BLOCK) + M * N * SIZE[c["out"]],
                "flops": 2 * M * N * K}
    if c["kind"] == "product":
        R, N, K = c["T"] * c["top"], c["N"], c["K"]
        experts = min(c["E"], R)  # an expert without rows is not read: this many have some at most
        return {"bytes": R * K + 4 * R * up(K, BLOCK) + experts * (N * K + 4 * up(N, BLOCK) * up(K, BLOCK)) + R * N * SIZE[c["out"]],
                "flops": 2 * R * N * K}
    T, top, K, s = c["T"], c["top"], c["K"], SIZE[c["dtype"]]
    if c["kind"] == "dispatch":
        row = K + 4 * up(K, BLOCK) if c["fp8"] else K * s
        return {"bytes": 12 * T * top + T * K * s + T * top * row, "flops": T * K}
    back = T * K * s + T * top * (2 * K * s + 12)  # the output's gradient, rows read, their gradient written
    again = T * top * K * s + T * K * s            # the rows' gradients summed over each token's copies
    return {"bytes": T * top * (K * s + 8) + T * K * s + (back + again if c["train"] else 0),
            "flops": 2 * T * top * K * (4 if c["train"] else 1)}


# ------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(g, M, K, dtype):
    """Tokens with channels of uneven size: lognormal scales and one channel in a hundred 20 times larger."""
    scale = torch.exp(torch.randn(K, generator=g, device="cuda"))
    big = torch.rand(K, generator=g, device="cuda") < 0.01
    return (torch.randn((M, K), generator=g, device="cuda") * torch.where(big, 20 * scale, scale)).to(dtype)


def _pitch(K):
    return up(K, 16) * 16


def _in_blocks(x, rows, cols):
    """x [..., n, k] -> [..., ceil(n/rows), rows, ceil(k/cols), cols], zeros at the edges."""
    n, k = x.shape[-2:]
    x = torch.nn.functional.pad(x, (0, -k % cols, 0, -n % rows))
    return x.reshape(*x.shape[:-2], up(n, rows), rows, up(k, cols), cols)


def _quantise(x, rows):
    """e4m3 codes [..., n, pitch] and scales [..., ceil(n/rows), ceil(k/128)] of x [..., n, k], in 32 bits."""
    n, k = x.shape[-2:]
    b = _in_blocks(x.float(), rows, BLOCK)
    top = b.abs().amax((-3, -1), keepdim=True)
    held = torch.where(top == 0, top, top.clamp_min(TINY))
    most = torch.full_like(held, E4M3_MAX)  # a tensor: a division by a number becomes a product
    codes = torch.where(held == 0, torch.zeros_like(b), (b * (most / held)).clamp(-E4M3_MAX, E4M3_MAX))
    codes = codes.reshape(*codes.shape[:-4], codes.shape[-4] * rows, -1)[..., :n, :k].to(torch.float8_e4m3fn)
    return codes, (held / most).squeeze(-1).squeeze(-2)


def _laid_out(codes):
    """Codes with each row padded to 16 bytes, as the framework keeps them."""
    k = codes.shape[-1]
    out = torch.zeros((*codes.shape[:-1], _pitch(k)), dtype=torch.uint8, device=codes.device)
    out[..., :k] = codes.view(torch.uint8)
    return out.view(torch.float8_e4m3fn)


def _router(g, T, top, E):
    """`top` different experts for each token from uneven router scores, one choice in 64 dropped (-1), and their weights."""
    score = torch.randn((T, E), generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda")
    best, ids = score.topk(min(top, E), dim=1)
    ids = ids.to(torch.int32)
    ids = torch.where(torch.rand(ids.shape, generator=g, device="cuda") < 1 / 64, torch.full_like(ids, -1), ids)
    return ids.contiguous(), torch.softmax(best, 1).contiguous()


def _sorted(ids, E):
    """offsets [E + 1], order and position [T, top] of a stable sort by expert; what is dropped has position -1."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.sort(key, stable=True).indices
    ends = torch.searchsorted(key[order], torch.arange(E + 1, device=ids.device))
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=ids.device)
    place = torch.where(key < E, place, torch.full_like(place, -1))
    return ends.to(torch.int32), order.to(torch.int32), place.to(torch.int32).reshape(ids.shape)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["kind"] == "weights":
        s["W"] = (torch.randn((c["E"], c["N"], c["K"]), generator=g, device="cuda") * 0.02).to(TYPES[c["dtype"]])
        s["codes"] = torch.zeros((c["E"], c["N"], _pitch(c["K"])), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        s["scales"] = torch.zeros((c["E"], up(c["N"], BLOCK), up(c["K"], BLOCK)), device="cuda")
    elif c["kind"] == "rows":
        s["X"] = _activations(g, c["M"], c["K"], TYPES[c["dtype"]])
        s["codes"] = torch.zeros((c["M"], _pitch(c["K"])), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        s["scales"] = torch.zeros((up(c["K"], BLOCK), c["M"]), device="cuda")
    elif c["kind"] == "linear":
        s["X"] = _activations(g, c["M"], c["K"], TYPES[c["dtype"]])
        W = torch.randn((c["N"], c["K"]), generator=g, device="cuda") * 0.02
        codes, s["w_scales"] = _quantise(W, BLOCK)
        s["w_scales"] = s["w_scales"].contiguous()
        s["w_codes"] = _laid_out(codes)
        s["Y"] = torch.zeros((c["M"], c["N"]), dtype=TYPES[c["out"]], device="cuda")
        # scratch of the quantised activations: codes, scales and room to align them
        s["workspace"] = torch.empty(c["M"] * _pitch(c["K"]) + 4 * c["M"] * up(c["K"], BLOCK) + 1024, dtype=torch.uint8, device="cuda")
    elif c["kind"] == "product":
        ids, _ = _router(g, c["T"], c["top"], c["E"])
        s["offsets"], order, _ = _sorted(ids, c["E"])
        s["longest"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        X = _activations(g, c["T"], c["K"], torch.float32)
        codes, scales = _quantise(X, 1)
        token = (order.long() // ids.shape[1])
        s["codes"], s["scales"] = _laid_out(codes.view(torch.uint8)[token].view(torch.float8_e4m3fn)), scales[token].t().contiguous()
        del X, codes, scales
        s["w_codes"] = torch.zeros((c["E"], c["N"], _pitch(c["K"])), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        s["w_scales"] = torch.empty((c["E"], up(c["N"], BLOCK), up(c["K"], BLOCK)), device="cuda")
        for e in range(c["E"]):
            W = torch.randn((c["N"], c["K"]), generator=g, device="cuda") * 0.02
            codes, s["w_scales"][e] = _quantise(W, BLOCK)
            s["w_codes"][e] = _laid_out(codes)
        s["Y"] = torch.zeros((token.numel(), c["N"]), dtype=TYPES[c["out"]], device="cuda")
    else:
        s["ids"], s["weights"] = _router(g, c["T"], c["top"], c["E"])
        T, top = s["ids"].shape
        R = T * top
        if c["kind"] == "dispatch":
            s["X"] = _activations(g, T, c["K"], TYPES[c["dtype"]])
            s["offsets"] = torch.zeros(c["E"] + 1, dtype=torch.int32, device="cuda")
            s["order"] = torch.zeros(R, dtype=torch.int32, device="cuda")
            s["position"] = torch.zeros((T, top), dtype=torch.int32, device="cuda")
            s["workspace"] = torch.empty((R // 512 + 2) * (c["E"] + 1) * 4 + 4096, dtype=torch.uint8, device="cuda")
            if c["fp8"]:
                s["codes"] = torch.zeros((R, _pitch(c["K"])), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                s["scales"] = torch.zeros((up(c["K"], BLOCK), R), device="cuda")
            else:
                s["rows"] = torch.zeros((R, c["K"]), dtype=TYPES[c["dtype"]], device="cuda")
        else:
            s["rows"] = torch.randn((R, c["K"]), generator=g, device="cuda").to(TYPES[c["dtype"]])
            s["position"] = _sorted(s["ids"], c["E"])[2]
            s["Y"] = torch.zeros((T, c["K"]), dtype=TYPES[c["dtype"]], device="cuda")
            if c["train"]:
                s["dY"] = torch.randn((T, c["K"]), generator=g, device="cuda").to(TYPES[c["dtype"]])
                s["d_rows"] = torch.zeros_like(s["rows"])
                s["d_weights"] = torch.zeros_like(s["weights"])
                s["dX"] = torch.zeros_like(s["dY"])
    return s


# ------------------------------------------------------------------------------------- one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import post_weight_quantization_tcgen05_b200 as hq
    c = s["case"]
    if c["kind"] == "weights":
        hq.hq_fp8_quantize_blocks(s["W"], s["codes"], s["scales"])
        return {"codes": s["codes"], "scales": s["scales"]}
    if c["kind"] == "rows":
        hq.hq_fp8_quantize_rows(s["X"], s["codes"], s["scales"])
        return {"codes": s["codes"], "scales": s["scales"]}
    if c["kind"] == "linear":
        hq.hq_fp8_linear(s["X"], s["w_codes"], s["w_scales"], s["Y"], s["workspace"])
        return s["Y"]
    if c["kind"] == "product":
        hq.hq_fp8_expert_gemm(s["codes"], s["scales"], s["offsets"], s["w_codes"], s["w_scales"], c["K"], s["Y"])
        return s["Y"]
    if c["kind"] == "dispatch":
        hq.hq_expert_sort(s["ids"], c["E"], s["offsets"], s["order"], s["position"], s["workspace"])
        plan = {k: s[k] for k in ("offsets", "order", "position")}
        if c["fp8"]:
            hq.hq_expert_dispatch_fp8(s["X"], s["position"], s["codes"], s["scales"])
            return {**plan, "codes": s["codes"], "scales": s["scales"]}
        hq.hq_expert_dispatch(s["X"], s["position"], s["rows"])
        return {**plan, "rows": s["rows"]}
    hq.hq_expert_combine(s["rows"], s["position"], s["weights"], s["Y"])
    if not c["train"]:
        return s["Y"]
    hq.hq_expert_combine_backward(s["dY"], s["rows"], s["position"], s["weights"], s["d_rows"], s["d_weights"])
    hq.hq_expert_combine(s["d_rows"], s["position"], None, s["dX"])  # the dispatch's gradient
    return {"Y": s["Y"], "d_rows": s["d_rows"], "d_weights": s["d_weights"], "dX": s["dX"]}


def _dequantised(codes, scales, rows, K):
    """codes [..., n, pitch] times the scales [..., ceil(n/rows), ceil(k/128)] of their blocks, in 32 bits."""
    n = codes.shape[-2]
    b = _in_blocks(codes[..., :K].float(), rows, BLOCK) * scales.unsqueeze(-2).unsqueeze(-1)
    return b.reshape(*b.shape[:-4], b.shape[-4] * rows, -1)[..., :n, :K]


def _plain(s):
    c = s["case"]
    if c["kind"] == "weights":
        codes, scales = _quantise(s["W"], BLOCK)
        return {"codes": _laid_out(codes), "scales": scales}
    if c["kind"] == "rows":
        codes, scales = _quantise(s["X"], 1)
        return {"codes": _laid_out(codes), "scales": scales.t()}
    if c["kind"] == "linear":
        codes, scales = _quantise(s["X"], 1)
        Y = _dequantised(codes, scales, 1, c["K"]) @ _dequantised(s["w_codes"], s["w_scales"], BLOCK, c["K"]).t()
        return Y.to(s["Y"].dtype)
    if c["kind"] == "product":
        A = _dequantised(s["codes"], s["scales"].t(), 1, c["K"])
        start, end = s["offsets"][:-1, None].long(), s["offsets"][1:, None].long()
        at = start + torch.arange(s["longest"], device="cuda")  # [E, longest]: each expert's rows, and some past them
        here = at < end
        P = torch.bmm(A[at.clamp(max=A.shape[0] - 1)], _dequantised(s["w_codes"], s["w_scales"], BLOCK, c["K"]).transpose(1, 2))
        Y = torch.zeros((A.shape[0] + 1, c["N"]), device="cuda")  # one row more, for those past an expert's rows
        Y[torch.where(here, at, torch.full_like(at, A.shape[0]))] = P
        return Y[:-1].to(s["Y"].dtype)
    if c["kind"] == "dispatch":
        top = s["ids"].shape[1]
        offsets, order, position = _sorted(s["ids"], c["E"])
        filled = torch.arange(order.numel(), device="cuda") < offsets[-1]
        order = torch.where(filled, order, torch.zeros_like(order))
        token = order.long() // top
        plan = {"offsets": offsets, "order": order, "position": position}
        if c["fp8"]:
            codes, scales = _quantise(s["X"], 1)
            codes = torch.where(filled[:, None], _laid_out(codes).view(torch.uint8)[token], 0).view(torch.float8_e4m3fn)
            return {**plan, "codes": codes, "scales": torch.where(filled[:, None], scales[token], 0.0).t()}
        return {**plan, "rows": torch.where(filled[:, None], s["X"][token], 0.0)}
    here = (s["position"] >= 0)[..., None]
    at = s["position"].clamp_min(0).long()
    w = s["weights"][..., None]
    Z = torch.where(here, s["rows"][at].float(), 0.0)
    Y = (w * Z).sum(1).to(s["Y"].dtype)
    if not c["train"]:
        return Y
    dY = s["dY"].float()[:, None]
    d_weights = (dY * Z).sum(2)
    d_rows = torch.zeros((s["rows"].shape[0] + 1, c["K"]), dtype=s["rows"].dtype, device="cuda")
    d_rows[torch.where(here[..., 0], at, torch.full_like(at, s["rows"].shape[0]))] = (w * dY).to(s["rows"].dtype)
    d_rows = d_rows[:-1]
    dX = torch.where(here, d_rows[at].float(), 0.0).sum(1).to(s["Y"].dtype)
    return {"Y": Y, "d_rows": d_rows, "d_weights": d_weights, "dX": dX}


# ------------------------------------------------------------------------------------- in 64 bits

def _codes64(X, rows):
    """The quantiser's definition, block maxima over `rows` rows and 128 columns: the scale is the 32-bit
    quotient a / 448, a code the e4m3 value next to the 32-bit product of x and the 32-bit quotient 448 / a.
    Each of the three is taken in 64 bits and rounded once; codes and scales come back in 64 bits."""
    n, k = X.shape
    x = X.double()
    a = torch.zeros((up(n, rows), up(k, BLOCK)), dtype=torch.float64, device=X.device)
    whole = k - k % BLOCK
    line = torch.cat([x[:, :whole].abs().reshape(n, -1, BLOCK).amax(2)] + ([x[:, whole:].abs().amax(1, keepdim=True)] if whole < k else []), 1)
    group = (torch.arange(n, device=X.device) // rows)[:, None].expand_as(line)
    a.scatter_reduce_(0, group, line, "amax")
    a = torch.where((a > 0) & (a < TINY), torch.full_like(a, TINY), a)
    scales = (a / E4M3_MAX).float().double()
    turn = torch.where(a > 0, (E4M3_MAX / a).float().double(), torch.zeros_like(a))
    col = torch.arange(k, device=X.device) // BLOCK
    row = torch.arange(n, device=X.device) // rows
    codes = (x * turn[row][:, col]).float().clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).double()
    return codes, scales, row, col


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] in ("weights", "rows"):
        parts = [_codes64(x, BLOCK if c["kind"] == "weights" else 1)[:2] for x in (s["W"] if c["kind"] == "weights" else [s["X"]])]
        pad = _pitch(c["K"]) - c["K"]
        codes = torch.stack([torch.nn.functional.pad(p[0], (0, pad)) for p in parts])
        scales = torch.stack([p[1] for p in parts])
        return {"codes": codes, "scales": scales} if c["kind"] == "weights" else {"codes": codes[0], "scales": scales[0].t()}
    if c["kind"] == "linear":
        codes, scales, row, col = _codes64(s["X"], 1)
        A = codes * scales[:, col]
        n = torch.arange(c["N"], device="cuda") // BLOCK
        return A @ (s["w_codes"][:, :c["K"]].double() * s["w_scales"].double()[n][:, col]).t()
    if c["kind"] == "product":
        if 2 * c["T"] * c["top"] * c["N"] * c["K"] > 4e12:
            return None
        col = torch.arange(c["K"], device="cuda") // BLOCK
        n = torch.arange(c["N"], device="cuda") // BLOCK
        Y = torch.zeros(s["Y"].shape, dtype=torch.float64, device="cuda")
        ends = s["offsets"].tolist()
        for e in range(c["E"]):
            if ends[e] < ends[e + 1]:
                A = s["codes"][ends[e]:ends[e + 1], :c["K"]].double() * s["scales"][:, ends[e]:ends[e + 1]].double().t()[:, col]
                Y[ends[e]:ends[e + 1]] = A @ (s["w_codes"][e, :, :c["K"]].double() * s["w_scales"][e].double()[n][:, col]).t()
        return Y
    ids = s["ids"].cpu().numpy()
    T, top = ids.shape
    if c["kind"] == "dispatch":
        lists = [np.flatnonzero(ids.reshape(-1) == e) for e in range(c["E"])]  # each expert's choices in token order
        offsets = np.cumsum([0] + [len(v) for v in lists])
        order, position = np.zeros(T * top, np.int32), np.full(T * top, -1, np.int32)
        filled = np.concatenate(lists)
        order[:len(filled)] = filled
        position[filled] = np.arange(len(filled))
        plan = {"offsets": torch.from_numpy(offsets.astype(np.int32)), "order": torch.from_numpy(order),
                "position": torch.from_numpy(position.reshape(T, top))}
        token = torch.from_numpy(filled // top).cuda()
        if c["fp8"]:
            codes, scales, _, _ = _codes64(s["X"], 1)
            laid = torch.zeros(s["codes"].shape, dtype=torch.float64, device="cuda")
            laid[:len(filled), :c["K"]] = codes[token]
            by = torch.zeros(s["scales"].shape, dtype=torch.float64, device="cuda")
            by[:, :len(filled)] = scales[token].t()
            return {**plan, "codes": laid, "scales": by}
        rows = torch.zeros(s["rows"].shape, dtype=torch.float64, device="cuda")
        rows[:len(filled)] = s["X"][token].double()
        return {**plan, "rows": rows}
    Y = torch.zeros((T, c["K"]), dtype=torch.float64, device="cuda")
    position = s["position"].long()
    for j in range(top):
        t = torch.nonzero(position[:, j] >= 0)[:, 0]
        Y[t] += s["weights"][t, j, None].double() * s["rows"][position[t, j]].double()
    if not c["train"]:
        return Y
    d_rows = torch.zeros(s["rows"].shape, dtype=torch.float64, device="cuda")
    d_weights = torch.zeros((T, top), dtype=torch.float64, device="cuda")
    dX = torch.zeros_like(Y)
    for j in range(top):
        t = torch.nonzero(position[:, j] >= 0)[:, 0]
        p = position[t, j]
        d_rows[p] = s["weights"][t, j, None].double() * s["dY"][t].double()
        d_weights[t, j] = torch.linalg.vecdot(s["dY"][t].double(), s["rows"][p].double())
        dX[t] += s["weights"][t, j, None].double() * s["dY"][t].double()
    return {"Y": Y, "d_rows": d_rows, "d_weights": d_weights, "dX": dX}
