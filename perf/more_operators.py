"""An expert layer's routing and its products in 8-bit integers: what is measured of them.

Five operators:

  sort      each token goes to `picks` experts: its row is brought to every one of its places among the rows sorted
            by expert (stable: rows of an expert by token, then by pick), with the experts' bounds and the permutation;
            gradient: each token's gradient is the sum over its rows
  combine   the way back: out[t] = sum_j weights[t][j] * Y[place of (t, j)];
            gradients: dY[place of (t, j)] = weights[t][j] * D[t], dweights[t][j] = <D[t], Y[place of (t, j)]>
  i8        C[m][n] = sx[m] * sw[n] * sum_k x[m][k] * w[n][k] with x and w in 8-bit integers: a scale for each token
            and for each output channel
  i8_grouped  the same with the tokens sorted by expert and one weight for each expert
  i8_quant  a matrix to that form, row by row, and back
"""
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
ROW = 16             # rows of 8-bit matrices start at multiples of 16 bytes, as the framework's quantisation lays them out


def listed():
    return [
        # one decoding step of 4 requests: latency counts
        dict(name="sort decode 4x2 rows", op="sort", way="forward", T=4, picks=2, G=8, H=512, drop=0.0, ids="int64", dtype="fp16"),
        # the training step of a layer of many small experts
        dict(name="sort train 8192x8 rows", op="sort", way="train", T=8192, picks=8, G=128, H=4096, drop=0.0, ids="int64", dtype="bf16"),
        # a padded prompt's way back, of a width that fits no 16-byte row; the experts' results are in FP32
        dict(name="combine prompt 3001x6 odd", op="combine", way="forward", T=3001, picks=6, G=60, H=2047, drop=0.3, weights="bf16", dtype="fp32", out="bf16"),
        # the training step: gradients of the experts' results and of the router's weights
        dict(name="combine backward 16384x2 rows", op="combine", way="backward", T=16384, picks=2, G=16, H=4096, drop=0.0, weights="fp32", dtype="bf16", out="bf16"),
        # one token through one layer
        dict(name="i8 1x4096x4096", op="i8", M=1, N=4096, K=4096, out="fp16", aligned=True),
        # a small batch of tokens
        dict(name="i8 33x14336x4096", op="i8", M=33, N=14336, K=4096, out="bf16", aligned=True),
        # a prompt whose sizes fit no tile, FP32 result
        dict(name="i8 3001x4999x2047", op="i8", M=3001, N=4999, K=2047, out="fp32", aligned=True),
        # a long prompt, or many at once
        dict(name="i8 8192x14336x4096", op="i8", M=8192, N=14336, K=4096, out="bf16", aligned=True),
        # one decoding step of a batch: every expert's weight is read for a few rows
        dict(name="i8 grouped decode 128 rows", op="i8_grouped", T=128, G=16, K=4096, N=2048, out="bf16", aligned=True),
        # a prompt through an expert layer
        dict(name="i8 grouped prompt 16384 rows", op="i8_grouped", T=16384, G=16, K=2048, N=4096, out="bf16", aligned=True),
        # the tokens of a decoding step, of an odd width
        dict(name="i8 quant 17x1001", op="i8_quant", M=17, K=1001, dtype="fp16"),
        # the tokens of a prompt
        dict(name="i8 quant 16384x4096", op="i8_quant", M=16384, K=4096, dtype="bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _extent(rng, lo, hi, odd):
    """A size between lo and hi, spread over its logarithm: any whole number in a share `odd`, else a multiple of 8."""
    n = _log_uniform(rng, lo, hi)
    return n if rng.random() < odd else max(8, n // 8 * 8)


def draw(rng):
    op = rng.choice(["sort", "sort", "combine", "combine", "i8", "i8", "i8", "i8_grouped", "i8_grouped", "i8_quant"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    out = rng.choice(["bf16", "fp16", "fp32"])
    if op in ("sort", "combine"):
        while True:
            c = dict(op=op, T=_log_uniform(rng, 1, 16384), picks=rng.randint(1, 8), G=_log_uniform(rng, 2, 256), H=_extent(rng, 64, 8192, 0.3), drop=rng.choice([0.0, 0.0, 0.1, 0.5]), dtype=dtype)
            if c["picks"] <= c["G"] and c["T"] * (c["picks"] + 1) * c["H"] * SIZE[dtype] <= 8192 * 9 * 4096 * 2:
                break
        if op == "sort":
            return dict(c, way=rng.choice(["forward", "train"]), ids=rng.choice(["int32", "int64"]))
        # 16-bit results give a result of their own type or FP32; FP32 results give any
        out = out if dtype == "fp32" else rng.choice([dtype, dtype, "fp32"])
        return dict(c, way=rng.choice(["forward", "backward"]), weights=rng.choice(["fp32", "fp32", out]), out=out)
    if op == "i8":
        while True:
            c = dict(op=op, M=_log_uniform(rng, 1, 8192), N=_extent(rng, 64, 14336, 0.3), K=_extent(rng, 64, 8192, 0.3), out=out, aligned=rng.random() < 0.7)
            if c["M"] * c["N"] * c["K"] <= 8192 * 14336 * 4096:
                return c
    if op == "i8_grouped":
        while True:
            c = dict(op=op, T=_log_uniform(rng, 1, 16384), G=_log_uniform(rng, 1, 64), K=_extent(rng, 64, 4096, 0.3), N=_extent(rng, 64, 5000, 0.3), out=out, aligned=rng.random() < 0.7)
            if c["G"] * c["K"] * c["N"] <= 2 ** 28 and c["T"] * c["K"] * c["N"] <= 2 ** 37:
                return c
    return dict(op=op, M=_log_uniform(rng, 1, 16384), K=_extent(rng, 64, 4096, 0.3), dtype=dtype)


def _bounds(case, seed):
    """Row bounds of the groups: uneven shares, as a router gives them, and one group without rows where there are four or more."""
    rng = random.Random(seed * 7919 + case["T"])
    share = [rng.expovariate(1.0) + 0.3 for _ in range(case["G"])]
    if case["G"] >= 4:
        share[1] = 0.0
    count = [0] * case["G"]
    for g in rng.choices(range(case["G"]), share, k=case["T"]):
        count[g] += 1
    bounds = [0]
    for n in count:
        bounds.append(bounds[-1] + n)
    return bounds


def _order(experts, G):
    """Bounds [G + 1], the place of each (token, pick) among the sorted rows, and the (token, pick) of each row."""
    T, picks = experts.shape
    ids = experts.reshape(-1).long()
    kept = (ids >= 0) & (ids < G)
    ids = torch.where(kept, ids, G)
    source = torch.argsort(ids, stable=True)
    position = torch.empty_like(source)
    position[source] = torch.arange(len(source), device=source.device)
    position = torch.where(kept, position, -1)
    offsets = torch.searchsorted(ids[source], torch.arange(G + 1, device=source.device))
    source = torch.where(torch.arange(len(source), device=source.device) < offsets[G], source, -1)
    return offsets.int(), position.view(T, picks).int(), source.int()


def _i8(values, aligned):
    """An 8-bit matrix whose rows start at multiples of ROW bytes (aligned), or one after another."""
    K = values.shape[-1]
    pad = -K % ROW if aligned else 0
    return torch.nn.functional.pad(values, (0, pad))[..., :K]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype):
        return torch.randn(shape, device="cuda", generator=gen).mul_(scale).to(DTYPES[dtype])

    def quantised(*shape):
        """Values of rows whose largest is 127, as quantisation leaves them, and a scale for each row."""
        q = torch.randn(shape, device="cuda", generator=gen).mul_(36).round_().clamp_(-127, 127).to(torch.int8)
        return _i8(q, case["aligned"]), torch.rand(shape[:-1], device="cuda", generator=gen).add_(0.5).mul_(shape[-1] ** -0.25 / 36)

    state = dict(case=case)
    if case["op"] in ("sort", "combine"):
        T, picks, G, H = case["T"], case["picks"], case["G"], case["H"]
        # distinct experts of uneven popularity; a share of the tokens is padding
        score = torch.randn(T, G, device="cuda", generator=gen) + torch.randn(G, device="cuda", generator=gen)
        best, experts = score.topk(picks, 1)
        if case["drop"]:
            experts[torch.rand(T, device="cuda", generator=gen) < case["drop"]] = -1
        if case["op"] == "sort":
            state.update(X=normal(T, H, dtype=case["dtype"]), experts=experts.int() if case["ids"] == "int32" else experts)
            if case["way"] == "train":
                state["D"] = normal(T * picks, H, dtype=case["dtype"])
        else:
            state["offsets"], state["position"], state["source"] = _order(experts, G)
            state.update(Y=normal(T * picks, H, dtype=case["dtype"]), weights=torch.softmax(best, 1).to(DTYPES[case["weights"]]))
            if case["way"] == "backward":
                state["D"] = normal(T, H, dtype=case["out"])
    elif case["op"] == "i8":
        state["x"], state["sx"] = quantised(case["M"], case["K"])
        state["w"], state["sw"] = quantised(case["N"], case["K"])
    elif case["op"] == "i8_grouped":
        state["bounds"] = _bounds(case, seed)
        state["offsets"] = torch.tensor(state["bounds"], dtype=torch.int32, device="cuda")
        state["x"], state["sx"] = quantised(case["T"], case["K"])
        state["w"], state["sw"] = quantised(case["G"], case["N"], case["K"])
    else:
        # activations: a few channels far above the others
        channel = torch.ones(case["K"], device="cuda")
        channel[torch.randint(0, case["K"], (max(1, case["K"] // 200),), device="cuda", generator=gen)] = 20.0
        state["X"] = (torch.randn(case["M"], case["K"], device="cuda", generator=gen) * channel).to(DTYPES[case["dtype"]])
    return state


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import fp32_sgemm_tuning_amd as lib

    c = s["case"]
    if c["op"] == "sort":
        rows, order = lib.sgemm_grouped_sort(s["X"], s["experts"], c["G"])
        if c["way"] == "forward":
            return rows, order.offsets, order.position, order.source
        return rows, order.offsets, order.position, order.source, lib.sgemm_grouped_combine(s["D"], order)
    if c["op"] == "combine":
        order = lib.GroupOrder(s["offsets"], s["position"], s["source"])
        if c["way"] == "forward":
            return lib.sgemm_grouped_combine(s["Y"], order, s["weights"], out_dtype=DTYPES[c["out"]])
        return lib.sgemm_grouped_combine_grad(s["D"], s["Y"], order, s["weights"])
    if c["op"] == "i8_quant":
        q = lib.sgemm_i8_quantize(s["X"])
        return lib.sgemm_i8_dequantize(q, DTYPES[c["dtype"]]), q.scales
    X, W = lib.I8Matrix(s["x"], s["sx"]), lib.I8Matrix(s["w"], s["sw"])
    if c["op"] == "i8":
        return lib.sgemm_i8(X, W, out_dtype=DTYPES[c["out"]])
    return lib.sgemm_i8_grouped(X, W, s["offsets"], out_dtype=DTYPES[c["out"]])


def _run_plain(s):
    c = s["case"]
    if c["op"] == "sort":
        offsets, position, source = _order(s["experts"], c["G"])
        live = (source >= 0)[:, None]
        rows = torch.where(live, s["X"][source.clamp(min=0) // c["picks"]], 0)
        if c["way"] == "forward":
            return rows, offsets, position, source
        D = torch.where((position >= 0)[:, :, None], s["D"][position.clamp(min=0)].float(), 0.0)
        return rows, offsets, position, source, D.sum(1).to(s["X"].dtype)
    if c["op"] == "combine":
        live, weights = s["position"] >= 0, s["weights"].float()
        Y = s["Y"][s["position"].clamp(min=0)].float()             # [T, picks, H]
        if c["way"] == "forward":
            return (Y * torch.where(live, weights, 0.0)[:, :, None]).sum(1).to(DTYPES[c["out"]])
        D = s["D"].float()
        dweights = torch.where(live, (Y * D[:, None]).sum(2), 0.0).to(s["weights"].dtype)
        at = s["source"].clamp(min=0).long()
        dY = torch.where((s["source"] >= 0)[:, None], D[at // c["picks"]] * weights.reshape(-1)[at][:, None], 0.0)
        return dY.to(s["Y"].dtype), dweights
    if c["op"] == "i8":
        return (s["x"].float() @ s["w"].float().T * s["sx"][:, None] * s["sw"]).to(DTYPES[c["out"]])
    if c["op"] == "i8_grouped":
        groups = [(g, slice(a, b)) for g, (a, b) in enumerate(zip(s["bounds"], s["bounds"][1:])) if b > a]
        x = s["x"].float()
        return torch.cat([x[r] @ s["w"][g].float().T * s["sx"][r, None] * s["sw"][g] for g, r in groups]).to(DTYPES[c["out"]])
    X = s["X"].float()
    top = X.abs().amax(1, keepdim=True)
    scales = torch.div(top, torch.full_like(top, 127.0)).clamp(min=torch.finfo(torch.float32).tiny)
    q = torch.round(X.double() / scales.double())                  # in 64 bits: values next to a border between two steps
    return (q.float() * scales).to(s["X"].dtype), scales[:, 0]


def work(case):
    op = case["op"]
    if op in ("sort", "combine"):
        size, T, H, picks = SIZE[case["dtype"]], case["T"], case["H"], case["picks"]
        rows = T * picks
        if op == "sort":
            plan = rows * (16 if case["ids"] == "int64" else 12) + 4 * case["G"]
            moved = size * (T * H + rows * H)
            return dict(bytes=plan + moved * (2 if case["way"] == "train" else 1), flops=rows * H if case["way"] == "train" else 0)
        kept, out, weights = rows * (1 - case["drop"]), SIZE[case["out"]], SIZE[case["weights"]]
        if case["way"] == "forward":
            return dict(bytes=rows * (4 + weights) + size * kept * H + out * T * H, flops=2 * kept * H)
        return dict(bytes=rows * (8 + 2 * weights) + size * (kept + rows) * H + out * T * (1 - case["drop"]) * H, flops=3 * kept * H)
    if op == "i8_quant":
        size = SIZE[case["dtype"]]
        return dict(bytes=case["M"] * (case["K"] * (2 * size + 2) + 8), flops=4 * case["M"] * case["K"])  # read, written, read, written back
    rows, used = (case["M"], 1) if op == "i8" else (case["T"], case["G"] * (1 - (1 - 1 / case["G"]) ** case["T"]))
    N, K = case["N"], case["K"]
    return dict(bytes=rows * (K + 4) + used * N * (K + 4) + SIZE[case["out"]] * rows * N, flops=2 * rows * N * K)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sort":
        flat = s["experts"].reshape(-1)
        found = [torch.nonzero(flat == g)[:, 0] for g in range(case["G"])]
        bounds = [0]
        for f in found:
            bounds.append(bounds[-1] + len(f))
        source, position = flat.new_full((len(flat),), -1), flat.new_full((len(flat),), -1)
        source[: bounds[-1]] = torch.cat(found)
        rows = s["X"].new_zeros(len(flat), case["H"], dtype=torch.float64)
        rows[: bounds[-1]] = s["X"].double()[torch.div(source[: bounds[-1]], case["picks"], rounding_mode="floor").long()]
        position[source[: bounds[-1]].long()] = torch.arange(bounds[-1], device="cuda", dtype=position.dtype)
        out = rows, torch.tensor(bounds, device="cuda"), position.view(case["T"], -1), source
        if case["way"] == "forward":
            return out
        dX = torch.zeros_like(s["X"], dtype=torch.float64)
        for j in range(case["picks"]):
            p = position.view(case["T"], -1)[:, j].long()
            dX[p >= 0] += s["D"][p[p >= 0]].double()
        return *out, dX
    if case["op"] == "combine":
        out = s["Y"].new_zeros(case["T"], case["H"], dtype=torch.float64)
        dY, dweights = torch.zeros_like(s["Y"], dtype=torch.float64), torch.zeros_like(s["weights"], dtype=torch.float64)
        for j in range(case["picks"]):
            t = torch.nonzero(s["position"][:, j] >= 0)[:, 0]
            p, w = s["position"][t, j].long(), s["weights"][t, j].double()[:, None]
            if case["way"] == "forward":
                out[t] += s["Y"][p].double() * w
            else:
                dY[p] = s["D"][t].double() * w
                dweights[t, j] = torch.linalg.vecdot(s["D"][t].double(), s["Y"][p].double())
        return out if case["way"] == "forward" else (dY, dweights)
    if case["op"] == "i8":
        return torch.mm(s["x"].double() * s["sx"].double()[:, None], (s["w"].double() * s["sw"].double()[:, None]).T)
    if case["op"] == "i8_grouped":
        C = s["sx"].new_zeros(case["T"], case["N"], dtype=torch.float64)
        row_group = torch.bucketize(torch.arange(case["T"], device="cuda"), s["offsets"][1:].long(), right=True)
        for g in range(case["G"]):
            r = torch.nonzero(row_group == g)[:, 0]
            C[r] = torch.mm(s["x"][r].double() * s["sx"][r].double()[:, None], (s["w"][g].double() * s["sw"][g].double()[:, None]).T)
        return C
    X = s["X"].double()
    low, high = torch.aminmax(X, dim=1)
    scale32 = (torch.maximum(-low, high) / 127).float().double()   # the scale is kept in 32 bits, and q chosen for it
    return torch.round(X / scale32[:, None]) * scale32[:, None], scale32
