"""The products of a language model that go beyond a plain matrix product: what is measured of them.

Four operators on 16-bit inputs with FP32 accumulation:

  grouped   the rows of A come in groups (tokens sorted by expert), each group has a weight of its own:
            C[rows of g] = A[rows of g] @ op(B[g]); its backward pass is the same product with the weights turned
            round, and one product per group over the group's rows: dB[g] = A[rows of g]^T @ dC[rows of g]
  xent      the output layer with its loss: l = X @ W^T, lse = log(sum(exp(l))), loss = lse - l[target], and the
            gradients of sum(dloss * loss) with respect to X and W, without the logits being kept
  w4        C = X @ Wq^T, the weights in 4 bits with one scale (and one zero point) per group along K
  w4_pack   a 16-bit weight to that form, and back
"""
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CHUNK = 128          # the packed form keeps 128 consecutive k of a row together


def listed():
    return [
        # one decoding step of 4 requests, two experts each: latency counts
        dict(name="grouped decode 8 rows", op="grouped", way="forward", T=8, G=8, K=512, N=1024, trans_b=True, dtype="fp16", out="same"),
        # one decoding step of a batch: every expert's weight is read for a few rows
        dict(name="grouped decode 128 rows", op="grouped", way="forward", T=128, G=16, K=4096, N=2048, trans_b=True, dtype="bf16", out="same"),
        # a prompt whose sizes fit no tile and no 16-byte row, uneven experts, FP32 result
        dict(name="grouped prompt 3001x4999x2047", op="grouped", way="forward", T=3001, G=5, K=2047, N=4999, trans_b=False, dtype="fp16", out="fp32"),
        # the training step of one expert layer: gradients of the rows and of every expert's weight
        dict(name="grouped backward 16384 rows", op="grouped", way="backward", T=16384, G=16, K=2048, N=4096, trans_b=False, dtype="bf16", out="same"),
        # scoring a short answer: the loss alone
        dict(name="xent score 17x32000x1024", op="xent", way="forward", T=17, V=32000, H=1024, ignore=0.0, dtype="fp16"),
        # a fine-tuning step: odd vocabulary, a third of the rows belongs to the prompt and is ignored
        dict(name="xent train 2047x50021x2048", op="xent", way="train", T=2047, V=50021, H=2048, ignore=0.35, dtype="bf16"),
        # a training step over a large vocabulary
        dict(name="xent train 8192x128000x4096", op="xent", way="train", T=8192, V=128000, H=4096, ignore=0.0, dtype="bf16"),
        # one token through one layer
        dict(name="w4 1x4096x4096", op="w4", M=1, N=4096, K=4096, group=128, zeros=False, dtype="fp16", out="same"),
        # a small batch of tokens, with zero points and short groups
        dict(name="w4 8x14336x4096 zeros", op="w4", M=8, N=14336, K=4096, group=32, zeros=True, dtype="bf16", out="same"),
        # a prompt through the same form of weights
        dict(name="w4 2048x8192x4096", op="w4", M=2048, N=8192, K=4096, group=64, zeros=True, dtype="fp16", out="fp32"),
        # a small odd weight
        dict(name="w4 pack 1001x1000", op="w4_pack", N=1001, K=1000, group=32, zeros=True, dtype="fp16"),
        # one layer's weight
        dict(name="w4 pack 14336x4096", op="w4_pack", N=14336, K=4096, group=128, zeros=False, dtype="bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _extent(rng, lo, hi, odd):
    """A size between lo and hi, spread over its logarithm: any whole number in a share `odd`, else a multiple of 8."""
    n = _log_uniform(rng, lo, hi)
    return n if rng.random() < odd else max(8, n // 8 * 8)


def draw(rng):
    op = rng.choice(["grouped", "grouped", "xent", "xent", "w4", "w4", "w4_pack"])
    dtype = rng.choice(["bf16", "fp16"])
    out = rng.choice(["same", "same", "fp32"])
    if op == "grouped":
        while True:
            c = dict(op=op, way=rng.choice(["forward", "backward"]), T=_log_uniform(rng, 1, 16384), G=_log_uniform(rng, 1, 64), K=_extent(rng, 64, 4096, 0.2), N=_extent(rng, 64, 5000, 0.2),
                     trans_b=rng.choice([False, True]), dtype=dtype, out=out)
            if c["G"] * c["K"] * c["N"] <= 2 ** 28 and c["T"] * c["K"] * c["N"] <= 2 ** 37:
                return c
    if op == "xent":
        while True:
            c = dict(op=op, way=rng.choice(["forward", "train"]), T=_log_uniform(rng, 1, 8192), V=_log_uniform(rng, 1000, 128000), H=_extent(rng, 64, 4096, 0.2),
                     ignore=rng.choice([0.0, 0.1, 0.5]), dtype=dtype)
            if c["T"] * c["V"] * c["H"] <= 2 ** 40:
                return c
    c = dict(op=op, M=_log_uniform(rng, 1, 2048), N=_extent(rng, 64, 14336, 0.3), K=_extent(rng, 64, 8192, 0.2), group=rng.choice([32, 64, 128]), zeros=rng.choice([False, True]),
             dtype=dtype, out=out)
    if op == "w4_pack":
        del c["M"], c["out"]
    return c


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


def _ceil(n, to):
    return (n + to - 1) // to * to


def _pack(q):
    """4-bit values q [N, multiple of 128] in the framework's packed form: 32 bits hold 8 consecutive k, element 2i in
    bits 4i and element 2i + 1 in bits 16 + 4i; the four words of k = 8 j.. + 32 s, s = 0..3, lie side by side."""
    N, K = q.shape
    w = q.view(N, K // CHUNK, 4, 4, 4, 2).to(torch.int32)                        # chunk, s, j, i, parity
    shift = torch.tensor([[4 * i + 16 * p for p in range(2)] for i in range(4)], device=q.device, dtype=torch.int32)
    words = (w << shift).sum((-1, -2), dtype=torch.int32)                        # chunk, s, j
    return words.transpose(2, 3).contiguous().view(torch.uint8).view(N, K // 2)  # chunk, j, s


def _unpack(packed):
    N, half = packed.shape
    words = packed.view(torch.int32).view(N, half * 2 // CHUNK, 4, 4).transpose(2, 3).reshape(N, half * 2 // CHUNK, 4, 4, 1, 1)
    shift = torch.tensor([[4 * i + 16 * p for p in range(2)] for i in range(4)], device=packed.device, dtype=torch.int32)
    return ((words >> shift) & 15).reshape(N, half * 2)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=case["dtype"]):
        return torch.randn(shape, device="cuda", generator=gen).mul_(scale).to(DTYPES[dtype])

    if case["op"] == "grouped":
        T, G, K, N = case["T"], case["G"], case["K"], case["N"]
        bounds = _bounds(case, seed)
        state = dict(A=normal(T, K), B=normal(*((G, N, K) if case["trans_b"] else (G, K, N)), scale=K ** -0.5), bounds=bounds,
                     offsets=torch.tensor(bounds, dtype=torch.int32, device="cuda"))
        if case["way"] == "backward":
            state["D"] = normal(T, N)
    elif case["op"] == "xent":
        T, V, H = case["T"], case["V"], case["H"]
        target = torch.randint(0, V, (T,), device="cuda", generator=gen)
        if case["ignore"]:
            target[torch.rand(T, device="cuda", generator=gen) < case["ignore"]] = -100
        # logits of deviation 3, so that a row's few largest share most of its probability
        state = dict(X=normal(T, H), W=normal(V, H, scale=3 * H ** -0.5), target=target)
        # gradients of a mean with a weight for each row; FP16 training scales its loss
        scale = (1024.0 if case["dtype"] == "fp16" else 1.0) / T
        state["dloss"] = torch.rand(T, device="cuda", generator=gen).add_(0.5).mul_(scale)
    else:
        N, K, group = case["N"], case["K"], case["group"]
        if case["op"] == "w4_pack":
            state = dict(W=normal(N, K, scale=K ** -0.5))
        else:
            Kp = _ceil(K, CHUNK)
            q = torch.randn(N, Kp, device="cuda", generator=gen).mul_(2.5).add_(8).round_().clamp_(0, 15)
            scales = torch.rand(N, Kp // group, device="cuda", generator=gen).add_(0.5).mul_(0.4 * K ** -0.5).to(DTYPES[case["dtype"]])
            zeros = torch.randint(5, 12, (N, Kp // group), device="cuda", generator=gen, dtype=torch.uint8) if case["zeros"] else None
            state = dict(X=normal(case["M"], K), packed=_pack(q.to(torch.uint8)), scales=scales, zeros=zeros)
    return dict(state, case=case, out=DTYPES[case["dtype"] if case.get("out", "same") == "same" else case["out"]])


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import fp32_sgemm_tuning_amd as lib

    c = s["case"]
    if c["op"] == "grouped":
        if c["way"] == "forward":
            return lib.sgemm_grouped(s["A"], s["B"], s["offsets"], trans_b=c["trans_b"], out_dtype=s["out"])
        dA = lib.sgemm_grouped(s["D"], s["B"], s["offsets"], trans_b=not c["trans_b"], out_dtype=s["out"])
        first, second = (s["D"], s["A"]) if c["trans_b"] else (s["A"], s["D"])
        return dA, lib.sgemm_grouped_wgrad(first, second, s["offsets"], out_dtype=s["out"])
    if c["op"] == "xent":
        loss, lse = lib.sgemm_xent(s["X"], s["W"], s["target"])
        if c["way"] == "forward":
            return loss, lse
        return (loss, lse, *lib.sgemm_xent_grad(s["X"], s["W"], s["target"], lse, s["dloss"]))
    if c["op"] == "w4":
        return lib.sgemm_w4(s["X"], lib.W4Weight(s["packed"], s["scales"], s["zeros"], c["K"], c["group"]), out_dtype=s["out"])
    packed = lib.sgemm_w4_quantize(s["W"], group=c["group"], zeros=c["zeros"])
    values = lib.sgemm_w4_dequantize(packed)
    return (values, packed.scales, packed.zeros) if c["zeros"] else (values, packed.scales)


def _run_plain(s):
    c, out = s["case"], s["out"]
    if c["op"] == "grouped":
        groups = [(g, slice(a, b)) for g, (a, b) in enumerate(zip(s["bounds"], s["bounds"][1:]))]
        A, turn = s["A"].float(), c["trans_b"] != (c["way"] == "backward")
        rows = s["D"].float() if c["way"] == "backward" else A
        products = [rows[r] @ (s["B"][g].float().T if turn else s["B"][g].float()) for g, r in groups if r.stop > r.start]
        if c["way"] == "forward":
            return torch.cat(products).to(out)
        first, second = (rows, A) if c["trans_b"] else (A, rows)
        return torch.cat(products).to(out), torch.stack([first[r].T @ second[r] for _, r in groups]).to(out)
    if c["op"] == "xent":
        X, W = s["X"].float(), s["W"].float()
        valid = s["target"] != -100
        at = s["target"].clamp(min=0)[:, None]
        logits = X @ W.T
        top = logits.amax(1, keepdim=True)
        lse = (logits - top).exp().sum(1, keepdim=True).log() + top
        loss = torch.where(valid, (lse - logits.gather(1, at))[:, 0], 0.0)
        lse_out = torch.where(valid, lse[:, 0], 0.0)
        if c["way"] == "forward":
            return loss, lse_out
        P = logits.sub_(lse).exp_()
        P.scatter_add_(1, at, torch.full_like(lse, -1.0))
        P.mul_(torch.where(valid, s["dloss"], 0.0)[:, None])
        return loss, lse_out, (P @ W).to(out), (P.T @ X).to(out)
    if c["op"] == "w4":
        N, Kp = s["packed"].shape[0], s["packed"].shape[1] * 2
        q = _unpack(s["packed"]).view(N, Kp // c["group"], c["group"])
        zero = 8.0 if s["zeros"] is None else s["zeros"].float()[:, :, None]
        W = ((q - zero) * s["scales"].float()[:, :, None]).view(N, Kp)[:, : c["K"]]
        return (s["X"].float() @ W.T).to(out)
    W, N, K, group = s["W"].float(), c["N"], c["K"], c["group"]
    W = torch.nn.functional.pad(W, (0, _ceil(K, CHUNK) - K)).view(N, -1, group)
    if c["zeros"]:
        low = W.amin(2).clamp(max=0)
        scales = torch.div(W.amax(2).clamp(min=0) - low, torch.full_like(low, 15.0)).to(out)
        step = torch.where(scales == 0, 1.0, scales.float())
        zero = torch.round(-low / step).clamp(0, 15)
    else:
        top = W.abs().amax(2)
        scales = torch.div(top, torch.full_like(top, 7.0)).to(out)
        step = torch.where(scales == 0, 1.0, scales.float())
        zero = torch.full_like(top, 8.0)
    q = torch.where((scales == 0)[:, :, None], zero[:, :, None], (torch.round(W / step[:, :, None]) + zero[:, :, None]).clamp(0, 15))
    values = ((q - zero[:, :, None]) * scales.float()[:, :, None]).view(N, -1)[:, :K].to(out)
    return (values, scales, zero.to(torch.uint8)) if c["zeros"] else (values, scales)


def work(case):
    op, size = case["op"], 2
    out = 4 if case.get("out") == "fp32" else 2
    if op == "grouped":
        T, G, K, N = case["T"], case["G"], case["K"], case["N"]
        used = G * (1 - (1 - 1 / G) ** T)             # groups that have rows, about
        if case["way"] == "forward":
            return dict(bytes=size * (T * K + used * K * N) + out * T * N, flops=2 * T * K * N)
        return dict(bytes=size * (T * K + T * N + used * K * N) + out * (T * K + G * K * N), flops=4 * T * K * N)
    if op == "xent":
        T, V, H = case["T"], case["V"], case["H"]
        valid = T * (1 - case["ignore"])
        train = case["way"] == "train"
        return dict(bytes=size * (valid * H + V * H) * (2 if train else 1) + 16 * T, flops=(6 if train else 2) * valid * V * H)
    N, K, groups = case["N"], case["K"], -(-case["K"] // case["group"])
    packed = N * K // 2 + N * groups * (3 if case["zeros"] else 2)
    if op == "w4":
        return dict(bytes=packed + case["M"] * (size * K + out * N), flops=2 * case["M"] * N * K)
    return dict(bytes=2 * packed + 2 * size * N * K, flops=6 * N * K)  # read, written packed, read packed, written


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "grouped":
        row_group = torch.bucketize(torch.arange(case["T"], device="cuda"), s["offsets"][1:].long(), right=True)
        B = s["B"].double()
        B = B.mT if case["trans_b"] else B            # [G, K, N]
        A = s["A"].double()
        if case["way"] == "forward":
            C = A.new_zeros(case["T"], case["N"])
            for g in range(case["G"]):
                rows = (row_group == g).nonzero()[:, 0]
                C[rows] = torch.mm(A[rows], B[g])
            return C
        D, dA, dB = s["D"].double(), torch.zeros_like(A), torch.zeros_like(B)
        for g in range(case["G"]):
            rows = (row_group == g).nonzero()[:, 0]
            dA[rows] = torch.mm(D[rows], B[g].T)
            dB[g] = torch.mm(A[rows].T, D[rows])
        return dA, (dB.mT if case["trans_b"] else dB)
    if case["op"] == "xent":
        X, W, t = s["X"].double(), s["W"].double(), s["target"]
        loss, lse = X.new_zeros(case["T"]), X.new_zeros(case["T"])
        dX, dW = torch.zeros_like(X), torch.zeros_like(W)
        for rows in torch.nonzero(t != -100)[:, 0].split(1024):
            l = torch.mm(X[rows], W.T)
            lse[rows] = torch.logsumexp(l, 1)
            loss[rows] = lse[rows] - l[torch.arange(len(rows), device="cuda"), t[rows]]
            if case["way"] == "train":
                dl = torch.softmax(l, 1)
                dl[torch.arange(len(rows), device="cuda"), t[rows]] -= 1
                dl *= s["dloss"][rows].double()[:, None]
                dX[rows] = torch.mm(dl, W)
                dW += torch.mm(dl.T, X[rows])
        return (loss, lse, dX, dW) if case["way"] == "train" else (loss, lse)
    if case["op"] == "w4":
        words = s["packed"].view(torch.int32).long() & 0xFFFFFFFF
        k = torch.arange(case["K"], device="cuda")
        inside = k % CHUNK
        word = k // CHUNK * 16 + inside % 32 // 8 * 4 + inside // 32
        bit = 4 * (k % 8 // 2) + 16 * (k % 2)
        q = ((words[:, word] >> bit) & 15).double()
        zero = 8.0 if s["zeros"] is None else s["zeros"].double()[:, k // case["group"]]
        return torch.mm(s["X"].double(), ((q - zero) * s["scales"].double()[:, k // case["group"]]).T)
    W, group, dtype = s["W"].double(), case["group"], s["out"]
    k = torch.arange(case["K"], device="cuda") // group
    groups = _ceil(case["K"], CHUNK) // group
    top, low = W.new_zeros(case["N"], groups), W.new_zeros(case["N"], groups)
    top.scatter_reduce_(1, k.expand_as(W), W if case["zeros"] else W.abs(), "amax")
    low.scatter_reduce_(1, k.expand_as(W), W, "amin")
    scales = ((top - low) / 15 if case["zeros"] else top / 7).to(dtype).double()
    step = torch.where(scales == 0, 1.0, scales)
    zero = torch.round(-low / step).clamp(0, 15) if case["zeros"] else torch.full_like(top, 8.0)
    values = (torch.round(W / step[:, k]).clamp(-zero[:, k], 15 - zero[:, k])) * scales[:, k]
    return (values, scales, None) if case["zeros"] else (values, scales)
