"""Cases, plain forms and 64-bit definitions of the operators around the update.

Three operators that a training step needs next to the Adam update of the
library: the orthogonalisation of matrices by Newton-Schulz products, the
update of weight matrices by orthogonalised momentum, and the embedding table
at both of its ends (the scaled lookup that reads the BF16 weights an update
wrote, and the gradient, summed by sorted tokens, that an update reads).

run() makes one pass in the plain form (elementary torch operations in 32
bits), or through the library when `own` is set.  exact() evaluates the same
definitions in 64 bits.
"""
import math

import torch

own = False

COEF = (3.4445, -4.7750, 2.0315)     # quintic of the iteration: p(s) = a s + b s^3 + c s^5
STEPS = 5
EPS = 1e-7
LR, BETA, DECAY = 1e-3, 0.95, 0.01

# the 14 LoRA tensors of each of 22 TinyLlama layers (rank 8), by shape
ADAPTERS = "132x8x2048 22x8x5632 66x2048x8 44x256x8 44x5632x8"
# the seven projections of one TinyLlama layer: q, (k, v), o, (gate, up), down
TINY_LAYER = "1x2048x2048 2x256x2048 1x2048x2048 2x5632x2048 1x2048x5632"


def listed():
    return [
        # every adapter gradient of the LoRA workload in one call: 308 tiny matrices, FP32, launch-bound
        dict(name="ortho_adapters", op="ortho", shapes=ADAPTERS, x="f32", y="f32", pad=0),
        # the k projections of all 22 TinyLlama layers, BF16 gradients to BF16 updates
        dict(name="ortho_kv_bf16", op="ortho", shapes="22x256x2048", x="bf16", y="bf16", pad=0),
        # ragged odd matrices held as column slices of wider ones (row strides that are no multiple of anything)
        dict(name="ortho_ragged_f32", op="ortho", shapes="1x1000x777 1x333x2049 2x65x64 1x1x500 1x129x31", x="f32",
             y="f32", pad=3),
        # one MLP projection of LLaMA-7B alone: a large matrix product chain
        dict(name="ortho_mlp_bf16", op="ortho", shapes="1x11008x4096", x="bf16", y="bf16", pad=0),
        # FP32 adapters updated without a BF16 copy, all 308 in one call
        dict(name="muon_adapters", op="muon", shapes=ADAPTERS, grad="f32", weight=False),
        # the seven matrices of one TinyLlama layer, as a layer-wise training loop updates them
        dict(name="muon_layer", op="muon", shapes=TINY_LAYER, grad="bf16", weight=True),
        # the down projection of a 70B-shaped layer: the largest matrix of the streamed workload
        dict(name="muon_down_70b", op="muon", shapes="1x8192x28672", grad="f32", weight=True),
        # a batch of 64 sequences that take one token each: latency
        dict(name="lookup_decode", op="lookup", tokens=64, vocab=32000, width=4096, index="i64", weight="bf16", out="bf16"),
        # a training batch of 8 x 2048 tokens, TinyLlama width
        dict(name="lookup_train", op="lookup", tokens=16384, vocab=32000, width=2048, index="i64", weight="bf16", out="bf16"),
        # a short odd batch: nearly all of the gradient's rows are zero
        dict(name="grad_short", op="grad", tokens=257, vocab=32000, width=2048, index="i64", dy="bf16", grad="bf16",
             add=False),
        # a training batch of 16 x 2048 tokens at LLaMA-7B width, BF16 gradients as the update reads them
        dict(name="grad_train", op="grad", tokens=32768, vocab=32000, width=4096, index="i64", dy="bf16", grad="bf16",
             add=False),
        # one of several long micro-batches added into FP32 gradients at 70B width
        dict(name="grad_add_f32", op="grad", tokens=131072, vocab=32000, width=8192, index="i32", dy="bf16", grad="f32",
             add=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["ortho", "muon", "lookup", "grad"])
    if op in ("ortho", "muon"):
        groups = []
        for _ in range(rng.randint(1, 3)):
            a = _log(rng, 1, 4096)
            b = _log(rng, a, max(a, min(16384, (1 << 25) // a)))
            most = max(1, min(64, (1 << 24) // (a * b)))
            r, c = rng.choice([(a, b), (b, a)])
            groups.append("%dx%dx%d" % (_log(rng, 1, most), r, c))
        if op == "ortho":
            return dict(op=op, shapes=" ".join(groups), x=rng.choice(["bf16", "f32"]), y=rng.choice(["bf16", "f32"]),
                        pad=rng.choice([0, 0, 1, 8, 24]))
        return dict(op=op, shapes=" ".join(groups), grad=rng.choice(["bf16", "f32"]), weight=rng.random() < 0.7)
    width = _log(rng, 8, 8192)
    if rng.random() < 0.7:
        width = max(8, width // 8 * 8)
    vocab = _log(rng, 100, 128000)
    tokens = _log(rng, 1, 131072)
    if op == "lookup":
        return dict(op=op, tokens=tokens, vocab=vocab, width=width, index=rng.choice(["i32", "i64"]),
                    weight=rng.choice(["bf16", "bf16", "f32"]), out=rng.choice(["bf16", "f32"]))
    vocab = min(vocab, 32000 * 8192 // width)
    return dict(op=op, tokens=tokens, vocab=vocab, width=width, index=rng.choice(["i32", "i64"]),
                dy=rng.choice(["bf16", "bf16", "f32"]), grad=rng.choice(["bf16", "f32"]), add=rng.random() < 0.4)


# ------------------------------------------------------------------- inputs

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "i32": torch.int32, "i64": torch.int64}


def _shapes(text):
    return [tuple(int(v) for v in part.split("x")) for part in text.split()]


def _gradient(gen, count, rows, cols):
    """Gradient-like matrices: noise of 1e-3 under a few directions of falling strength."""
    g = torch.randn(count, rows, cols, generator=gen, device="cuda")
    k = min(6, rows, cols)
    u = torch.randn(count, rows, k, generator=gen, device="cuda") * (4.0 / 2.0 ** torch.arange(k, device="cuda"))
    v = torch.randn(count, cols, k, generator=gen, device="cuda")
    return g.baddbmm_(u, v.mT.contiguous()).mul_(1e-3)


def _tokens(gen, n, vocab, dtype):
    """Token ids by a Zipf-like law over shuffled ids; about one in 64 positions is padding (-1)."""
    p = 1.0 / (torch.arange(vocab, device="cuda", dtype=torch.float32) + 2.7)
    ids = torch.randperm(vocab, generator=gen, device="cuda")
    t = ids[torch.multinomial(p, n, replacement=True, generator=gen)]
    t[torch.rand(n, generator=gen, device="cuda") < 1 / 64] = -1
    return t.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "ortho":
        s["x"], s["y"] = [], []
        for count, rows, cols in _shapes(case["shapes"]):
            wide = torch.zeros(count, rows, cols + case["pad"], dtype=DTYPE[case["x"]], device="cuda")
            wide[:, :, :cols] = _gradient(gen, count, rows, cols)
            s["x"].append(wide[:, :, :cols])
            s["y"].append(torch.zeros(count, rows, cols, dtype=DTYPE[case["y"]], device="cuda"))
    elif case["op"] == "muon":
        # one flat array of each kind, matrix after matrix, as in a layer block
        shapes = _shapes(case["shapes"])
        grads = [_gradient(gen, *g) for g in shapes]
        s["grad"] = torch.cat([g.flatten() for g in grads]).to(DTYPE[case["grad"]])
        s["m"] = torch.cat([(0.8 * g + 0.3 * _gradient(gen, *k)).flatten() for g, k in zip(grads, shapes)])
        s["master"] = torch.randn(s["grad"].numel(), generator=gen, device="cuda") * 0.02
        s["weight"] = s["master"].to(torch.bfloat16) if case["weight"] else None
    else:
        n, vocab, width = case["tokens"], case["vocab"], case["width"]
        s["tokens"] = _tokens(gen, n, vocab, DTYPE[case["index"]])
        s["scale"] = math.sqrt(width)
        if case["op"] == "lookup":
            s["weight"] = (torch.randn(vocab, width, generator=gen, device="cuda") * 0.02).to(DTYPE[case["weight"]])
            s["out"] = torch.zeros(n, width, dtype=DTYPE[case["out"]], device="cuda")
        else:
            s["dy"] = (torch.randn(n, width, generator=gen, device="cuda") * 1e-3).to(DTYPE[case["dy"]])
            s["grad"] = torch.zeros(vocab, width, dtype=DTYPE[case["grad"]], device="cuda")
            if case["add"]:
                s["grad"].normal_(0.0, 1e-3, generator=gen)
    if own:
        _plan(s)
    return s


def _plan(s):
    """Tables and workspaces that a program makes once and keeps."""
    import layer_streamed_optimizer_amd as lso
    case = s["case"]
    nbytes = 0
    if case["op"] == "ortho":
        s["table"] = lso.MatrixTable.from_rows(
            dict(x=x[i], y=y[i], rows=x.shape[1], cols=x.shape[2], ld_x=x.stride(1), ld_y=y.stride(1), x_dtype=lso.dtype_of(x),
                 y_dtype=lso.dtype_of(y)) for x, y in zip(s["x"], s["y"]) for i in range(x.shape[0]))
        nbytes = lso.orthogonalize_workspace_bytes(s["table"])
    elif case["op"] == "muon":
        rows_, at, gb = [], 0, s["grad"].element_size()
        for count, rows, cols in _shapes(case["shapes"]):
            for _ in range(count):
                rows_.append(dict(rows=rows, cols=cols, master=s["master"].data_ptr() + 4 * at, m=s["m"].data_ptr() + 4 * at,
                                  grad=s["grad"].data_ptr() + gb * at, grad_dtype=lso.dtype_of(s["grad"]),
                                  weight=s["weight"].data_ptr() + 2 * at if case["weight"] else None, lr=LR, beta=BETA,
                                  weight_decay=DECAY, scale=_scale(rows, cols), nesterov=True))
                at += rows * cols
        s["table"] = lso.MuonTable.from_rows(rows_)
        nbytes = lso.muon_workspace_bytes(s["table"])
    elif case["op"] == "grad":
        nbytes = lso.embed_grad_workspace_bytes(case["tokens"], case["vocab"], case["width"])
    s["workspace"], s["workspace_bytes"] = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda"), nbytes


# -------------------------------------------------------------- one pass

def run(s):
    if own:
        return _own(s)
    return {"ortho": _plain_ortho, "muon": _plain_muon, "lookup": _plain_lookup, "grad": _plain_grad}[s["case"]["op"]](s)


def _own(s):
    import layer_streamed_optimizer_amd as lso
    op = s["case"]["op"]
    if op == "ortho":
        lso.orthogonalize(s["table"], s["workspace"], s["workspace_bytes"], steps=STEPS, eps=EPS)
        return s["y"]
    if op == "muon":
        lso.muon_step(s["table"], s["workspace"], s["workspace_bytes"], steps=STEPS, eps=EPS)
        return _state(s)
    if op == "lookup":
        lso.embed_lookup(s["tokens"], s["weight"], s["out"], scale=s["scale"])
        return s["out"]
    lso.embed_grad(s["tokens"], s["dy"], s["grad"], s["workspace"], s["workspace_bytes"], scale=s["scale"], accumulate=s["case"]["add"])
    return s["grad"]


def _state(s):
    out = dict(master=s["master"], m=s["m"])
    if s["weight"] is not None:
        out["weight"] = s["weight"]
    return out


def _scale(rows, cols):
    return 0.2 * math.sqrt(max(rows, cols))


def _newton_schulz(x):
    """x: FP32 batch of matrices."""
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.mT.contiguous()
    x = x / (torch.sqrt(torch.sum(x * x, dim=(1, 2), keepdim=True)) + EPS)
    a, b, c = COEF
    for _ in range(STEPS):
        gram = torch.bmm(x, x.mT.contiguous())
        x = torch.baddbmm(x, torch.baddbmm(gram, gram, gram, beta=b, alpha=c), x, beta=a)
    return x.mT if tall else x


def _plain_ortho(s):
    for x, y in zip(s["x"], s["y"]):
        y.copy_(_newton_schulz(x.float()))
    return s["y"]


def _plain_muon(s):
    g = s["grad"].float()
    s["m"].mul_(BETA).add_(g, alpha=1 - BETA)
    u = s["m"] * BETA + g * (1 - BETA)
    step, at = torch.empty_like(u), 0
    for count, rows, cols in _shapes(s["case"]["shapes"]):
        n = count * rows * cols
        step[at:at + n].view(count, rows, cols).copy_(_newton_schulz(u[at:at + n].view(count, rows, cols))).mul_(-LR * _scale(rows, cols))
        at += n
    s["master"].mul_(1 - LR * DECAY).add_(step)
    if s["weight"] is not None:
        s["weight"].copy_(s["master"])
    return _state(s)


def _plain_lookup(s):
    t = s["tokens"].long()
    real = (t >= 0) & (t < s["case"]["vocab"])
    rows = s["weight"][t.clamp(0, s["case"]["vocab"] - 1)].float() * s["scale"]
    s["out"].copy_(torch.where(real[:, None], rows, 0.0))
    return s["out"]


def _plain_grad(s):
    t = s["tokens"].long()
    real = (t >= 0) & (t < s["case"]["vocab"])
    total = torch.zeros(s["case"]["vocab"], s["case"]["width"], device="cuda")
    total.index_add_(0, t.clamp(0, s["case"]["vocab"] - 1), torch.where(real[:, None], s["dy"].float(), 0.0))
    total.mul_(s["scale"])
    s["grad"].copy_(total.add_(s["grad"].float()) if s["case"]["add"] else total)
    return s["grad"]


# ------------------------------------------------- what a pass cannot do without

_BYTES = {"f32": 4, "bf16": 2, "i32": 4, "i64": 8}


def _products(rows, cols):
    """Operations of the iteration on one matrix: its Gram matrix and the square of that are symmetric (half
    of each suffices), the product with the matrix is whole."""
    m, n = min(rows, cols), max(rows, cols)
    return STEPS * (3 * m * m * n + m * m * m)


def work(case):
    if case["op"] in ("ortho", "muon"):
        shapes = _shapes(case["shapes"])
        params = sum(k * r * c for k, r, c in shapes)
        flops = sum(k * _products(r, c) for k, r, c in shapes)
        if case["op"] == "ortho":
            return dict(bytes=params * (_BYTES[case["x"]] + _BYTES[case["y"]]), flops=flops)
        return dict(bytes=params * (16 + _BYTES[case["grad"]] + (2 if case["weight"] else 0)), flops=flops)
    n, width, vocab = case["tokens"], case["width"], case["vocab"]
    if case["op"] == "lookup":
        rows = min(n, vocab)   # a row that several tokens share is read once
        return dict(bytes=n * (_BYTES[case["index"]] + width * _BYTES[case["out"]]) + rows * width * _BYTES[case["weight"]],
                    flops=n * width)
    # added to, only the rows of the batch's tokens have to be read and written; else every row is written
    table = (2 * min(n, vocab) if case["add"] else vocab) * width * _BYTES[case["grad"]]
    return dict(bytes=n * (_BYTES[case["index"]] + width * _BYTES[case["dy"]]) + table, flops=n * width)


# ------------------------------------------------------- definitions in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "ortho":
        return [torch.stack([_orthogonal64(m) for m in x]) for x in s["x"]]
    if case["op"] == "muon":
        g = s["grad"].double()
        m = BETA * s["m"].double() + (1 - BETA) * g
        u = BETA * m + (1 - BETA) * g
        master, at = (1 - LR * DECAY) * s["master"].double(), 0
        for count, rows, cols in _shapes(case["shapes"]):
            for _ in range(count):
                n = rows * cols
                master[at:at + n] -= LR * 0.2 * max(rows, cols) ** 0.5 * _orthogonal64(u[at:at + n].view(rows, cols)).flatten()
                at += n
        out = dict(master=master, m=m)
        if case["weight"]:
            out["weight"] = master
        return out
    tokens = s["tokens"].tolist()
    real = [i for i, t in enumerate(tokens) if 0 <= t < case["vocab"]]
    at = torch.tensor(real, dtype=torch.int64, device="cuda")
    ids = torch.tensor([tokens[i] for i in real], dtype=torch.int64, device="cuda")
    if case["op"] == "lookup":
        out = torch.zeros(case["tokens"], case["width"], dtype=torch.float64, device="cuda")
        out[at] = s["weight"].double()[ids] * s["scale"]
        return out
    out = s["grad"].double() if case["add"] else torch.zeros(case["vocab"], case["width"], dtype=torch.float64, device="cuda")
    for part in range(0, len(real), 8192):
        out.index_add_(0, ids[part:part + 8192], s["dy"][at[part:part + 8192]].double(), alpha=s["scale"])
    return out


def _orthogonal64(g):
    """The quintic's iterations on the matrix scaled by its Frobenius norm, the smaller side first."""
    x = g.double()
    if x.shape[0] > x.shape[1]:
        return _orthogonal64(x.T.contiguous()).T
    x = x / (torch.linalg.vector_norm(x) + EPS)
    eye = torch.eye(x.shape[0], dtype=torch.float64, device=x.device)
    for _ in range(STEPS):
        s = x @ x.T
        x = (COEF[0] * eye + COEF[1] * s + COEF[2] * (s @ s)) @ x
    return x
