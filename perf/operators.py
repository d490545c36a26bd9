"""The training operators beside the optimizer step, as cases to time and compare.

The operators make the gradients that the library's optimizer steps take, from
activations kept in 8 bits: the RMS norm with the residual's addition and the
gated unit (both write 8-bit copies of what their backward passes read), the
weight gradient of a linear layer from an 8-bit activation, and the embedding
lookup with its gradient.

8-bit values: groups of 32 consecutive columns share a scale 2^e, the smallest
with max |v| <= 448 * 2^e and -117 <= e <= 119; each value is v / 2^e rounded to
the 8-bit floating type with 4 exponent and 3 mantissa bits (float8_e4m3fn).

Each case is a dict: "op" names the operator and its direction, the other
entries its sizes, types and options.  `own` selects the library's kernels;
otherwise `run` computes the same in elementary torch operations.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 32
EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one new token through a narrow block: only the call's latency counts
        dict(name="norm_fwd_1x768", op="norm_fwd", rows=1, cols=768, dtype="bf16", residual=True),
        # a training batch of 16 K tokens through the norm of a 4096-wide block
        dict(name="norm_fwd_16384x4096", op="norm_fwd", rows=16384, cols=4096, dtype="bf16", residual=True),
        # the same block's backward pass, the residual's gradient added
        dict(name="norm_bwd_16384x4096", op="norm_bwd", rows=16384, cols=4096, dtype="bf16", residual=True),
        # a ragged batch in 32 bits, rows that no vector load is aligned to
        dict(name="norm_bwd_4099x1001_f32", op="norm_bwd", rows=4099, cols=1001, dtype="f32", residual=False),
        # the gated unit of a narrow block, a batch with an odd number of tokens
        dict(name="gate_fwd_2049x1536", op="gate_fwd", rows=2049, cols=1536, dtype="bf16"),
        # the gated unit's backward pass at the wide block's inner width
        dict(name="gate_bwd_8192x14336", op="gate_bwd", rows=8192, cols=14336, dtype="bf16"),
        # the smallest matrix of the optimizer's workloads, a short batch whose activation is packed in the pass
        dict(name="wgrad_256_256x768", op="wgrad", tokens=256, n=256, k=768, out="f32", add=False, gain=False, pack=True),
        # a narrow projection (80 outputs) over a long ragged batch, added to the gradient of an earlier micro-batch
        dict(name="wgrad_16001_80x1536", op="wgrad", tokens=16001, n=80, k=1536, out="f32", add=True, gain=False, pack=False),
        # the widest matrix of the transformer set behind a norm whose gain is folded in
        dict(name="wgrad_8192_14336x4096", op="wgrad", tokens=8192, n=14336, k=4096, out="bf16", add=False, gain=True, pack=False),
        # the lookup of a training batch in a table of 32000 x 4096
        dict(name="embed_16384_32000x4096", op="embed_fwd", tokens=16384, vocab=32000, cols=4096, table="bf16", dtype="bf16",
             ids="i64", ignored=0.0),
        # a few tokens' gradient into a small table: latency
        dict(name="embed_grad_37_1000x64", op="embed_bwd", tokens=37, vocab=1000, cols=64, table="f32", dtype="f32", ids="i64",
             ignored=0.1),
        # the gradient of a 32 K-token batch, words as frequent as in text, a tenth of the tokens padding
        dict(name="embed_grad_32768_32000x4096", op="embed_bwd", tokens=32768, vocab=32000, cols=4096, table="f32",
             dtype="bf16", ids="i32", ignored=0.1),
    ]


def _size(rng, lo, hi):
    """Spread over the logarithm; every other one a multiple of 32 where that fits."""
    n = min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))
    if rng.random() < 0.5 and -(-n // 32) * 32 <= hi:
        n = -(-n // 32) * 32
    return n


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "gate_fwd", "gate_bwd", "wgrad", "wgrad", "embed_fwd", "embed_bwd", "embed_bwd"])
    pick = lambda *v: rng.choice(v)  # noqa: E731
    while True:
        if op.startswith("norm"):
            c = dict(op=op, rows=_size(rng, 1, 32768), cols=_size(rng, 40, 12288), dtype=pick("bf16", "bf16", "f32"),
                     residual=rng.random() < 0.7)
            ok = c["rows"] * c["cols"] <= 16384 * 4096
        elif op.startswith("gate"):
            c = dict(op=op, rows=_size(rng, 1, 16384), cols=_size(rng, 40, 14336), dtype=pick("bf16", "bf16", "f32"))
            ok = c["rows"] * c["cols"] <= 8192 * 14336 // 2
        elif op == "wgrad":
            c = dict(op=op, tokens=_size(rng, 1, 16384), n=_size(rng, 24, 14336), k=_size(rng, 24, 14336),
                     out=pick("f32", "bf16"), add=rng.random() < 0.3, gain=rng.random() < 0.4, pack=rng.random() < 0.3)
            ok = c["tokens"] * c["n"] * c["k"] <= 8192 * 14336 * 4096 // 2
        else:
            c = dict(op=op, tokens=_size(rng, 1, 32768), vocab=_size(rng, 100, 50000), cols=_size(rng, 40, 6000),
                     table=pick("f32", "bf16"), dtype=pick("f32", "bf16"), ids=pick("i32", "i64"),
                     ignored=pick(0.0, 0.05, 0.5))
            ok = max(c["tokens"], c["vocab"]) * c["cols"] <= 32768 * 4096
        if ok:
            return c


# ---------------------------------------------------------------- inputs ----
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _stream(g, rows, cols, dtype):
    """Values like a residual stream's: a spread of token sizes, a few columns far larger than the rest."""
    x = _randn(g, rows, cols) * torch.exp2(torch.randint(-2, 3, (rows, 1), generator=g, device=DEV).float())
    x[:, torch.randint(0, cols, (max(1, cols // 256),), generator=g, device=DEV)] *= 16.0
    return x.to(dtype)


def _pack(x):
    """(codes, biased exponents) of the 8-bit form of a matrix."""
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    v = torch.nn.functional.pad(x.float(), (0, groups * GROUP - cols)).view(rows, groups, GROUP)
    e = _exponent(v.abs().amax(-1))
    codes = (v * torch.exp2(-e).unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.view(rows, -1)[:, :cols].contiguous(), (e + 127.0).to(torch.uint8)


def _exponent(amax):
    """The smallest e with amax <= 448 * 2^e, in [-117, 119]."""
    m, e = torch.frexp(amax)                      # amax = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = e.to(amax.dtype) - 9.0 + (m > 0.875).to(amax.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, -117.0)).clamp(-117.0, 119.0)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case=case)
    if op == "norm_fwd":
        dt = TYPES[case["dtype"]]
        s["x"] = _stream(g, case["rows"], case["cols"], dt)
        s["r"] = _randn(g, case["rows"], case["cols"]).to(dt) if case["residual"] else None
        s["gain"] = 1.0 + 0.2 * _randn(g, case["cols"])
    elif op == "norm_bwd":
        dt = TYPES[case["dtype"]]
        x = _stream(g, case["rows"], case["cols"], torch.float32)
        rstd = torch.rsqrt(x.square().mean(1) + EPS)
        s["codes"], s["scales"] = _pack(x * rstd[:, None])
        s["rstd"] = rstd
        s["gain"] = 1.0 + 0.2 * _randn(g, case["cols"])
        s["dy"] = _randn(g, case["rows"], case["cols"]).to(dt)
        s["dres"] = _randn(g, case["rows"], case["cols"]).to(dt) if case["residual"] else None
    elif op == "gate_fwd":
        # gate and up are the two halves of one projection's output
        s["gu"] = (2.0 * _randn(g, case["rows"], 2 * case["cols"])).to(TYPES[case["dtype"]])
    elif op == "gate_bwd":
        s["gate"] = _pack(2.0 * _randn(g, case["rows"], case["cols"]))
        s["up"] = _pack(2.0 * _randn(g, case["rows"], case["cols"]))
        s["da"] = _randn(g, case["rows"], case["cols"]).to(TYPES[case["dtype"]])
    elif op == "wgrad":
        x = _stream(g, case["tokens"], case["k"], torch.float32)
        x = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
        if case["pack"]:
            s["x"] = x.bfloat16()
        else:
            s["codes"], s["scales"] = _pack(x)
        s["dy"] = _randn(g, case["tokens"], case["n"]).bfloat16()
        s["gain"] = 1.0 + 0.2 * _randn(g, case["k"]) if case["gain"] else None
        s["base"] = (math.sqrt(case["tokens"]) * _randn(g, case["n"], case["k"])).to(TYPES[case["out"]]) if case["add"] else None
    else:
        n, v = case["tokens"], case["vocab"]
        # word frequencies fall off as 1 / rank; ids are ranks shuffled over the table
        rank = torch.exp(torch.rand(n, generator=g, device=DEV) * math.log(v)).long().clamp(max=v) - 1
        ids = torch.randperm(v, generator=g, device=DEV)[rank]
        if case["ignored"]:
            ids = torch.where(torch.rand(n, generator=g, device=DEV) < case["ignored"], torch.full_like(ids, -1), ids)
        s["ids"] = ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)
        s["scale"] = math.sqrt(case["cols"])
        if op == "embed_fwd":
            s["table"] = (0.02 * _randn(g, v, case["cols"])).to(TYPES[case["table"]])
        else:
            s["dy"] = _randn(g, n, case["cols"]).to(TYPES[case["dtype"]])
    return s


# ------------------------------------------------------------ plain form ----
def _unpack(codes, scales):
    cols = codes.shape[1]
    s = torch.exp2(scales.float() - 127.0).repeat_interleave(GROUP, dim=1)[:, :cols]
    return codes.float() * s


def _rounded(x):
    """The values that the 8-bit form of x stands for (bfloat16 holds them exactly)."""
    return _unpack(*_pack(x)).bfloat16()


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "norm_fwd":
        dt = s["x"].dtype
        h = s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()
        rstd = torch.rsqrt((h * h).mean(1) + EPS)
        n = h * rstd[:, None]
        out = dict(y=(n * s["gain"]).to(dt), n=_rounded(n), rstd=rstd)
        if s["r"] is not None:
            out["h"] = h.to(dt)
        return out
    if op == "norm_bwd":
        n = _unpack(s["codes"], s["scales"])
        dy = s["dy"].float()
        gd = dy * s["gain"]
        dx = s["rstd"][:, None] * (gd - n * (gd * n).mean(1, keepdim=True))
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        return dict(dx=dx.to(s["dy"].dtype), dgain=(dy * n).sum(0))
    if op == "gate_fwd":
        k = c["cols"]
        gate, up = s["gu"][:, :k].float(), s["gu"][:, k:].float()
        a = gate / (1.0 + torch.exp(-gate)) * up
        return dict(a=a.to(s["gu"].dtype), gate=_rounded(gate), up=_rounded(up))
    if op == "gate_bwd":
        gate, up, da = _unpack(*s["gate"]), _unpack(*s["up"]), s["da"].float()
        sig = 1.0 / (1.0 + torch.exp(-gate))
        act = gate * sig
        dt = s["da"].dtype
        return dict(dgate=(da * up * (sig + act * (1.0 - sig))).to(dt), dup=(da * act).to(dt), a=_rounded(act * up))
    if op == "wgrad":
        codes, scales = _pack(s["x"]) if c["pack"] else (s["codes"], s["scales"])
        dw = s["dy"].float().t() @ _unpack(codes, scales)
        if s["gain"] is not None:
            dw = dw * s["gain"]
        if s["base"] is not None:
            dw = dw + s["base"].float()
        return dict(dw=dw.to(TYPES[c["out"]]))
    ids, v = s["ids"].long(), c["vocab"]
    valid = (ids >= 0) & (ids < v)
    if op == "embed_fwd":
        rows = s["table"][torch.where(valid, ids, torch.zeros_like(ids))].float() * s["scale"]
        return dict(out=(rows * valid[:, None]).to(TYPES[c["dtype"]]))
    # ignored tokens are added to a row past the table's end
    grad = torch.zeros(v + 1, c["cols"], device=s["dy"].device)
    grad.index_add_(0, torch.where(valid, ids, torch.full_like(ids, v)), s["dy"].float() * s["scale"])
    return dict(grad=grad[:v].to(TYPES[c["table"]]))


# ------------------------------------------------------- the library's own ----
def _library(s):
    import matrix_aware_optimizer_libmuon_amd as muon
    c = s["case"]
    op = c["op"]
    if op == "norm_fwd":
        h, y, n8, rstd = muon.rmsnorm_act8(s["x"], s["gain"], residual=s["r"], eps=EPS)
        out = dict(y=y, n=muon.act8_unpack(n8), rstd=rstd)
        if s["r"] is not None:
            out["h"] = h
        return out
    if op == "norm_bwd":
        dx, dgain = muon.rmsnorm_act8_grad(s["dy"], muon.Act8(s["codes"], s["scales"]), s["rstd"], s["gain"], dres=s["dres"])
        return dict(dx=dx, dgain=dgain)
    if op == "gate_fwd":
        k = c["cols"]
        a, gate8, up8 = muon.swiglu_act8(s["gu"][:, :k], s["gu"][:, k:])
        return dict(a=a, gate=muon.act8_unpack(gate8), up=muon.act8_unpack(up8))
    if op == "gate_bwd":
        dgate, dup, a8 = muon.swiglu_act8_grad(s["da"], muon.Act8(*s["gate"]), muon.Act8(*s["up"]))
        return dict(dgate=dgate, dup=dup, a=muon.act8_unpack(a8))
    if op == "wgrad":
        x8 = muon.act8_pack(s["x"]) if c["pack"] else muon.Act8(s["codes"], s["scales"])
        if s["base"] is not None:
            dw = muon.act8_wgrad(s["dy"], x8, col_gain=s["gain"], out=s["base"].clone(), accumulate=True)
        else:
            dw = muon.act8_wgrad(s["dy"], x8, col_gain=s["gain"], dtype=TYPES[c["out"]])
        return dict(dw=dw)
    if op == "embed_fwd":
        return dict(out=muon.embed(s["table"], s["ids"], scale=s["scale"], dtype=TYPES[c["dtype"]]))
    return dict(grad=muon.embed_grad(s["dy"], s["ids"], c["vocab"], scale=s["scale"], dtype=TYPES[c["table"]]))


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------ work ----
def work(case):
    op, size = case["op"], {"f32": 4, "bf16": 2}
    if op.startswith(("norm", "gate")):
        rows, cols, b = case["rows"], case["cols"], size[case["dtype"]]
        el, e8 = rows * cols, rows * (cols + -(-cols // GROUP))
        if op == "norm_fwd":   # x (r) -> y (h), n8, rstd; then n8 -> its values
            return dict(bytes=(4 if case["residual"] else 2) * b * el + 2 * e8 + 2 * el + 4 * rows + 4 * cols, flops=8 * el)
        if op == "norm_bwd":   # dy (dres), n8, rstd -> dx; gain -> dgain
            return dict(bytes=(3 if case["residual"] else 2) * b * el + e8 + 4 * rows + 8 * cols, flops=10 * el)
        if op == "gate_fwd":   # gate, up -> a, gate8, up8; then their values
            return dict(bytes=3 * b * el + 4 * e8 + 4 * el, flops=12 * el)
        return dict(bytes=3 * b * el + 4 * e8 + 2 * el, flops=16 * el)  # da, gate8, up8 -> dgate, dup, a8; then a8's values
    if op == "wgrad":
        m, n, k, b = case["tokens"], case["n"], case["k"], size[case["out"]]
        x8 = m * (k + -(-k // GROUP))
        moved = 2 * m * n + x8 + b * n * k * (2 if case["add"] else 1) + (4 * k if case["gain"] else 0)
        return dict(bytes=moved + (2 * m * k + x8 if case["pack"] else 0), flops=2 * m * n * k)
    n, v, cols = case["tokens"], case["vocab"], case["cols"]
    ids = n * (4 if case["ids"] == "i32" else 8)
    used = int(n * (1.0 - case["ignored"]))
    if op == "embed_fwd":   # each row of the table that occurs is read once; rank r does with 1 - exp(-used / (r ln v))
        rank = torch.arange(1, v + 1, dtype=torch.float64)
        rows = float((1.0 - torch.exp(-used / (rank * math.log(v)))).sum())
        return dict(bytes=ids + rows * cols * size[case["table"]] + n * cols * size[case["dtype"]], flops=n * cols)
    return dict(bytes=ids + used * cols * size[case["dtype"]] + v * cols * size[case["table"]], flops=used * cols)


# ------------------------------------------------------- in 64 bits, apart ----
def _values(pair):
    """What codes and scales stand for, from their bits."""
    codes, scales = pair
    b = codes.view(torch.uint8).to(torch.int64)
    exp, man = (b >> 3) & 15, (b & 7).double()
    v = torch.where(exp == 0, man * 2.0 ** -9, (8.0 + man) * torch.pow(2.0, (exp - 10).double()))
    v = torch.where(b >= 128, -v, v)
    group = torch.arange(codes.shape[1], device=codes.device) // GROUP
    return v * torch.pow(2.0, scales.double() - 127.0)[:, group]


def exact(case, seed):
    """The outputs of `run` in 64 bits.  In the place of 8-bit values: the values before their rounding, so that
    the error of those outputs is the 8-bit form's own."""
    s, op = prepare(case, seed), case["op"]
    if op == "norm_fwd":
        h = s["x"].double()
        if s["r"] is not None:
            h = h + s["r"].double()
        rstd = 1.0 / torch.sqrt(torch.linalg.vecdot(h, h) / case["cols"] + EPS)
        n = torch.einsum("ij,i->ij", h, rstd)
        out = dict(y=n * s["gain"].double(), n=n, rstd=rstd)
        return dict(out, h=h) if s["r"] is not None else out
    if op == "norm_bwd":
        # the Jacobian of n(h) in rows: rstd (I - n n^T / cols), applied to g * dy
        n, dy = _values((s["codes"], s["scales"])), s["dy"].double()
        gd = torch.einsum("ij,j->ij", dy, s["gain"].double())
        along = torch.einsum("ij,ij->i", gd, n) / case["cols"]
        dx = torch.einsum("i,ij->ij", s["rstd"].double(), gd - torch.einsum("i,ij->ij", along, n))
        if s["dres"] is not None:
            dx += s["dres"].double()
        return dict(dx=dx, dgain=torch.einsum("ij,ij->j", dy, n))
    if op == "gate_fwd":
        gate, up = s["gu"].double().chunk(2, dim=1)
        return dict(a=gate * torch.sigmoid(gate) * up, gate=gate, up=up)
    if op == "gate_bwd":
        gate, up, da = _values(s["gate"]), _values(s["up"]), s["da"].double()
        sig = torch.sigmoid(gate)
        return dict(dgate=da * up * sig * (1.0 + gate * torch.sigmoid(-gate)), dup=da * gate * sig, a=gate * sig * up)
    if op == "wgrad":
        x = _values(_pack(s["x"])) if case["pack"] else _values((s["codes"], s["scales"]))
        dw = torch.zeros(case["n"], case["k"], dtype=torch.float64, device=DEV)
        for at in range(0, case["tokens"], 4096):
            dw.addmm_(s["dy"][at:at + 4096].double().t().contiguous(), x[at:at + 4096])
        if s["gain"] is not None:
            dw *= s["gain"].double()
        return dict(dw=dw if s["base"] is None else dw + s["base"].double())
    ids, v = s["ids"].long(), case["vocab"]
    live = torch.nonzero((ids >= 0) & (ids < v)).flatten()
    if op == "embed_fwd":
        out = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device=DEV)
        out[live] = s["table"].double()[ids[live]] * s["scale"]
        return dict(out=out)
    # the tokens in the order of their ids, summed run by run
    grad = torch.zeros(v, case["cols"], dtype=torch.float64, device=DEV)
    order = live[torch.argsort(ids[live], stable=True)]
    keys, counts = torch.unique_consecutive(ids[order], return_counts=True)
    if len(order):
        grad[keys] = torch.segment_reduce(s["dy"].double()[order] * s["scale"], "sum", lengths=counts)
    return dict(grad=grad)
