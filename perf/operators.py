"""The operators of the 8-bit block-scaled path, as cases to measure: the e4m3
matrix product with a scale for each block of 128, the root-mean-square norm
with the residual's addition and an e4m3 output, and the quantiser of
activations.

``run`` computes a case in elementary torch operations in 32 bits, or, with
``own`` set, through the public entry points of the package.

Formulas (G = ceil(K / 128) groups of 128 columns, the last may be short):
  quantise   a = max |x| over a group, raised to 2^-100 if it is smaller and
             not 0;  scale = a / 448;  code = e4m3(x * (448 / a)), 0 for a = 0
  rms norm   h = round16(x + residual);  y = h / sqrt(mean(h^2) + eps) * weight;
             codes and scales of y as above, and y in 16 bits where asked for
  product    Y[m, n] = sum_g sx[m, g] sw[n / 128, g] sum_{k in g} xq[m, k] wq[n, k]
             (+ bias[n]), rounded once to 16 bits
"""
import torch

own = False

GROUP = 128
E4M3_MAX = 448.0
TINY = 2.0 ** -100
EPS = 1e-5
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _matmul(name, M, K, N, dtype, bias=False, acts="codes"):
    return {"name": name, "op": "matmul", "M": M, "K": K, "N": N, "dtype": dtype, "bias": bias, "acts": acts}


def _norm(name, M, K, dtype, residual=True, normed=False):
    return {"name": name, "op": "norm", "M": M, "K": K, "dtype": dtype, "residual": residual, "normed": normed}


def _quantise(name, M, K, dtype):
    return {"name": name, "op": "quantise", "M": M, "K": K, "dtype": dtype}


def listed():
    return [
        # one new token against the largest feed-forward expansion: a decode step's weight stream
        _matmul("token 12288 to 49152", 1, 12288, 49152, "fp16"),
        # a batch of 32 sequences, one token each, in a square projection
        _matmul("32 tokens 8192 square", 32, 8192, 8192, "bf16"),
        # 16 tokens in 16 bits, as a layer gets them where no norm stands before it (an output projection)
        _matmul("16 tokens 8192, 16-bit in", 16, 8192, 8192, "fp16", acts="16 bits"),
        # odd sizes: a short prompt in a small model, with the layer's bias
        _matmul("37 by 1040 by 784, bias", 37, 1040, 784, "fp16", bias=True),
        # a chunk of a prompt, between decode and prefill
        _matmul("chunk 384, 5120 to 20480", 384, 5120, 20480, "bf16"),
        # the feed-forward contraction of a 13B-sized model on a prompt of 2048
        _matmul("prompt 20480 to 5120", 2048, 20480, 5120, "bf16"),
        # the largest: the expansion of a 175B-sized model on the same prompt
        _matmul("prompt 12288 to 49152", 2048, 12288, 49152, "fp16"),
        # before a layer's projections: one token, and a prompt
        _norm("norm of a token, 12288", 1, 12288, "bf16"),
        _norm("norm of a prompt, 12288", 2048, 12288, "fp16"),
        # odd sizes, the first norm of a model (no residual yet), its 16-bit output wanted too
        _norm("norm 513 by 1040, 16-bit too", 513, 1040, "bf16", residual=False, normed=True),
        # activations between two feed-forward products: a decode step's and a prompt's
        _quantise("quantise 8 by 20480", 8, 20480, "fp16"),
        _quantise("quantise prompt, 20480", 2048, 20480, "bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _multiple_of_16(rng, lo, hi):
    return 16 * max(1, round(_log_uniform(rng, lo, hi) / 16))


def draw(rng):
    op = rng.choice(["matmul"] * 6 + ["norm"] * 3 + ["quantise"] * 2)
    M = _log_uniform(rng, 1, 2048)
    K = _multiple_of_16(rng, 256, 20480)
    dtype = rng.choice(["fp16", "bf16"])
    if op == "matmul":
        N = _multiple_of_16(rng, 256, 49152)
        while M * K * N > 2048 * 12288 * 49152 or K * N > 12288 * 49152:
            N = max(16, N // 32 * 16)
        c = _matmul("", M, K, N, dtype, rng.random() < 0.5, rng.choice(["codes", "codes", "16 bits"]))
    elif op == "norm":
        c = _norm("", M, K, dtype, rng.random() < 0.7, rng.random() < 0.4)
    else:
        c = _quantise("", M, K, dtype)
    del c["name"]
    return c


def _groups(K):
    return -(-K // GROUP)


def _group_amax(x):
    """max |x| over each group of 128 columns of the rows of x [M, K] (fp32 or fp64)."""
    M, K = x.shape
    G = _groups(K)
    x = torch.nn.functional.pad(x.abs(), (0, G * GROUP - K))
    return x.view(M, G, GROUP).amax(-1)


def _spread(s, K):
    """One value per group to one value per column."""
    return s.repeat_interleave(GROUP, dim=1)[:, :K]


def _quantise_rows(x):
    """Codes and scales of the rows of x, fp32."""
    a = _group_amax(x)
    a = torch.where(a == 0, a, a.clamp(min=TINY))
    r = torch.where(a == 0, a, torch.full_like(a, E4M3_MAX) / a)  # number / tensor would round twice
    return (x * _spread(r, x.shape[1])).to(torch.float8_e4m3fn), a / E4M3_MAX


def _activations(M, K, dtype, g):
    """Activations as a layer's input has them: ordinary channels of mean |x|
    0.5, and 7 channels a hundred times larger in three rows of four."""
    x = torch.randn(M, K, generator=g, device="cuda").mul_(0.627).clamp_(-5.5, 5.5)
    cols = torch.randperm(K, generator=g, device="cuda")[:7]
    big = torch.rand(M, 7, generator=g, device="cuda") * 130
    keep = torch.rand(M, 7, generator=g, device="cuda") < 0.75
    x[:, cols] = torch.where(keep, big * torch.sign(x[:, cols]), x[:, cols])
    return x.to(dtype)


def _column_major(s):
    """The scales' layout of the package: [M, G] values, each group's M
    contiguous, groups a multiple of 4 apart."""
    M, G = s.shape
    t = torch.zeros(G, -(-M // 4) * 4, dtype=s.dtype, device=s.device)
    t[:, :M] = s.t()
    return t.t()[:M]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    M, K = case["M"], case["K"]
    st = {"case": case, "dtype": dtype, "x": _activations(M, K, dtype, g)}
    if case["op"] == "matmul":
        N, G, NB = case["N"], _groups(K), _groups(case["N"])
        # a weight as a checkpoint holds it: e4m3 codes [N, K], one scale for
        # each 128 x 128 block
        w = torch.randn(N, K, generator=g, device="cuda").mul_(0.02)
        a = _group_amax(_group_amax(w).t().contiguous()).t().clamp_(min=TINY)
        st["w_scales"] = (a / E4M3_MAX).contiguous()
        w /= _spread(st["w_scales"], K).repeat_interleave(GROUP, dim=0)[:N]
        st["w_codes"] = w.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        del w
        assert st["w_scales"].shape == (NB, G)
        st["bias"] = torch.randn(N, generator=g, device="cuda").mul_(0.1).to(dtype) if case["bias"] else None
        if case["acts"] == "codes":
            st["codes"], s = _quantise_rows(st.pop("x").float())
            st["scales"] = _column_major(s)
        if own:
            import int8_quantized_matmul_outlier_b200 as m

            st["m"] = m
            st["w"] = m.int8mm_block_prepare_codes(st["w_codes"], st["w_scales"])
    else:
        if case["op"] == "norm":
            st["weight"] = (1 + 0.2 * torch.randn(K, generator=g, device="cuda")).to(dtype)
            # the residual stream grows with depth: wider than a layer's output
            st["residual"] = (2 * torch.randn(M, K, generator=g, device="cuda")).to(dtype) if case["residual"] else None
        if own:
            import int8_quantized_matmul_outlier_b200 as m

            st["m"] = m
    return st


def run(st):
    case = st["case"]
    if own:
        m = st["m"]
        if case["op"] == "quantise":
            return m.int8mm_block_quantize(st["x"])
        if case["op"] == "norm":
            return m.int8mm_block_rms_norm(st["x"], st["weight"], EPS, residual=st["residual"], normed=case["normed"])
        if case["acts"] == "codes":
            return m.int8mm_block_matmul(st["w"], st["codes"], st["scales"], bias=st["bias"], dtype=st["dtype"])
        return m.int8mm_block_forward(st["w"], st["x"], bias=st["bias"])
    if case["op"] == "quantise":
        return _quantise_rows(st["x"].float())
    if case["op"] == "norm":
        h, out = st["x"], None
        if st["residual"] is not None:
            h = out = (h.float() + st["residual"].float()).to(st["dtype"])
        h = h.float()
        y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * st["weight"].float()
        codes, scales = _quantise_rows(y)
        return codes, scales, out, y.to(st["dtype"]) if case["normed"] else None
    if case["acts"] == "codes":
        codes, s = st["codes"], st["scales"]
    else:
        codes, s = _quantise_rows(st["x"].float())
    K, N = case["K"], case["N"]
    x = codes.float() * _spread(s, K)
    w = st["w_codes"].float() * _spread(st["w_scales"], K).repeat_interleave(GROUP, dim=0)[:N]
    y = x @ w.t()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    return y.to(st["dtype"])


def work(case):
    """Each input read once, each output written once; 2 M N K for a product."""
    M, K = case["M"], case["K"]
    G = _groups(K)
    codes = M * K + 4 * M * G
    if case["op"] == "quantise":
        return {"bytes": 2 * M * K + codes, "flops": 3 * M * K}
    if case["op"] == "norm":
        sixteen = 1 + 2 * case["residual"] + case["normed"]
        return {"bytes": 2 * M * K * sixteen + 2 * K + codes, "flops": 8 * M * K}
    N = case["N"]
    acts = codes if case["acts"] == "codes" else 2 * M * K
    return {"bytes": acts + N * K + 4 * _groups(N) * G + 2 * M * N + 2 * N * case["bias"], "flops": 2 * M * N * K}


def _exact_quantised(y):
    """(the values that the codes stand for before their rounding to 8 bits,
    the scales) of y, fp64."""
    M, K = y.shape
    top = torch.zeros(M, _groups(K), dtype=torch.float64, device=y.device)
    for g in range(_groups(K)):
        top[:, g] = y[:, g * GROUP:(g + 1) * GROUP].abs().max(1).values
    top = torch.where(top > 0, top.clamp(min=TINY), top)
    unit = torch.where(top > 0, E4M3_MAX / top, top)
    group = torch.arange(K, device=y.device) // GROUP
    return y * unit[:, group], top / E4M3_MAX


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quantise":
        return _exact_quantised(st["x"].double())
    if case["op"] == "norm":
        h, out = st["x"].double(), None
        if st["residual"] is not None:
            out = h + st["residual"].double()
            h = out.to(st["dtype"]).double()  # the norm is of what the residual stream holds
        y = h * (h.square().sum(1, keepdim=True) / case["K"] + EPS).rsqrt() * st["weight"].double()
        return (*_exact_quantised(y), out, y if case["normed"] else None)
    if case["acts"] == "codes":
        codes, s = st["codes"].double(), st["scales"].double()
    else:  # the codes are rounded by definition: in 32 bits, as it says
        a = torch.stack([c.abs().max(1).values for c in st["x"].float().split(GROUP, dim=1)], 1)
        a = torch.where(a > 0, a.clamp(min=TINY), a)
        r = torch.where(a > 0, torch.full_like(a, E4M3_MAX) / a, a)
        group = torch.arange(case["K"], device="cuda") // GROUP
        codes, s = (st["x"].float() * r[:, group]).to(torch.float8_e4m3fn).double(), a.double() / E4M3_MAX
    y = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
    ws = st["w_scales"].double().repeat_interleave(GROUP, dim=0)[:case["N"]]
    for g in range(_groups(case["K"])):
        k = slice(g * GROUP, (g + 1) * GROUP)
        y += (codes[:, k] * s[:, g:g + 1]) @ (st["w_codes"][:, k].double() * ws[:, g:g + 1]).t()
    return y if st["bias"] is None else y + st["bias"].double()
