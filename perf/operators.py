"""Cases of the microscaled (MX) operators around the routed-expert layer: what each computes,
in plain torch and through the library's entry points.

  norm          moe_rmsnorm: residual addition and RMS norm of every row, the normalised row in
                bf16 / fp32 and / or MXFP8 (E4M3 elements, one E8M0 scale per 32)
  combine_norm  moe_combine_rmsnorm: the same with the gate-weighted sum of the token's expert
                rows as what is added
  entry         moe_entry_quantize, then moe_entry_dequantize: whole (layer, expert) entries to
                MXFP4 and back
  ffn           moe_expert_ffn with MXFP8 activations and MXFP4 weights: the SwiGLU expert FFNs
                over the grouped rows, the intermediate in MXFP8 too

MXFP8 and MXFP4 results are returned as the values they stand for, in bf16 (which holds every
such value exactly).  The FFN's rows are returned in bf16: its intermediate is rounded to E4M3,
and sums taken in another order move a few of its elements by one E4M3 step.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


def listed():
    decode = {"op": "ffn", "E": 256, "k": 6, "d": 4096, "f": 2048, "alpha": 0.2}
    return [
        # one sequence's decode step: the norm in front of the router and the experts
        {"name": "norm_one_token", "op": "norm", "T": 1, "d": 4096, "x": "bf16", "delta": "f32",
         "gamma": "bf16", "y": "bf16", "mx8": True},
        # the same in front of a prefill's experts, which take MXFP8 rows only
        {"name": "norm_prefill", "op": "norm", "T": 8192, "d": 4096, "x": "bf16", "delta": "bf16",
         "gamma": "bf16", "y": "none", "mx8": True},
        # an fp32 residual stream of a width that is no power of two, no addition
        {"name": "norm_f32_odd", "op": "norm", "T": 1021, "d": 2112, "x": "f32", "delta": "none",
         "gamma": "f32", "y": "f32", "mx8": False},
        # end of a decode layer: combine, residual, the next norm
        {"name": "combine_norm_decode", "op": "combine_norm", "T": 8, "k": 6, "d": 4096, "yp": "f32",
         "x": "bf16", "gamma": "bf16", "y": "bf16", "mx8": True},
        # end of a prefill layer
        {"name": "combine_norm_prefill", "op": "combine_norm", "T": 8192, "k": 6, "d": 4096,
         "yp": "bf16", "x": "bf16", "gamma": "bf16", "y": "bf16", "mx8": False},
        # one small fp32 entry whose rows end inside a 128-element tile
        {"name": "entry_small", "op": "entry", "n": 1, "d": 320, "f": 192, "src": "f32"},
        # a load-time batch: 32 of a layer's 256 experts
        {"name": "entry_batch", "op": "entry", "n": 32, "d": 4096, "f": 2048, "src": "bf16"},
        # decode of one sequence, of a small batch and of a large one
        dict(decode, name="ffn_one_token", T=1),
        dict(decode, name="ffn_decode", T=8),
        dict(decode, name="ffn_decode_64", T=64),
        # a ragged chunk of a prompt on the smaller layer (128 experts, 8 a token)
        {"name": "ffn_chunk", "op": "ffn", "T": 333, "E": 128, "k": 8, "d": 2048, "f": 768, "alpha": 1.0},
        # prefill
        dict(decode, name="ffn_prefill", T=8192),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "combine_norm", "entry", "ffn", "ffn"])
    if op == "norm":
        y = rng.choice(["none", "bf16", "f32"])
        return {"op": op, "T": _log(rng, 1, 8192), "d": 64 * _log(rng, 1, 128), "x": rng.choice(["bf16", "f32"]),
                "delta": rng.choice(["none", "bf16", "f32"]), "gamma": rng.choice(["bf16", "f32"]), "y": y,
                "mx8": y == "none" or rng.random() < 0.5}
    if op == "combine_norm":
        y = rng.choice(["none", "bf16", "f32"])
        return {"op": op, "T": _log(rng, 1, 4096), "k": rng.randint(1, 8), "d": 64 * _log(rng, 1, 64),
                "yp": rng.choice(["bf16", "f32"]), "x": rng.choice(["bf16", "f32"]), "gamma": rng.choice(["bf16", "f32"]),
                "y": y, "mx8": y == "none" or rng.random() < 0.5}
    if op == "entry":
        return {"op": op, "n": _log(rng, 1, 32), "d": 64 * _log(rng, 1, 64), "f": 64 * _log(rng, 1, 32),
                "src": rng.choice(["bf16", "f32"])}
    E = rng.choice([8, 24, 64, 128, 200, 256])
    return {"op": op, "T": _log(rng, 1, 4096), "E": E, "k": rng.randint(1, 8), "d": 64 * _log(rng, 4, 64),
            "f": 64 * _log(rng, 2, 32), "alpha": rng.choice([0.2, 0.5, 1.0])}


# ---------------------------------------------------------------- inputs
def _quantise_mxfp8(v):
    """MXFP8 rows of v [rows, d] as one byte buffer: codes [rows, d], then the rows' d/32 scales, each
    row of them filled up to a multiple of 4 bytes."""
    rows, d = v.shape
    b = v.float().reshape(rows, d // 32, 32)
    s = (((b.abs().amax(2).view(torch.int32) >> 23) & 255) - 8).clamp_min(0)
    q = (b * torch.exp2((127 - s).double()).float()[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = torch.nn.functional.pad(s.to(torch.uint8), (0, -(d // 32) % 4))
    return torch.cat([q.view(torch.uint8).reshape(-1), s.reshape(-1)])


def _random_entries(n, d, f, g):
    """n MXFP4 entries of N(0, 1/d) weights: codes of gate, up and down, then their scales; each
    matrix in strips of 16 rows, the 32-element blocks of a strip in order, row by row inside."""
    out = torch.empty((n, 3 * d * f * 17 // 32), dtype=torch.uint8, device="cuda")
    chunk = max(1, (1 << 28) // (3 * d * f))
    for i in range(0, n, chunk):
        m = min(chunk, n - i)
        parts = []
        for R, K in ((f, d), (f, d), (d, f)):
            v = torch.randn((m, R // 16, 16, K // 32, 32), device="cuda", generator=g).mul_(d ** -0.5).transpose(2, 3)
            s = (((v.abs().amax(-1).view(torch.int32) >> 23) & 255) - 2).clamp_min(0)
            a = v * torch.exp2((127 - s).double()).float()[..., None]
            c = (v < 0).to(torch.uint8) * 8
            for edge in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
                c += a.abs() > edge
            parts.append(((c[..., 0::2] | (c[..., 1::2] << 4)).reshape(m, -1), s.to(torch.uint8).reshape(m, -1)))
        out[i:i + m] = torch.cat([p[0] for p in parts] + [p[1] for p in parts], 1)
    return out


def _grouped(T, E, k, alpha, g):
    """Top-k routing of N(0, 1) logits with a Zipf(1.1) bias of strength alpha, grouped by expert."""
    rank = torch.randperm(E, device="cuda", generator=g) + 1
    logits = torch.randn((T, E), device="cuda", generator=g) - alpha * 1.1 * rank.float().log()
    top = logits.topk(k, dim=1)
    ids = top.indices.reshape(-1)
    perm = torch.sort(ids, stable=True).indices
    counts = torch.bincount(ids, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k, device="cuda")
    return dict(ids=ids, w=top.values.softmax(1), perm=perm.int(), inv=inv.int(), offsets=offsets.int(),
                most=int(counts.max()))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, device="cuda", generator=g)  # noqa: E731
    st = {"case": case}
    op, d = case["op"], case["d"]
    if op in ("norm", "combine_norm"):
        T = case["T"]
        # a residual stream has grown to a few units and has some rows and columns far above the rest
        st["x"] = (3 * randn(T, d) * (0.5 + randn(T, 1).abs()) * (1 + 4 * (randn(1, d) > 2.5))).to(TORCH[case["x"]])
        st["gamma"] = (1 + 0.2 * randn(d)).to(TORCH[case["gamma"]])
        if op == "norm":
            if case["delta"] != "none":
                st["delta"] = randn(T, d).to(TORCH[case["delta"]])
        else:
            st.update(_grouped(T, 256, case["k"], 0.2, g))
            st["yp"] = randn(T * case["k"], d).to(TORCH[case["yp"]])
    elif op == "entry":
        st["src"] = torch.empty((case["n"], 3 * d * case["f"]), dtype=TORCH[case["src"]], device="cuda")
        for row in st["src"]:
            row.copy_(randn(row.numel()).mul_(d ** -0.5))
    else:
        T, E, f = case["T"], case["E"], case["f"]
        st.update(_grouped(T, E, case["k"], case["alpha"], g))
        st["x8"] = _quantise_mxfp8(randn(T, d))
        st["arena"] = _random_entries(E, d, f, g)
    return st


# ---------------------------------------------------------------- the plain forms
def _rounded(a, least, mantissa):
    """a to the nearest value with `mantissa` fraction bits, ties to even, exponents from `least` on."""
    step = torch.exp2((torch.frexp(a).exponent - 1).clamp_min(least).float() - mantissa)
    return torch.round(a / step) * step


def _mx(v, emax, least, mantissa, most):
    """v [..., n * 32] as the values that its microscaled blocks stand for."""
    b = v.reshape(-1, 32)
    e = (torch.frexp(b.abs().amax(1)).exponent - 1 - emax).clamp_min(-127)
    x = torch.exp2(e.float())[:, None]
    return (_rounded(b / x, least, mantissa).clamp(-most, most) * x).reshape(v.shape)


def _mxfp8(v):
    return _mx(v, 8, -6, 3, 448.0)


def _mxfp4(v):
    return _mx(v, 2, 0, 1, 6.0)


def _rows_of(x8, rows, d):
    q = x8[:rows * d].view(torch.float8_e4m3fn).float().reshape(rows, d // 32, 32)
    s = torch.exp2(x8[rows * d:].float() - 127).reshape(rows, -1, 1)[:, :d // 32]
    return (q * s).reshape(rows, d)


def _matrix_of(entries, part, R, K):
    """Matrix `part` (0 gate, 1 up, 2 down) of each entry in fp32, [n, R, K]."""
    n, fd = entries.shape[0], R * K
    c = entries[:, part * fd // 2:(part + 1) * fd // 2]
    s = entries[:, 3 * fd // 2 + part * fd // 32:3 * fd // 2 + (part + 1) * fd // 32]
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=c.device)
    v = torch.stack([table[(c & 15).int()], table[(c >> 4).int()]], -1).reshape(n, R // 16, K // 32, 16, 32)
    v = v * torch.exp2(s.float() - 127).reshape(n, R // 16, K // 32, 16, 1)
    return v.transpose(2, 3).reshape(n, R, K)


def _plain_norm(st, case, add):
    x = st["x"].float()
    s = (x if add is None else x + add).to(st["x"].dtype)
    v = s.float()
    y = v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS) * st["gamma"].float()
    return {"residual": None if add is None else s, "y": None if case["y"] == "none" else y.to(TORCH[case["y"]]),
            "y8": _mxfp8(y).bfloat16() if case["mx8"] else None}


def _plain_ffn(st, case):
    T, E, k, d, f = (case[n] for n in ("T", "E", "k", "d", "f"))
    x = _rows_of(st["x8"], T, d)
    perm = st["perm"].long()
    if T * k <= E:  # few rows: each takes its expert's weights
        entries = st["arena"][st["ids"][perm]]
        rows = x[perm // k][:, None]
    else:  # many: each expert takes its rows, padded to the most that one has
        entries, offsets = st["arena"], st["offsets"].long()
        at = offsets[:-1, None] + torch.arange(st["most"], device=x.device)
        real = at < offsets[1:, None]
        rows = x[perm[at.clamp_max(T * k - 1)] // k]
    g = torch.bmm(rows, _matrix_of(entries, 0, f, d).transpose(1, 2))
    u = torch.bmm(rows, _matrix_of(entries, 1, f, d).transpose(1, 2))
    h = _mxfp8(g / (1 + torch.exp(-g)) * u)
    y = torch.bmm(h, _matrix_of(entries, 2, d, f).transpose(1, 2)).bfloat16()
    return y[:, 0] if T * k <= E else y[real]


def _plain(st):
    case = st["case"]
    if case["op"] == "norm":
        return _plain_norm(st, case, st["delta"].float() if "delta" in st else None)
    if case["op"] == "combine_norm":
        rows = st["yp"][st["inv"].long()].float().reshape(case["T"], case["k"], case["d"])
        return _plain_norm(st, case, (rows * st["w"][..., None]).sum(1))
    if case["op"] == "entry":
        return _mxfp4(st["src"].float()).to(st["src"].dtype)
    return _plain_ffn(st, case)


# ---------------------------------------------------------------- the library's calls
def _plan(moe, st):
    """The buffers that a program keeps for these calls."""
    case = st["case"]
    op, d = case["op"], case["d"]
    code = {"f32": moe.MOE_F32, "bf16": moe.MOE_BF16, "none": moe.MOE_BF16}
    new = lambda dtype, *shape: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    if op == "entry":
        eb = moe.moe_entry_bytes(d, case["f"], moe.MOE_MXFP4)
        return dict(src=code[case["src"]], eb=eb, mx=new(torch.uint8, case["n"], eb), out=torch.empty_like(st["src"]))
    T = case["T"]
    if op == "ffn":
        nws = moe.moe_expert_ffn_workspace_bytes(T, case["k"], case["f"], moe.MOE_MXFP8)
        return dict(nws=nws, ws=new(torch.uint8, nws), y=new(torch.bfloat16, T * case["k"], d),
                    eb=moe.moe_entry_bytes(d, case["f"], moe.MOE_MXFP4), status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    p = dict(x=code[case["x"]], gamma=code[case["gamma"]], y=code[case["y"]], add=code[case.get("delta", case.get("yp"))],
             residual=None, out=None, x8=None, values=None)
    if case.get("delta") != "none":
        p["residual"] = torch.empty_like(st["x"])
    if case["y"] != "none":
        p["out"] = new(TORCH[case["y"]], T, d)
    if case["mx8"]:
        p["x8"], p["values"] = new(torch.uint8, moe.moe_mxfp8_bytes(T, d)), new(torch.bfloat16, T, d)
    return p


def _calls(st):
    import expert_ffn_cache_amd as moe
    case = st["case"]
    p = st.get("plan") or st.setdefault("plan", _plan(moe, st))
    op, d = case["op"], case["d"]
    if op == "entry":
        n, f, elem = case["n"], case["f"], st["src"].element_size()
        moe.moe_entry_quantize(st["src"], p["src"], 3 * d * f * elem, n, d, f, p["mx"], p["eb"])
        moe.moe_entry_dequantize(p["mx"], p["eb"], n, d, f, p["out"], p["src"], 3 * d * f * elem)
        return p["out"]
    T = case["T"]
    if op == "ffn":
        moe.moe_expert_ffn(st["x8"], moe.MOE_MXFP8, st["perm"], st["offsets"], T, case["k"], case["E"], d, case["f"], None,
                           st["arena"], p["eb"], moe.MOE_MXFP4, None, None, 0, p["ws"], p["nws"], p["y"], moe.MOE_BF16,
                           moe.MOE_PATH_AUTO, p["status"])
        return p["y"]
    if op == "norm":
        moe.moe_rmsnorm(st["x"], p["x"], st.get("delta"), p["add"], st["gamma"], p["gamma"], EPS, T, d, p["residual"], p["out"],
                        p["y"], p["x8"])
    else:
        moe.moe_combine_rmsnorm(st["yp"], p["add"], st["inv"], st["w"], case["k"], st["x"], p["x"], st["gamma"], p["gamma"], EPS,
                                T, d, p["residual"], p["out"], p["y"], p["x8"])
    if case["mx8"]:
        moe.moe_mxfp8_dequantize(p["x8"], T, d, p["values"], moe.MOE_BF16)
    return {"residual": p["residual"], "y": p["out"], "y8": p["values"]}


def run(state):
    return _calls(state) if own else _plain(state)


def work(case):
    size = {"f32": 4, "bf16": 2, "none": 0}
    op, d = case["op"], case["d"]
    if op == "entry":
        e = case["n"] * 3 * d * case["f"]
        return {"bytes": e * (2 * size[case["src"]] + 17 / 32), "flops": 4 * e}
    T = case["T"]
    if op == "ffn":
        E, k, f = case["E"], case["k"], case["f"]
        used = E * (1 - (1 - k / E) ** T)  # experts that some token picks, were all as likely
        return {"bytes": used * 3 * d * f * 17 / 32 + T * d * 33 / 32 + T * k * d * 2 + 4 * (T * k + E + 1),
                "flops": 6 * T * k * d * f}
    out = size[case["y"]] + (2 if case["mx8"] else 0)
    if op == "norm":
        add = size[case["delta"]]
        return {"bytes": T * d * (size[case["x"]] * (2 if add else 1) + add + out) + d * size[case["gamma"]], "flops": 6 * T * d}
    k = case["k"]
    return {"bytes": T * d * (2 * size[case["x"]] + k * size[case["yp"]] + out) + d * size[case["gamma"]] + 8 * T * k,
            "flops": (2 * k + 6) * T * d}


# ---------------------------------------------------------------- the definitions in 64 bits
def _nearest(v, grid):
    """Each of v (float64, its magnitude at most the grid's last) at the nearest grid value; a tie
    goes to the even index."""
    grid = torch.tensor(grid, dtype=torch.float64, device=v.device)
    a = v.abs().clamp_max(float(grid[-1])).contiguous()
    lo = (torch.bucketize(a, grid, right=True, out_int32=True) - 1).clamp_max(len(grid) - 2)
    below, above = a - grid[lo], grid[lo + 1] - a
    lo = lo + ((above < below) | ((above == below) & (lo % 2 == 1))).int()
    return torch.copysign(grid[lo], v)


def _exact_mx(v, grid):
    """Blocks of 32 of v (float64): scale 2^(floor(log2 of the largest) - the grid's largest exponent)."""
    b = v.reshape(-1, 32)
    top = b.abs().amax(1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
    e = e + (torch.exp2(e + 1) <= top).double() - (torch.exp2(e) > top).double()
    x = torch.exp2(torch.where(top > 0, e - math.floor(math.log2(grid[-1])), torch.full_like(e, -127.0)).clamp_min(-127))
    return (_nearest(b / x, grid) * x).reshape(v.shape)


E4M3 = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]


def exact(case, seed):
    st = prepare(case, seed)
    op, d = case["op"], case["d"]
    if op == "entry":
        return torch.stack([_exact_mx(row.double(), list(E2M1)).to(st["src"].dtype) for row in st["src"]])
    T = case["T"]
    if op != "ffn":
        s = st["x"].double()
        add = None
        if op == "norm" and "delta" in st:
            add = st["delta"].double()
        elif op == "combine_norm":
            add = torch.zeros_like(s)
            for j in range(case["k"]):
                add += st["w"][:, j:j + 1].double() * st["yp"][st["inv"].view(T, -1)[:, j].long()].double()
        if add is not None:
            s = (s + add).to(st["x"].dtype).double()
        y = s / torch.sqrt((s * s).sum(1, keepdim=True) / d + EPS) * st["gamma"].double()
        return {"residual": s if add is not None else None, "y": y if case["y"] != "none" else None,
                "y8": _exact_mx(y, E4M3) if case["mx8"] else None}
    k, f = case["k"], case["f"]
    x = st["x8"][:T * d].view(torch.float8_e4m3fn).double().view(T, d)
    x = x * torch.exp2(st["x8"][T * d:].double().view(T, -1)[:, :d // 32] - 127).repeat_interleave(32, 1)
    values = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")
    at, y = st["offsets"].tolist(), torch.empty((T * k, d), dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        if at[e] == at[e + 1]:
            continue
        entry, co, so, mats = st["arena"][e], 0, 3 * d * f // 2, []
        for R, K in ((f, d), (f, d), (d, f)):
            c, s = entry[co:co + R * K // 2], entry[so:so + R * K // 32]
            co, so = co + R * K // 2, so + R * K // 32
            w = torch.empty((R * K // 32, 32), dtype=torch.float64, device="cuda")
            w[:, 0::2], w[:, 1::2] = values[(c & 15).int()].view(-1, 16), values[(c >> 4).int()].view(-1, 16)
            w *= torch.exp2(s.double() - 127)[:, None]
            mats.append(w.view(R // 16, K // 32, 16, 32).permute(0, 2, 1, 3).reshape(R, K))
        rows = x[st["perm"][at[e]:at[e + 1]].long() // k]
        gate, up = rows @ mats[0].t(), rows @ mats[1].t()
        y[at[e]:at[e + 1]] = _exact_mx(gate * torch.sigmoid(gate) * up, E4M3) @ mats[2].t()
    return y
