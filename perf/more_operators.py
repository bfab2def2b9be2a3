"""Performance cases of further operators of a layer around the short
convolution: the gated delta rule (prefill, training step, decode step), the
layer norm (forward, training step), and the block tables and slot maps of a
paged cache.

With ``own`` false, ``run`` computes an operator from elementary torch
operations; with ``own`` true it calls the library.  Both take the tensors
that ``prepare`` makes.  ``exact`` computes the same outputs from the
definitions in 64 bits.

Formulas:

    delta rule  per value head h and token t of one sequence, S a K x V matrix:
                S' = exp(g_t) S,  u = beta_t (v_t - S'^T k_t),
                S = S' + k_t u^T,  out_t = scale S^T q_t
                (q and k belong to key head h // (value heads / key heads))
    layer norm  s = x + residual, n = (s - mean(s)) / sqrt(var(s) + eps),
                out = n * weight + bias
    metadata    request r brings query_lens[r] tokens after context_lens[r]
                earlier ones; blocks that its table lacks come from the free
                list, in the order of the requests; slot = block * size + offset
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "bf16": 2}
EPS = 1e-5
PAD = -1
CHUNK = 64  # tokens of the plain form's chunks

if torch.cuda.is_available():
    DEVICE = "cuda"
else:
    DEVICE = "cpu"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One decode step of a small batch: the call's latency is the cost.
        dict(name="delta update 4x16x64", op="delta_update", rows=4, pads=0, slots=64, kh=8, vh=16,
             dk=64, dv=64, dtype="bf16", gates="f32"),
        # A decode step of a large batch with padded rows: bytes of the states.
        dict(name="delta update 256x32x128", op="delta_update", rows=256, pads=9, slots=300, kh=16,
             vh=32, dk=128, dv=128, dtype="bf16", gates="f32"),
        # Prefill of eight equal prompts, two value heads a key head.
        dict(name="delta prefill 8x4096x32", op="delta_prefill", total=32768, seqs=8, ragged=False,
             kh=16, vh=32, dk=128, dv=128, slots=64, inits=4, pads=0, dtype="bf16", gates="f32"),
        # A mixed batch of ragged prompts, some that continue from a state, one
        # padded sequence, odd head sizes, 32-bit.
        dict(name="delta prefill 16 ragged f32", op="delta_prefill", total=9001, seqs=16,
             ragged=True, kh=5, vh=5, dk=96, dv=77, slots=40, inits=8, pads=1, dtype="f32",
             gates="f32"),
        # Training on long documents: forward and gradients.
        dict(name="delta train 2x8192x16", op="delta_train", total=16384, seqs=2, ragged=False,
             kh=16, vh=16, dk=128, dv=128, inits=0, dtype="bf16", gates="f32"),
        # Training on packed short documents with states carried over (their
        # gradients too), three value heads a key head, odd sizes, 32-bit.
        dict(name="delta train 12 ragged f32", op="delta_train", total=3001, seqs=12, ragged=True,
             kh=2, vh=6, dk=64, dv=72, inits=7, dtype="f32", gates="f32"),
        # The norm before a layer in a decode step.
        dict(name="layer norm 256x1024", op="norm", rows=256, dim=1024, dtype="bf16"),
        # A training step's norm, forward and gradients.
        dict(name="layer norm train 32768x4096", op="norm_train", rows=32768, dim=4096,
             dtype="bf16"),
        # The same on few rows of an odd width.
        dict(name="layer norm train 1023x1001 f32", op="norm_train", rows=1023, dim=1001,
             dtype="f32"),
        # The metadata of a decode step: one token a request.
        dict(name="metadata 256 decode", op="metadata", requests=256, tokens=256, padded=256,
             context=16384, block_size=16),
        # A mixed step: a few prompts among decoding requests, rows padded.
        dict(name="metadata 64 mixed", op="metadata", requests=64, tokens=16384, padded=17000,
             context=8192, block_size=16),
        # A large offline batch with odd blocks.
        dict(name="metadata 1000 offline", op="metadata", requests=1000, tokens=65536,
             padded=65536, context=4001, block_size=24),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta_update", "delta_prefill", "delta_train", "norm", "norm_train",
                     "metadata"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "metadata":
        requests = _log_int(rng, 1, 1024)
        tokens = requests * _log_int(rng, 1, 65536 // requests)
        return dict(op=op, requests=requests, tokens=tokens, padded=tokens + rng.randint(0, 512),
                    context=_log_int(rng, 1, 16384), block_size=rng.choice([8, 16, 24, 32, 64]))
    if op in ("norm", "norm_train"):
        rows, dim = _log_int(rng, 1, 32768), _log_int(rng, 64, 8192)
        return dict(op=op, rows=min(rows, (1 << 27) // dim), dim=dim, dtype=dtype)
    group, kh = rng.choice([1, 1, 2, 3, 4]), rng.randint(1, 8)
    case = dict(op=op, kh=kh, vh=group * kh, dk=rng.choice([64, 128, rng.randint(16, 128)]),
                dv=rng.choice([64, 128, rng.randint(16, 256)]), dtype=dtype,
                gates=rng.choice(["f32", dtype]))
    if op == "delta_update":
        rows = _log_int(rng, 1, 256)
        return case | dict(rows=rows, pads=rng.randint(0, rows // 4), slots=rows + rng.randint(0, 64))
    # a 32-bit product is dear, and so are gradients
    most = 32768 * 32 // (16 if dtype == "f32" else 2) // (2 if op == "delta_train" else 1)
    total = _log_int(rng, 1, min(16384, most // case["vh"]))
    seqs = _log_int(rng, 1, 32)
    case |= dict(total=total, seqs=seqs, ragged=True, inits=rng.randint(0, seqs))
    if op == "delta_prefill":
        case |= dict(slots=seqs + rng.randint(0, 16), pads=rng.randint(0, seqs // 4))
    return case


def work(case):
    op = case["op"]
    if op == "metadata":
        r, bs = case["requests"], case["block_size"]
        return {"bytes": 24 * case["padded"] + 12 * r + 8 * (case["tokens"] // bs + r),
                "flops": 8 * case["padded"]}
    es = SIZES[case["dtype"]]
    if op in ("norm", "norm_train"):
        n = case["rows"] * case["dim"]
        if op == "norm":
            return {"bytes": 4 * n * es + 2 * es * case["dim"], "flops": 8 * n}
        return {"bytes": 7 * n * es + (2 * es + 8) * case["dim"], "flops": 20 * n}
    gs, kv = SIZES[case["gates"]], case["dk"] * case["dv"]
    if op == "delta_update":
        live, rows = case["rows"] - case["pads"], case["rows"]
        row = es * (2 * case["kh"] * case["dk"] + 2 * case["vh"] * case["dv"]) + 2 * gs * case["vh"]
        return {"bytes": rows * row + live * 8 * case["vh"] * kv, "flops": 7 * live * case["vh"] * kv}
    t, state = case["total"], 4 * case["vh"] * kv
    row = es * (2 * case["kh"] * case["dk"] + 2 * case["vh"] * case["dv"]) + 2 * gs * case["vh"]
    if op == "delta_prefill":
        return {"bytes": t * row + state * (case["seqs"] + case["inits"]),
                "flops": 7 * t * case["vh"] * kv}
    # forward, and backward from dout: each input and each gradient once
    states = state * 4 * case["seqs"] if case["inits"] else 0
    return {"bytes": 2 * t * row + states, "flops": 21 * t * case["vh"] * kv}


# ---------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(seed)


def _randn(gen, shape, dtype=torch.float32, scale=1.0):
    t = torch.randn(shape, generator=gen, device=DEVICE, dtype=dtype)
    return t.mul_(scale) if scale != 1.0 else t


def _offsets(case, gen):
    """int32 [seqs + 1]: equal lengths, or random cuts (empty ones happen)."""
    seqs, total = case["seqs"], case["total"]
    if case["ragged"]:
        cuts = torch.randint(0, total + 1, (seqs - 1,), generator=gen, device=DEVICE).sort().values
    else:
        cuts = torch.arange(1, seqs, device=DEVICE) * (total // seqs)
    ends = torch.tensor([0, total], device=DEVICE)
    return torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)


def _some(gen, n, count):
    """bool [n] with `count` true entries at random places."""
    m = torch.zeros(n, dtype=torch.bool, device=DEVICE)
    m[torch.randperm(n, generator=gen, device=DEVICE)[:count]] = True
    return m


def _slots(gen, slots, rows, pads):
    """int32 [rows]: distinct state slots, PAD in `pads` of them."""
    idx = torch.randperm(slots, generator=gen, device=DEVICE)[:rows].to(torch.int32)
    return torch.where(_some(gen, rows, pads), torch.full_like(idx, PAD), idx)


def _delta_inputs(gen, case, n):
    """q and k of unit length, values, log decays (rates from 0.001 to 0.3 by
    head) and betas in (0, 1), for n tokens."""
    dtype, gates = DTYPES[case["dtype"]], DTYPES[case["gates"]]
    s = {}
    for name in ("q", "k"):
        t = _randn(gen, (n, case["kh"], case["dk"]))
        s[name] = (t / t.norm(dim=2, keepdim=True)).to(dtype)
    s["v"] = _randn(gen, (n, case["vh"], case["dv"]), dtype)
    rate = torch.exp(torch.rand(case["vh"], generator=gen, device=DEVICE) * math.log(300.0)) * 1e-3
    steps = torch.log1p(torch.exp(_randn(gen, (n, case["vh"]))))
    s["g"] = (-rate * steps).to(gates)
    s["beta"] = torch.sigmoid(_randn(gen, (n, case["vh"]))).to(gates)
    return s


def _metadata_lengths(gen, case):
    """int32 [requests] lengths of this step (their sum is `tokens`; most are
    one where the prompts among them are few) and of the tokens before it."""
    n, tokens = case["requests"], case["tokens"]
    weight = torch.rand(n, generator=gen, device=DEVICE, dtype=torch.float64).pow(6)
    share = torch.floor(weight.cumsum(0) / weight.sum().clamp_min(1e-300) * (tokens - n)).long()
    share[-1] = tokens - n
    query = 1 + torch.diff(share, prepend=share.new_zeros(1))
    context = torch.randint(0, case["context"] + 1, (n,), generator=gen, device=DEVICE)
    return query.to(torch.int32), context.to(torch.int32)


def prepare(case, seed):
    gen, op = _generator(seed), case["op"]
    s = dict(case=case)
    if op == "metadata":
        n, bs = case["requests"], case["block_size"]
        s["query_lens"], s["context_lens"] = _metadata_lengths(gen, case)
        width = (case["context"] + case["tokens"]) // bs + 1
        most = (case["tokens"] // bs + n) + n * (case["context"] // bs + 1)
        ids = torch.randperm(most, generator=gen, device=DEVICE).to(torch.int32)
        have = (s["context_lens"].long() + bs - 1) // bs
        first = have.cumsum(0) - have
        col = torch.arange(width, device=DEVICE)
        at = (first[:, None] + col).clamp_max(most - 1)
        s["block_table"] = torch.where(col < have[:, None], ids[at], PAD).to(torch.int32)
        s["free_blocks"] = ids[n * (case["context"] // bs + 1):].contiguous()
        s["query_start_loc"] = torch.zeros(n + 1, dtype=torch.int32, device=DEVICE)
        for name, dt in (("seq_idx", torch.int32), ("query_start", torch.int32),
                         ("positions", torch.int64), ("slot_mapping", torch.int64)):
            s[name] = torch.zeros(case["padded"], dtype=dt, device=DEVICE)
        s["blocks_used"] = torch.zeros(1, dtype=torch.int32, device=DEVICE)
        return s
    if op in ("norm", "norm_train"):
        shape, dtype = (case["rows"], case["dim"]), DTYPES[case["dtype"]]
        s["x"], s["residual"] = _randn(gen, shape, dtype), _randn(gen, shape, dtype, 2.0)
        s["weight"] = _randn(gen, (case["dim"],), dtype, 0.1).add_(1.0)
        s["bias"] = _randn(gen, (case["dim"],), dtype, 0.1)
        s["sum"] = torch.empty(shape, dtype=dtype, device=DEVICE)
        if op == "norm_train":
            s["dout"], s["dsum"] = _randn(gen, shape, dtype), _randn(gen, shape, dtype)
        return s
    n = case["rows"] if op == "delta_update" else case["total"]
    s |= _delta_inputs(gen, case, n)
    shape = (case["vh"], case["dk"], case["dv"])
    if op != "delta_train":
        many = n if op == "delta_update" else case["seqs"]
        s["states"] = _randn(gen, (case["slots"], *shape), scale=0.3)
        s["indices"] = _slots(gen, case["slots"], many, case["pads"])
        s["out"] = torch.zeros_like(s["v"])
    if op == "delta_update":
        return s
    s["qsl"] = _offsets(case, gen)
    s["has_init"] = _some(gen, case["seqs"], case["inits"]) if case["inits"] else None
    if op == "delta_train":
        s["dout"] = _randn(gen, s["v"].shape, s["v"].dtype)
        if case["inits"]:
            s["initial"] = _randn(gen, (case["seqs"], *shape), scale=0.3)
            s["dfinal"] = _randn(gen, (case["seqs"], *shape), scale=0.3)
    return s


# ---------------------------------------------------------------- the operators

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_delta_update(s):
    import depthwise_causal_conv1d_amd as lib
    lib.gated_delta_rule_update(s["q"], s["k"], s["v"], s["g"], s["beta"], s["states"],
                                s["indices"], pad_slot_id=PAD, out=s["out"])
    return {"out": s["out"], "states": s["states"]}


def _own_delta_prefill(s):
    import depthwise_causal_conv1d_amd as lib
    lib.gated_delta_rule_varlen_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["states"],
                                    s["qsl"], s["indices"], s["has_init"], pad_slot_id=PAD,
                                    out=s["out"])
    return {"out": s["out"], "states": s["states"]}


def _own_delta_train(s):
    import depthwise_causal_conv1d_amd as lib
    args = s["q"], s["k"], s["v"], s["g"], s["beta"]
    states = s["initial"].clone() if s["has_init"] is not None else None
    dinitial = torch.empty_like(states) if states is not None else None
    marks = lib.gated_delta_rule_checkpoints(s["k"], s["v"], s["qsl"])
    out = lib.gated_delta_rule_varlen_fwd(*args, states, s["qsl"], None, s["has_init"],
                                          checkpoints=marks)
    grads = lib.gated_delta_rule_varlen_bwd(s["dout"], *args, marks, s["qsl"], None, s["has_init"],
                                            dfinal_states=s.get("dfinal"),
                                            dinitial_states=dinitial)
    got = {"out": out} | dict(zip(("dq", "dk", "dv", "dg", "dbeta"), grads))
    if states is not None:
        got |= {"final": states, "dinitial": dinitial}
    return got


def _own_norm(s):
    import depthwise_causal_conv1d_amd as lib
    out = lib.layer_norm_fwd(s["x"], s["weight"], s["bias"], EPS, residual=s["residual"],
                             residual_out=s["sum"])
    return {"out": out, "sum": s["sum"]}


def _own_norm_train(s):
    import depthwise_causal_conv1d_amd as lib
    got = _own_norm(s)
    dx, dweight, dbias = lib.layer_norm_bwd(s["dout"], s["sum"], s["weight"], EPS,
                                            dresidual=s["dsum"])
    return got | {"dx": dx, "dweight": dweight, "dbias": dbias}


METADATA = ("block_table", "query_start_loc", "seq_idx", "query_start", "positions",
            "slot_mapping", "blocks_used")


def _own_metadata(s):
    import depthwise_causal_conv1d_amd as lib
    lib.sconv_paged_metadata(s["query_lens"], s["context_lens"], s["free_blocks"],
                             s["block_table"], s["case"]["block_size"], s["query_start_loc"],
                             s["seq_idx"], s["query_start"], s["positions"], s["slot_mapping"],
                             s["blocks_used"])
    return {name: s[name] for name in METADATA}


# ---------------------------------------------------------------- plain forms (32 bits)

def _heads(s, name):
    """q or k for every value head, in 32 bits."""
    t = s[name].float()
    return t.repeat_interleave(s["v"].shape[1] // t.shape[1], 1)


def _plain_delta_update(s):
    idx = s["indices"].long()
    rows = torch.nonzero(idx != PAD)[:, 0]
    slot = idx[rows]
    q, k, v = _heads(s, "q")[rows], _heads(s, "k")[rows], s["v"].float()[rows]
    g, beta = s["g"].float()[rows], s["beta"].float()[rows]
    state = s["states"][slot] * torch.exp(g)[:, :, None, None]
    u = beta[:, :, None] * (v - (state * k[:, :, :, None]).sum(2))
    state = state + k[:, :, :, None] * u[:, :, None, :]
    s["states"][slot] = state
    out = (state * q[:, :, :, None]).sum(2) * q.shape[2] ** -0.5
    s["out"][rows] = out.to(s["out"].dtype)
    return {"out": s["out"], "states": s["states"]}


def _chunked(s, q, k, v, g, beta, h0):
    """The delta rule by chunks over padded sequences: out [total, vh, dv] and
    the last states, all in 32 bits; q, k, v, g, beta are [total, vh, ...].
    Padded tokens have beta and g of zero, which leave a state as it is."""
    qsl, total = s["qsl"].long(), v.shape[0]
    n, c, vh, dk = qsl.numel() - 1, CHUNK, v.shape[1], k.shape[2]
    tokens = torch.arange(total, device=v.device)
    seq = torch.searchsorted(qsl[1:].contiguous(), tokens, right=True)
    count = max(1, -(-int((qsl[1:] - qsl[:-1]).max()) // c))
    place = seq * (count * c) + tokens - qsl[seq]

    def lay(t):  # [total, vh, d] -> [count, n * vh, c, d]
        d = t.shape[2]
        p = t.new_zeros(n * count * c, vh, d).index_copy(0, place, t)
        return p.view(n, count, c, vh, d).permute(1, 0, 3, 2, 4).reshape(count, n * vh, c, d)

    # sums and differences of log decays lose in 32 bits what the gradients need
    cum = lay(g[:, :, None].double()).cumsum(2)
    q, k, v, beta = lay(q) * dk ** -0.5, lay(k), lay(v), lay(beta[:, :, None])
    lower = torch.ones(c, c, dtype=torch.bool, device=v.device).tril()
    between = torch.exp((cum - cum.transpose(2, 3)).masked_fill(~lower, -math.inf)).float()
    grown, left = torch.exp(cum).float(), torch.exp(cum[:, :, -1:] - cum).float()
    whole = torch.exp(cum[:, :, -1:]).float()
    kt = k.transpose(2, 3).contiguous()
    p = (q @ kt) * between
    a = ((k @ kt) * between * beta).tril(-1)
    # (I + A)^-1 = (I - A)(I + A^2)(I + A^4)... : A^64 is zero
    eye = torch.eye(c, device=v.device)
    inverse, power = eye - a, a @ a
    for _ in range(5):
        inverse = inverse + inverse @ power
        power = power @ power
    state, outs = h0.reshape(n * vh, dk, -1), []
    for i in range(count):
        u = inverse[i] @ (beta[i] * (v[i] - grown[i] * (k[i] @ state)))
        outs.append(grown[i] * (q[i] @ state) + p[i] @ u)
        state = whole[i] * state + kt[i] @ (left[i] * u)
    out = torch.stack(outs).view(count, n, vh, c, -1).permute(1, 0, 3, 2, 4)
    return out.reshape(n * count * c, vh, -1)[place], state.view(n, vh, dk, -1), seq


def _plain_delta_prefill(s):
    idx = s["indices"].long()
    live = idx != PAD
    h0 = s["states"][idx.clamp_min(0)]
    has = s["has_init"]
    h0 = h0 * has[:, None, None, None] if has is not None else torch.zeros_like(h0)
    out, last, seq = _chunked(s, _heads(s, "q"), _heads(s, "k"), s["v"].float(), s["g"].float(),
                              s["beta"].float(), h0)
    s["states"][idx[live]] = last[live]
    out = torch.where(live[seq][:, None, None], out.to(s["v"].dtype), s["out"])
    return {"out": out, "states": s["states"]}


def _plain_delta_train(s):
    has, n = s["has_init"], s["qsl"].numel() - 1
    leaves = [s[name].float().requires_grad_() for name in ("q", "k", "v", "g", "beta")]
    q, k, v, g, beta = leaves
    group = v.shape[1] // q.shape[1]
    if has is not None:
        initial = s["initial"].clone().requires_grad_()
        h0 = initial * has[:, None, None, None]
    else:
        h0 = v.new_zeros(n, v.shape[1], k.shape[2], v.shape[2])
    out, last, _ = _chunked(s, q.repeat_interleave(group, 1), k.repeat_interleave(group, 1), v, g,
                            beta, h0)
    tops, given = [out], [s["dout"].float()]
    if has is not None:
        leaves, tops, given = leaves + [initial], tops + [last], given + [s["dfinal"]]
    grads = torch.autograd.grad(tops, leaves, given)
    got = {"out": out.detach().to(s["v"].dtype)}
    for name, t in zip(("q", "k", "v", "g", "beta"), grads):
        got["d" + name] = t.to(s[name].dtype)
    if has is not None:
        got |= {"final": last.detach(), "dinitial": grads[5]}
    return got


def _normed(s):
    z = s["x"].float() + s["residual"].float()
    d = z - z.mean(1, keepdim=True)
    rstd = torch.rsqrt(d.square().mean(1, keepdim=True) + EPS)
    return z, d * rstd * s["weight"].float() + s["bias"].float()


def _plain_norm(s):
    z, y = _normed(s)
    s["sum"].copy_(z)
    return {"out": y.to(s["x"].dtype), "sum": s["sum"]}


def _plain_norm_train(s):
    got = _plain_norm(s)
    # the backward pass takes the sum as it was stored
    z, g, w = got["sum"].float(), s["dout"].float(), s["weight"].float()
    d = z - z.mean(1, keepdim=True)
    rstd = torch.rsqrt(d.square().mean(1, keepdim=True) + EPS)
    hat, wg = d * rstd, w * g
    dx = rstd * (wg - wg.mean(1, keepdim=True) - hat * (wg * hat).mean(1, keepdim=True))
    return got | {"dx": (dx + s["dsum"].float()).to(s["x"].dtype),
                  "dweight": (g * hat).double().sum(0).float(), "dbias": g.double().sum(0).float()}


def _plain_metadata(s):
    bs, table = s["case"]["block_size"], s["block_table"]
    query, context = s["query_lens"].long(), s["context_lens"].long()
    ends = query.cumsum(0)
    s["query_start_loc"][1:] = ends.to(torch.int32)
    have = (context + bs - 1) // bs
    need = (context + query + bs - 1) // bs - have
    first = need.cumsum(0) - need
    s["blocks_used"].copy_(need.sum())
    col = torch.arange(table.shape[1], device=table.device) - have[:, None]
    fresh = (col >= 0) & (col < need[:, None])
    at = first[:, None] + col
    free = s["free_blocks"]
    ids = torch.where(at < free.numel(), free[at.clamp(0, free.numel() - 1)], PAD)
    table.copy_(torch.where(fresh, ids, table))
    t = torch.arange(s["positions"].numel(), device=table.device)
    live = t < ends[-1]
    r = torch.searchsorted(ends, t, right=True).clamp_max(query.numel() - 1)
    start = (ends - query)[r]
    pos = context[r] + t - start
    block = table[r, (pos // bs).clamp_max(table.shape[1] - 1)].long()
    slot = torch.where(live & (block >= 0), block * bs + pos % bs, PAD)
    for name, v in (("seq_idx", r * live), ("query_start", start * live), ("positions", pos * live),
                    ("slot_mapping", slot)):
        s[name].copy_(v)
    return {name: s[name] for name in METADATA}


_own = {"delta_update": _own_delta_update, "delta_prefill": _own_delta_prefill,
        "delta_train": _own_delta_train, "norm": _own_norm, "norm_train": _own_norm_train,
        "metadata": _own_metadata}
_plain = {"delta_update": _plain_delta_update, "delta_prefill": _plain_delta_prefill,
          "delta_train": _plain_delta_train, "norm": _plain_norm, "norm_train": _plain_norm_train,
          "metadata": _plain_metadata}


# ---------------------------------------------------------------- 64 bits, from the definitions

def _padded(s, *names):
    """Inputs in 64 bits as [longest, seqs, heads, ...] (zeros behind each
    sequence's end), q and k for every value head; the mask of real tokens."""
    bounds = s["qsl"].tolist()
    n = len(bounds) - 1
    longest = max([hi - lo for lo, hi in zip(bounds[:-1], bounds[1:])])
    real = torch.zeros(longest, n, dtype=torch.bool, device=s["v"].device)
    got = [torch.zeros(longest, n, s["v"].shape[1], *s[name].shape[2:], dtype=torch.float64,
                       device=s["v"].device) for name in names]
    for b, (lo, hi) in enumerate(zip(bounds[:-1], bounds[1:])):
        real[:hi - lo, b] = True
        for p, name in zip(got, names):
            t = s[name][lo:hi].double()
            p[:hi - lo, b] = t.repeat_interleave(p.shape[2] // t.shape[1], 1)
    return got, real


def _packed(s, p):
    """[longest, seqs, ...] back to [total, ...]."""
    bounds = s["qsl"].tolist()
    return torch.cat([p[:hi - lo, b] for b, (lo, hi) in enumerate(zip(bounds[:-1], bounds[1:]))])


def _token(state, q, k, v, g, beta, scale):
    """One token of every head: the decayed state, the error, the new state
    and the output."""
    old = state * torch.exp(g)[..., None, None]
    err = v - torch.einsum("...kv,...k->...v", old, k)
    new = old + k[..., :, None] * (beta[..., None] * err)[..., None, :]
    return old, err, new, scale * torch.einsum("...kv,...k->...v", new, q)


def _exact_delta_update(s):
    group = s["v"].shape[1] // s["q"].shape[1]
    live = (s["indices"] != PAD).nonzero()[:, 0]
    slot = s["indices"][live].long()
    q, k = (s[n].double().repeat_interleave(group, 1)[live] for n in ("q", "k"))
    v, g, beta = (s[n].double()[live] for n in ("v", "g", "beta"))
    states, out = s["states"].double(), torch.zeros(s["v"].shape, dtype=torch.float64,
                                                    device=s["v"].device)
    _, _, states[slot], out[live] = _token(states[slot], q, k, v, g, beta, q.shape[2] ** -0.5)
    return {"out": out, "states": states}


def _exact_forward(s, state):
    """Outputs [longest, seqs, ...], the last states, and the state before
    every 64th token."""
    (q, k, v, g, beta), real = _padded(s, "q", "k", "v", "g", "beta")
    out, marks, scale = torch.zeros_like(v), [], k.shape[3] ** -0.5
    for t in range(v.shape[0]):
        if t % 64 == 0:
            marks.append(state)
        # behind its end a sequence's g, beta and k are zero: its state stays
        _, _, state, out[t] = _token(state, q[t], k[t], v[t], g[t], beta[t], scale)
    return out, state, marks, (q, k, v, g, beta)


def _exact_delta_prefill(s):
    bounds, slots = s["qsl"].tolist(), s["indices"].tolist()
    has = s["has_init"].tolist() if s["has_init"] is not None else [False] * len(slots)
    states = s["states"].double()
    h0 = torch.stack([states[p] if p != PAD and y else torch.zeros_like(states[0])
                      for p, y in zip(slots, has)])
    out, last, _, _ = _exact_forward(s, h0)
    out = _packed(s, out)
    for b, p in enumerate(slots):
        if p == PAD:
            out[bounds[b]:bounds[b + 1]] = 0
        else:
            states[p] = last[b]
    return {"out": out, "states": states}


def _exact_delta_train(s):
    has, n = s["has_init"], s["qsl"].numel() - 1
    shape = (n, s["v"].shape[1], s["k"].shape[2], s["v"].shape[2])
    h0 = torch.zeros(shape, dtype=torch.float64, device=s["v"].device)
    ds = torch.zeros_like(h0)
    if has is not None:
        h0, ds = s["initial"].double() * has[:, None, None, None], s["dfinal"].double()
    out, last, marks, (q, k, v, g, beta) = _exact_forward(s, h0)
    (dout,), real = _padded(s, "dout")
    scale = k.shape[3] ** -0.5
    dq, dk, dv, dg, dbeta = (torch.zeros_like(t) for t in (q, k, v, g, beta))
    for c in range(len(marks) - 1, -1, -1):
        lo, hi = 64 * c, min(64 * c + 64, v.shape[0])
        states, state = [], marks[c]
        for t in range(lo, hi):
            old, err, new, _ = _token(state, q[t], k[t], v[t], g[t], beta[t], scale)
            states.append((state, old, err, new))
            state = new
        for t in range(hi - 1, lo - 1, -1):
            before, old, err, new = states[t - lo]
            dq[t] = scale * torch.einsum("...kv,...v->...k", new, dout[t])
            ds = ds + scale * q[t][..., :, None] * dout[t][..., None, :]
            du = torch.einsum("...kv,...k->...v", ds, k[t])
            dbeta[t] = (du * err).sum(-1)
            de = beta[t][..., None] * du
            dv[t] = de
            dk[t] = (torch.einsum("...kv,...v->...k", ds, beta[t][..., None] * err)
                     - torch.einsum("...kv,...v->...k", old, de))
            ds = ds - k[t][..., :, None] * de[..., None, :]
            dg[t] = (ds * old).sum((-1, -2))
            ds = ds * torch.exp(g[t])[..., None, None]
    kh = s["q"].shape[1]
    got = {"out": out, "dv": dv, "dg": dg, "dbeta": dbeta,
           "dq": dq.unflatten(2, (kh, -1)).sum(3), "dk": dk.unflatten(2, (kh, -1)).sum(3)}
    got = {name: _packed(s, t) for name, t in got.items()}
    if has is not None:
        got |= {"final": last, "dinitial": ds * has[:, None, None, None]}
    return {name: got[name] for name in ("out", "dq", "dk", "dv", "dg", "dbeta", "final",
                                         "dinitial") if name in got}


def _exact_norm(s):
    z = s["x"].double() + s["residual"].double()
    var, mean = torch.var_mean(z, 1, correction=0, keepdim=True)
    return {"out": (z - mean) / torch.sqrt(var + EPS) * s["weight"].double() + s["bias"].double(),
            "sum": z}


def _exact_norm_train(s):
    """Automatic differentiation at the rows as they were stored."""
    got = _exact_norm(s)
    t = got["sum"].to(s["x"].dtype).double().requires_grad_()
    w, b = (s[n].double().requires_grad_() for n in ("weight", "bias"))
    var, mean = torch.var_mean(t, 1, correction=0, keepdim=True)
    y = (t - mean) / torch.sqrt(var + EPS) * w + b
    dx, dw, db = torch.autograd.grad(y, (t, w, b), s["dout"].double())
    return got | {"dx": dx + s["dsum"].double(), "dweight": dw, "dbias": db}


def _exact_metadata(s):
    """Whole numbers, request by request."""
    bs, dev = s["case"]["block_size"], s["positions"].device
    table, free = s["block_table"].tolist(), s["free_blocks"].tolist()
    padded = s["positions"].numel()
    qsl, used = [0], 0
    rows = {name: [] for name in ("seq_idx", "query_start", "positions", "slot_mapping")}
    for r, (m, c) in enumerate(zip(s["query_lens"].tolist(), s["context_lens"].tolist())):
        for j in range(-(-c // bs), -(-(c + m) // bs)):
            table[r][j] = free[used]
            used += 1
        for pos in range(c, c + m):
            rows["seq_idx"].append(r)
            rows["query_start"].append(qsl[-1])
            rows["positions"].append(pos)
            rows["slot_mapping"].append(table[r][pos // bs] * bs + pos % bs)
        qsl.append(qsl[-1] + m)
    got = {"block_table": table, "query_start_loc": qsl}
    for name, v in rows.items():
        got[name] = v + [PAD if name == "slot_mapping" else 0] * (padded - len(v))
    got["blocks_used"] = [used]
    return {name: torch.tensor(v, dtype=s[name].dtype, device=dev) for name, v in got.items()}


_exact = {"delta_update": _exact_delta_update, "delta_prefill": _exact_delta_prefill,
          "delta_train": _exact_delta_train, "norm": _exact_norm, "norm_train": _exact_norm_train,
          "metadata": _exact_metadata}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact[case["op"]](s)
