"""Cases, plain forms and exact values of the operators between a head's logits and its loss.

Four operators are measured, as a rollout or a training step calls them:

  adapter  logits of a shared head with low-rank adapters, one per row:
           z_i = W h_i + s_a B_a (A_a h_i),  a = adapter of row i (-1: none)
  shape    penalties, biases, grammar masks and temperature on logits:
           z' = (rep(z) - f c - p [c > 0] + b) / T,  -inf where not allowed
  logp     selected-token log-prob and LSE under the shaped logits
  grad     gradient of the shaped log-prob with respect to the raw logits

Run with ``own`` false, ``run`` is elementary torch operations in fp32; with
``own`` true it makes the calls of the package.
"""
import math

import torch

own = False

NEG = float("-inf")


# ------------------------------------------------------------------ cases
def _adapter(name, rows, D, V, adapters, rank, out, prompts):
    return {"name": name, "kind": "adapter", "rows": rows, "D": D, "V": V, "adapters": adapters, "rank": rank,
            "out": out, "prompts": prompts}


def _logits(name, kind, rows, V, hist, dtype, seq, grammar):
    """hist: longest history; seq: rows that share one growing history (0: each row has its own);
    grammar: whether part of the rows carries an allow mask."""
    return {"name": name, "kind": kind, "rows": rows, "V": V, "hist": hist, "dtype": dtype, "seq": seq,
            "grammar": grammar}


def listed():
    return [
        # one token of one request, on the packed workload's head: latency
        _adapter("adapter 1 token", 1, 2048, 32000, 4, 16, "bf16", False),
        # an ordinary decode batch on the 8B vocabulary, requests spread over 16 adapters
        _adapter("adapter 64 tokens 8B", 64, 4096, 151936, 16, 16, "bf16", False),
        # a ragged batch on the selective log-prob head, fp32 logits
        _adapter("adapter 37 tokens ragged", 37, 1000, 5000, 5, 8, "fp32", False),
        # prompts of several requests on the 8B vocabulary: rows of a request are consecutive
        _adapter("adapter prompts 8B", 2048, 4096, 151936, 8, 32, "bf16", True),
        # one request's next token
        _logits("shape 1 token", "shape", 1, 32000, 700, "bf16", 0, False),
        # a full decode batch, a part of it under a grammar
        _logits("shape 256 tokens 8B", "shape", 256, 151936, 4096, "bf16", 0, True),
        # fp32 logits of an odd vocabulary: no row but the first starts on a 16-byte boundary
        _logits("shape 129 tokens odd", "shape", 129, 32003, 1500, "fp32", 0, True),
        # the behaviour log-probs of a decode batch
        _logits("logp 256 tokens 8B", "logp", 256, 151936, 4096, "bf16", 0, True),
        # a training micro-batch of the 8B-vocabulary workload: 8 sequences of 1024 tokens
        _logits("logp 8192 tokens 8B", "logp", 8192, 151936, 1024, "bf16", 1024, False),
        # the small GRPO workload in fp32: 8 sequences of 128 tokens
        _logits("logp 1024 tokens small", "logp", 1024, 4096, 128, "fp32", 128, True),
        # the gradient of that training micro-batch
        _logits("grad 8192 tokens 8B", "grad", 8192, 151936, 1024, "bf16", 1024, False),
        # the gradient of packed sequences over an odd vocabulary
        _logits("grad 1531 tokens odd", "grad", 1531, 32003, 377, "bf16", 377, True),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["adapter", "shape", "logp", "grad"])
    V = _logu(rng, 1000, 151936)
    if rng.random() < 0.5:
        V = V // 8 * 8
    if kind == "adapter":
        prompts = rng.random() < 0.4
        return {"kind": kind, "rows": _logu(rng, 100, 2048) if prompts else _logu(rng, 1, 256),
                "D": 8 * _logu(rng, 8, 512), "V": V, "adapters": _logu(rng, 1, 24), "rank": rng.choice([8, 16, 32, 64]),
                "out": rng.choice(["bf16", "fp32"]), "prompts": prompts}
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if kind == "shape" or (kind == "logp" and rng.random() < 0.5):
        return {"kind": kind, "rows": _logu(rng, 1, 384), "V": V, "hist": _logu(rng, 1, 8192), "dtype": dtype,
                "seq": 0, "grammar": rng.random() < 0.5}
    seq = _logu(rng, 16, 1024)
    return {"kind": kind, "rows": _logu(rng, 64, 4096), "V": V, "hist": seq, "dtype": dtype, "seq": seq,
            "grammar": rng.random() < 0.3}


# ------------------------------------------------------------------ inputs
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _normal(g, shape, std, dtype):
    """Normal values, drawn in slices of rows (a whole fp32 draw of the largest logits is 5 GB)."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device="cuda").mul_(std)
    return out


def _ids(g, n, V):
    """Token ids as text has them: few frequent ones, a long tail, spread over the vocabulary."""
    rank = (V * _rand(g, n) ** 4).long().clamp_(max=V - 1)
    return ((rank * 7919) % V).to(torch.int32)


def _prepare_adapter(c, g):
    n, D, V, m, r = c["rows"], c["D"], c["V"], c["adapters"], c["rank"]
    if c["prompts"]:
        cuts = torch.sort((_rand(g, 11) * n).long())[0]
        req = torch.searchsorted(cuts, torch.arange(n, device="cuda"), right=True)
        ids = (_rand(g, 12) * (m + 1)).to(torch.int32)[req] - 1
    else:
        ids = (_rand(g, n) * (m + 0.5)).to(torch.int32)
        ids = torch.where(ids >= m, torch.full_like(ids, -1), ids)
    return {"H": _normal(g, (n, D), 1.0, torch.bfloat16),
            "W": _normal(g, (V, D), D ** -0.5, torch.bfloat16),
            "A": _normal(g, (m, r, D), D ** -0.5, torch.bfloat16),
            "B": _normal(g, (m, V, r), 0.3 * r ** -0.5, torch.bfloat16),
            "scale": 0.5 + _rand(g, m), "ids": ids.contiguous(),
            "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


def _prepare_logits(c, g):
    n, V, L = c["rows"], c["V"], c["hist"]
    s = {"logits": _normal(g, (n, V), 2.5, _TYPES[c["dtype"]])}
    row = torch.arange(n, device="cuda")
    if c["seq"]:
        # packed sequences: row i sees the tokens of its sequence before it
        T = c["seq"]
        nseq = -(-n // T)
        seq, pos = row // T, row % T
        s["tokens"] = _ids(g, nseq * T, V)
        s["begin"] = (seq * T).to(torch.int64)
        s["len"] = pos.to(torch.int32)
        prompt = (T * (0.05 + 0.2 * _rand(g, nseq))).long()
        s["prompt"] = prompt[seq].to(torch.int32)
        live = (T * (0.4 + 0.6 * _rand(g, nseq))).long()
        s["mask"] = ((pos >= prompt[seq]) & (pos < live[seq])).to(torch.uint8)
        s["targets"] = s["tokens"][:n].clone()
        group = seq
    else:
        # a decode batch: every row has a history of its own
        length = (L * (0.1 + 0.9 * _rand(g, n))).long().clamp_(min=1)
        begin = torch.cumsum(length, 0) - length
        s["tokens"] = _ids(g, int(length.sum()), V)
        s["begin"] = begin
        s["len"] = length.to(torch.int32)
        s["prompt"] = (length * _rand(g, n)).to(torch.int32)
        s["mask"] = torch.ones(n, dtype=torch.uint8, device="cuda")
        s["targets"] = _ids(g, n, V)
        group = row
    ngroup = int(group[-1]) + 1
    pick = lambda t: t[group].contiguous()  # noqa: E731
    s["rep"] = pick(1.0 + 0.3 * _rand(g, ngroup))
    s["pres"] = pick(0.5 * _rand(g, ngroup))
    s["freq"] = pick(0.3 * _rand(g, ngroup))
    s["temp"] = pick(0.6 + 0.6 * _rand(g, ngroup))
    # eight lists of 32 biased tokens, each token once in a list; every second group uses one
    nset, per = 8, 32
    s["bias_off"] = (torch.arange(nset + 1, device="cuda") * per).to(torch.int32)
    s["bias_tok"] = torch.stack([torch.randperm(V, generator=g, device="cuda")[:per] for _ in range(nset)]).view(-1).to(
        torch.int32)
    s["bias_val"] = 4 * _rand(g, nset * per) - 2
    sets = (_rand(g, ngroup) * 2 * nset).to(torch.int32)
    s["bias_set"] = pick(torch.where(sets >= nset, torch.full_like(sets, -1), sets))
    if c["grammar"]:
        # four masks: two that leave a few tokens (inside a string, a key), two that bar a few
        words = -(-V // 32)
        keep = torch.tensor([0.002, 0.01, 0.9, 0.97], device="cuda")
        ok = _rand(g, 4, words * 32) < keep[:, None]
        ok[:, :32] = True
        bits = (ok.view(4, words, 32).long() << torch.arange(32, device="cuda")).sum(-1)
        s["allow"] = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)
        which = (_rand(g, ngroup) * 8).to(torch.int32)
        s["allow_row"] = pick(torch.where(which >= 4, torch.full_like(which, -1), which))
        first = (s["targets"] % 32).to(torch.int32)     # allowed everywhere
        s["targets"] = torch.where(s["allow_row"] >= 0, first, s["targets"]).to(torch.int32)
    if c["kind"] == "grad":
        # what a forward leaves: the LSE of each row, and d loss / d logp (0 where the clip cut it off)
        lse = torch.empty(n, device="cuda")
        step = max(1, (1 << 28) // V)
        for i in range(0, n, step):
            lse[i:i + step] = torch.logsumexp(_shaped64(s, slice(i, min(n, i + step)))[0], 1).float()
        s["lse"] = torch.where(s["mask"] > 0, lse, torch.zeros_like(lse))
        coef = torch.randn(n, generator=g, device="cuda") / n
        coef[_rand(g, n) < 0.1] = 0.0
        s["coef"] = torch.where(s["mask"] > 0, coef, torch.zeros_like(coef))
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def prepare(case, seed):
    g = _gen(seed)
    state = _prepare_adapter(case, g) if case["kind"] == "adapter" else _prepare_logits(case, g)
    state["case"] = case
    return state


# ------------------------------------------------------------------ plain forms (fp32)
def _plain_adapter(s):
    c = s["case"]
    m, r, V = c["adapters"], c["rank"], c["V"]
    H = s["H"].float()
    z = H @ s["W"].float().t()
    u = (H @ s["A"].float().view(m * r, -1).t()).view(-1, m, r)
    on = (s["ids"][:, None] == torch.arange(m, device="cuda")).float() * s["scale"]
    u = (u * on[:, :, None]).view(-1, m * r)
    z += u @ s["B"].float().permute(0, 2, 1).reshape(m * r, V)
    return {"logits": z.to(_TYPES[c["out"]])}


def _plain_counts(s, V):
    """[n, V] counts of each token in the row's output, and whether it is in the row's history at all."""
    n = s["len"].numel()
    longest = int(s["case"]["hist"])
    at = torch.arange(longest, device="cuda")
    inside = at < s["len"][:, None]
    tok = s["tokens"][(s["begin"][:, None] + at).clamp_(max=s["tokens"].numel() - 1)].long()
    out = torch.zeros(n, V, device="cuda").scatter_add_(1, tok, (inside & (at >= s["prompt"][:, None])).float())
    seen = torch.zeros(n, V, device="cuda").scatter_add_(1, tok, inside.float())
    return out, seen > 0


def _plain_bias(s, z):
    per = int(s["bias_off"][1])
    lists = s["bias_tok"].view(-1, per).long()
    vals = s["bias_val"].view(-1, per)
    use = s["bias_set"] >= 0
    which = s["bias_set"].clamp(min=0).long()
    return z.scatter_add_(1, lists[which], vals[which] * use[:, None].float())


def _plain_allowed(s, V):
    bits = s["allow"][s["allow_row"].clamp(min=0).long()]
    ok = ((bits[:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1).view(bits.shape[0], -1)[:, :V]
    return (ok > 0) | (s["allow_row"] < 0)[:, None]


def _plain_shaped(s):
    """Shaped logits in fp32 and d shaped / d raw."""
    V = s["logits"].shape[1]
    z = s["logits"].float()
    out, seen = _plain_counts(s, V)
    rep = s["rep"][:, None]
    slope = torch.where(seen, torch.where(z > 0, 1 / rep, rep), torch.ones((), device="cuda"))
    z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
    z = z - s["freq"][:, None] * out - s["pres"][:, None] * (out > 0)
    z = _plain_bias(s, z)
    z = z / s["temp"][:, None]
    slope = slope / s["temp"][:, None]
    if "allow" in s:
        ok = _plain_allowed(s, V)
        z = torch.where(ok, z, torch.full((), NEG, device="cuda"))
        slope = slope * ok
    return z, slope


def _plain_logits(s):
    kind = s["case"]["kind"]
    z, slope = _plain_shaped(s)
    if kind == "shape":
        return {"logits": z.to(s["logits"].dtype)}
    live = s["mask"] > 0
    y = s["targets"].long()[:, None]
    if kind == "logp":
        top = z.max(1, keepdim=True)[0]
        lse = (z - top).exp().sum(1).log() + top[:, 0]
        zero = torch.zeros((), device="cuda")
        return {"logp": torch.where(live, z.gather(1, y)[:, 0] - lse, zero), "lse": torch.where(live, lse, zero)}
    p = (z - s["lse"][:, None]).exp()
    d = (-p).scatter_add_(1, y, torch.ones_like(p[:, :1]))
    d = torch.where((s["coef"] != 0)[:, None], d * s["coef"][:, None] * slope, torch.zeros((), device="cuda"))
    return {"dlogits": d.to(s["logits"].dtype)}


# ------------------------------------------------------------------ the package's calls
def _own(s):
    from gspo_logprob_gb300 import ops
    c = s["case"]
    if c["kind"] == "adapter":
        r = ops.grpo_adapter_logits(s["H"], s["W"], s["A"], s["B"], s["scale"], s["ids"], out_dtype=_TYPES[c["out"]],
                                    status=s["status"])
        return {"logits": r["logits"]}
    if "shaping" not in s:
        # the description of the batch's shaping, which a program keeps as long as it keeps these tensors
        s["shaping"] = ops.make_shaping(
            rows=c["rows"], V=c["V"], tokens=s["tokens"], hist_begin=s["begin"], hist_len=s["len"],
            prompt_len=s["prompt"], repetition=s["rep"], presence=s["pres"], frequency=s["freq"],
            temperature=s["temp"], bias_offsets=s["bias_off"], bias_tokens=s["bias_tok"], bias_values=s["bias_val"],
            bias_set=s["bias_set"], allow_bits=s.get("allow"), allow_row=s.get("allow_row"))
    if c["kind"] == "shape":
        return {"logits": ops.grpo_shape_logits(s["logits"], s["shaping"], status=s["status"])["logits"]}
    if c["kind"] == "logp":
        r = ops.grpo_shaped_logp(s["logits"], s["targets"], s["mask"], s["shaping"], status=s["status"])
        return {"logp": r["logp"], "lse": r["lse"]}
    r = ops.grpo_shaped_logp_backward(s["logits"], s["targets"], s["mask"], s["shaping"], s["lse"], s["coef"],
                                      status=s["status"])
    return {"dlogits": r["dlogits"]}


def run(state):
    if own:
        return _own(state)
    return _plain_adapter(state) if state["case"]["kind"] == "adapter" else _plain_logits(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    n, V = case["rows"], case["V"]
    if case["kind"] == "adapter":
        D, r = case["D"], case["rank"]
        used = min(case["adapters"], 12 if case["prompts"] else n)
        size = 2 if case["out"] == "bf16" else 4
        return {"bytes": 2 * (n * D + V * D + used * r * (D + V)) + size * n * V,
                "flops": 2 * n * D * V + 2 * n * r * (D + V)}
    size = 2 if case["dtype"] == "bf16" else 4
    # of a decode batch every row is live; of packed sequences the part after the prompt, up to the sequence's end
    live = 0.55 if case["seq"] else 1.0
    if case["kind"] == "grad":
        live *= 0.9
    # half the rows carry a mask, half of those masks bar nearly everything, and barred logits need not be read
    read = live * (0.75 if case["grammar"] else 1.0)
    hist = 4 * (n if case["seq"] else 0.55 * case["hist"] * n)
    mask = 4 * (V // 8) if case["grammar"] else 0
    written = {"shape": n * V * size, "logp": 8 * n, "grad": n * V * size}[case["kind"]]
    return {"bytes": int(read * n * V * size + written + hist + mask + 60 * n),
            "flops": int(read * n * V * {"shape": 4, "logp": 7, "grad": 8}[case["kind"]])}


# ------------------------------------------------------------------ exact values (64 bits)
def _shaped64(s, rows):
    """Shaped logits of a slice of rows and the slope d shaped / d raw, from the definition in 64 bits."""
    z = s["logits"][rows].double()
    n, V = z.shape
    begin, length, prompt = s["begin"][rows], s["len"][rows].long(), s["prompt"][rows].long()
    # every (row, place in its history) as one flat list, counted by row and token
    row = torch.repeat_interleave(torch.arange(n, device="cuda"), length)
    place = torch.arange(row.numel(), device="cuda") - (torch.cumsum(length, 0) - length)[row]
    key = row * V + s["tokens"][begin[row] + place].long()
    seen = (torch.bincount(key, minlength=n * V) > 0).view(n, V)
    count = torch.bincount(key[place >= prompt[row]], minlength=n * V).view(n, V).double()
    theta = s["rep"][rows].double().unsqueeze(1)
    slope = torch.ones_like(z)
    slope[seen & (z > 0)] = 0
    slope = torch.where(seen, torch.where(slope == 0, theta.reciprocal(), theta), slope)
    z = z * slope
    z -= s["freq"][rows].double().unsqueeze(1) * count
    z -= s["pres"][rows].double().unsqueeze(1) * (count >= 1).double()
    off = s["bias_off"].long().tolist()
    which = s["bias_set"][rows]
    for k in range(len(off) - 1):
        b = torch.zeros(V, dtype=torch.float64, device="cuda")
        b[s["bias_tok"][off[k]:off[k + 1]].long()] = s["bias_val"][off[k]:off[k + 1]].double()
        z[which == k] += b
    t = s["temp"][rows].double().unsqueeze(1)
    z, slope = z / t, slope / t
    if "allow" in s:
        col = torch.arange(V, device="cuda")
        for k in range(s["allow"].shape[0]):
            bar = ((s["allow"][k][col // 32] >> (col % 32).to(torch.int32)) & 1) == 0
            at = (s["allow_row"][rows] == k)[:, None] & bar
            z.masked_fill_(at, NEG)
            slope.masked_fill_(at, 0.0)
    return z, slope


def exact(case, seed):
    s = prepare(case, seed)
    n, V = case["rows"], case["V"]
    if case["kind"] == "adapter":
        H = s["H"].double()
        out = torch.empty(n, V, dtype=torch.float64, device="cuda")
        step = max(1, (1 << 28) // case["D"])
        for i in range(0, V, step):
            out[:, i:i + step] = H @ s["W"][i:i + step].double().t()
        for a in range(case["adapters"]):
            at = (s["ids"] == a).nonzero()[:, 0]
            if at.numel():
                low = H[at] @ s["A"][a].double().t()
                out[at] += s["scale"][a].double() * (low @ s["B"][a].double().t())
        return {"logits": out}
    step = max(1, (1 << 28) // V)
    parts = [slice(i, min(n, i + step)) for i in range(0, n, step)]
    if case["kind"] == "shape":
        return {"logits": torch.cat([_shaped64(s, p)[0] for p in parts])}
    if case["kind"] == "logp":
        logp = torch.zeros(n, dtype=torch.float64, device="cuda")
        lse = torch.zeros(n, dtype=torch.float64, device="cuda")
        for p in parts:
            z = _shaped64(s, p)[0]
            lse[p] = torch.logsumexp(z, 1)
            logp[p] = z[torch.arange(z.shape[0], device="cuda"), s["targets"][p].long()] - lse[p]
        off = s["mask"] == 0
        logp[off], lse[off] = 0.0, 0.0
        return {"logp": logp, "lse": lse}
    out = torch.empty(n, V, dtype=torch.float64, device="cuda")
    for p in parts:
        z, slope = _shaped64(s, p)
        d = -torch.exp(z - s["lse"][p].double()[:, None])
        d[torch.arange(d.shape[0], device="cuda"), s["targets"][p].long()] += 1
        coef = s["coef"][p].double()
        out[p] = d * coef[:, None] * slope
        out[p][coef == 0] = 0.0
    return {"dlogits": out}
