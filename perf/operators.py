"""Measured cases of the serving and adapter operators.

Three operators, each a function of the package:

* ``lx_draft_verify``: for a batch of sequences, accepts or rejects each
  sequence's drafted tokens against the target's probabilities, from given
  random numbers, and draws the token that follows the accepted ones.
* ``lx_lora_forward``: adds to a projection's output the low-rank adapters of
  many requests at once, each request (a run of rows) with its own adapter.
* ``lx_lora_backward``: the gradients of the rows and of every adapter.

``run`` computes them from elementary torch operations while ``own`` is false
and through the package where it is true.  ``exact`` follows the definitions
in float64, one sequence or one request at a time.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one request being answered: four drafted tokens, the smallest call of a decoding loop
        verify("verify_one_request", S=1, max_draft=4, V=151936, dtype="bf16", lens="full"),
        # a serving batch: 0 to 6 drafted tokens each, sampling temperatures mixed with greedy requests
        verify("verify_batch_ragged", S=32, max_draft=6, V=151936, dtype="bf16", lens="ragged", temps="mixed",
               accept=0.93),
        # drafts looked up in the prompt (no draft distribution), odd vocabulary, binary16 logits
        verify("verify_lookup_odd_vocabulary", S=256, max_draft=4, V=50001, dtype="f16", lens="ragged", draft="none",
               accept=0.655),
        # a large batch of fp32 logits over a large vocabulary, rows padded to a wider array
        verify("verify_large_fp32", S=96, max_draft=7, V=262144, dtype="f32", lens="full", pad=64),
        # one token of one request
        lora("lora_one_token", "forward", T=1, R=1, adapters=1, H=4096, N=4096, r=16, base="f32", y="f32"),
        # a decoding batch: one token per request, adapters of different ranks, some requests without one
        lora("lora_decode_batch", "forward", T=64, R=64, adapters=48, H=4096, N=4096, r=16, ranks="mixed", base="f32",
             y="f32"),
        # the same at the vocabulary projection: fp32 products in, bf16 logits out
        lora("lora_decode_logits", "forward", T=64, R=64, adapters=8, H=4096, N=151936, r=16, base="f32", y="bf16"),
        # prompts of many lengths packed into one batch
        lora("lora_prompts", "forward", T=8192, R=12, adapters=6, H=4096, N=4096, r=64, base="f32", y="f32"),
        # a small training step with sizes off every tile
        lora("lora_backward_small_odd", "backward", T=75, R=5, adapters=3, H=1160, N=520, r=24, ranks="mixed"),
        # a training batch of several users' adapters
        lora("lora_backward_batch", "backward", T=4096, R=16, adapters=4, H=4096, N=4096, r=16, base="f32"),
        # one adapter of a higher rank trained alone
        lora("lora_backward_one_adapter", "backward", T=8192, R=8, adapters=1, H=4096, N=4096, r=64, base="f32"),
        # adapters on the vocabulary projection: the gradient of a batch of logits
        lora("lora_backward_logits", "backward", T=2048, R=8, adapters=2, H=4096, N=151936, r=16),
    ]


def verify(name, S, max_draft, V, dtype, lens, temps="one", draft="logits", pad=0, accept=0.87):
    # accept: the share of drafted tokens that these inputs' acceptance test passes (greedy requests among them)
    return {"name": name, "op": "verify", "S": S, "max_draft": max_draft, "V": V, "dtype": dtype, "lens": lens,
            "temps": temps, "draft": draft, "pad": pad, "accept": accept}


def lora(name, way, T, R, adapters, H, N, r, ranks="full", base="none", y="f32"):
    return {"name": name, "op": "lora_" + way, "T": T, "R": R, "adapters": adapters, "H": H, "N": N, "r": r,
            "ranks": ranks, "base": base, "y": y}


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["verify", "verify", "forward", "forward", "backward", "backward"])
    if op == "verify":
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        V = _log_int(rng, 1000, 262144)
        max_draft = rng.randint(1, 8)
        most = max(1, min(256, 96 * 8 * 262144 // (V * (max_draft + 1))))
        draft = rng.choice(["logits", "logits", "none"])
        case = verify("", S=_log_int(rng, 1, most), max_draft=max_draft, V=V, dtype=dtype,
                      lens=rng.choice(["full", "ragged"]), temps=rng.choice(["one", "mixed"]), draft=draft,
                      pad=rng.choice([0, 0, 1, 8, 64]), accept=0.87 if draft == "logits" else 0.655)
    else:
        H = 8 * _log_int(rng, 8, 1024)
        N = 8 * _log_int(rng, 8, 2048)
        most = max(1, min(8192, (1 << 26) // max(H, N)))
        T = _log_int(rng, 1, most)
        decode = rng.random() < 0.3
        R = T if decode else _log_int(rng, 1, max(1, min(T, 64)))
        if R > 256:
            T = R = 256
        case = lora("", op, T=T, R=R, adapters=_log_int(rng, 1, max(1, min(R, 48))), H=H, N=N,
                    r=8 * rng.choice([1, 2, 2, 3, 4, 8, 8, 16]), ranks=rng.choice(["full", "mixed"]),
                    base=rng.choice(["none", "f32", "bf16"]) if op == "forward" else rng.choice(["none", "f32"]),
                    y=rng.choice(["f32", "bf16"]) if op == "forward" else "f32")
    del case["name"]
    return case


# ---------------------------------------------------------------- what a case's sizes fix

def _rng(case, what):
    return random.Random("%s %s" % (what, sorted((k, v) for k, v in case.items() if k != "name")))


def _draft_lengths(case):
    rng = _rng(case, "lengths")
    S, L = case["S"], case["max_draft"]
    return [L if case["lens"] == "full" else rng.randint(0, L) for _ in range(S)]


def _temperatures(case):
    rng = _rng(case, "temperatures")
    return [rng.choice([0.0, 0.6, 0.8, 1.0, 1.25]) if case["temps"] == "mixed" else 1.0 for _ in range(case["S"])]


def _requests(case):
    """(first row of each request and the end, adapter of each request, rank of each adapter)"""
    rng = _rng(case, "requests")
    T, R, n, r = case["T"], case["R"], case["adapters"], case["r"]
    if R == T:
        start = list(range(T + 1))
    else:
        start = [0] + sorted(rng.randint(0, T) for _ in range(R - 1)) + [T]
    # in a large batch about one request in eight has no adapter (-1)
    adapter = [-1 if R > 8 and rng.random() < 0.125 else rng.randrange(n) for _ in range(R)]
    if case["ranks"] == "mixed":
        rank = [rng.choice([r, r // 2, max(1, r - 3), max(1, r // 4)]) for _ in range(n)]
    else:
        rank = [r] * n
    return start, adapter, rank


def work(case):
    if case["op"] == "verify":
        # a sequence is settled by its first rejection: the rows behind it need not be read
        rows_t = rows_d = 0.0
        for n, temp in zip(_draft_lengths(case), _temperatures(case)):
            rows_t += sum(case["accept"] ** j for j in range(n + 1))
            if case["draft"] == "logits" and temp > 0:
                rows_d += sum(case["accept"] ** j for j in range(n))
        es = 4 if case["dtype"] == "f32" else 2
        # per logit: subtract, scale, exponential, add
        return {"bytes": int((rows_t + rows_d) * case["V"] * es), "flops": int(4 * (rows_t + rows_d) * case["V"])}
    start, adapter, rank = _requests(case)
    H, N, T = case["H"], case["N"], case["T"]
    used = {a for a, lo, hi in zip(adapter, start, start[1:]) if a >= 0 and hi > lo}
    ab = sum(rank[a] * (H + N) * 2 for a in used)
    tr = sum((hi - lo) * rank[a] for a, lo, hi in zip(adapter, start, start[1:]) if a >= 0)
    es = {"none": 0, "f32": 4, "bf16": 2}
    if case["op"] == "lora_forward":
        return {"bytes": T * H * 2 + ab + T * N * (es[case["base"]] + es[case["y"]]), "flops": 2 * tr * (H + N)}
    grads = case["adapters"] * case["r"] * (H + N) * 4
    return {"bytes": T * (H + N) * 2 + ab + T * H * (es[case["base"]] + 4) + grads, "flops": 6 * tr * (H + N)}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (_prepare_verify if case["op"] == "verify" else _prepare_lora)(case, g)


def _prepare_verify(case, g):
    dev, dt = "cuda", DTYPES[case["dtype"]]
    S, L, V = case["S"], case["max_draft"], case["V"]
    lens = _draft_lengths(case)
    start = torch.tensor([0] + lens, dtype=torch.int64, device=dev).cumsum(0)
    N = sum(lens)
    temps = torch.tensor(_temperatures(case), dtype=torch.float32, device=dev)
    # logits of a language model: a broad floor, a few dozen likely tokens and one that the model favours
    z = torch.empty(N + S, V + case["pad"], dtype=torch.float32, device=dev).normal_(0.0, 1.5, generator=g)[:, :V]
    few = min(32, V)
    where = torch.randint(V, (N + S, few), device=dev, generator=g)
    z.scatter_(1, where, torch.empty(N + S, few, device=dev).normal_(8.0, 2.0, generator=g))
    z.scatter_(1, where[:, :1], math.log(V) + 4.0)
    target = torch.empty(N + S, V + case["pad"], dtype=dt, device=dev)
    target.zero_()
    target[:, :V] = z
    # row of draft j of sequence i among the target's rows (which have one more per sequence)
    seq = torch.repeat_interleave(torch.arange(S, device=dev), torch.tensor(lens, device=dev))
    rows = torch.arange(N, device=dev) + seq
    draft = None
    if N == 0:
        tokens = torch.empty(0, dtype=torch.int64, device=dev)
        if case["draft"] == "logits":
            draft = torch.empty(0, V + case["pad"], dtype=dt, device=dev)[:, :V]
    elif case["draft"] == "logits":
        # the draft model: the target's logits with an error of its own
        noise = torch.empty(N, V, device=dev).normal_(0.0, 1.0, generator=g)
        wide = torch.empty(N, V + case["pad"], dtype=dt, device=dev)
        wide.zero_()
        wide[:, :V] = noise.add_(z[rows])
        draft = wide[:, :V]
        # drawn from the draft's distribution at the request's temperature
        t = temps[seq][:, None]
        race = torch.empty(N, V, device=dev).exponential_(generator=g).log_().neg_()
        tokens = torch.where(t > 0, draft.float() / t.clamp(min=0.1) + race, draft.float()).argmax(1)
        del race, noise
    else:
        likely = torch.rand(N, device=dev, generator=g) < 0.85
        tokens = torch.where(likely, target[:, :V][rows].argmax(1), torch.randint(V, (N,), device=dev, generator=g))
    out = {"n_accepted": torch.empty(S, dtype=torch.int64, device=dev),
           "tokens": torch.empty(S, L + 1, dtype=torch.int64, device=dev),
           "logprobs": torch.empty(S, L + 1, dtype=torch.float32, device=dev)}
    return {"op": "verify", "max_draft": L, "target": target[:, :V], "draft": draft, "draft_tokens": tokens,
            "draft_start": start, "temperature": temps if case["temps"] == "mixed" else None,
            "u_accept": torch.rand(N, device=dev, generator=g), "u_sample": torch.rand(S, device=dev, generator=g),
            "out": out}


def _prepare_lora(case, g):
    dev = "cuda"
    T, H, N, r, n = case["T"], case["H"], case["N"], case["r"], case["adapters"]
    start, adapter, rank = _requests(case)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=torch.float32, device=dev).normal_(0.0, std, generator=g).to(dtype)

    A = normal(n, r, H, std=H ** -0.5)
    B = normal(n, N, r, std=0.3)
    for a in range(n):  # adapters of a lower rank fill the stacked arrays with zeros
        A[a, rank[a]:] = 0
        B[a, :, rank[a]:] = 0
    state = {"op": case["op"], "x": normal(T, H), "A": A, "B": B,
             "adapter": torch.tensor(adapter, dtype=torch.int64, device=dev),
             "req_start": torch.tensor(start, dtype=torch.int64, device=dev),
             "rank": torch.tensor(rank, dtype=torch.int64, device=dev) if case["ranks"] == "mixed" else None,
             "scale": torch.empty(n, device=dev).uniform_(0.5, 2.0, generator=g)}
    if case["op"] == "lora_forward":
        state["base"] = None if case["base"] == "none" else normal(T, N, dtype=DTYPES[case["base"]])
        state["y"] = torch.empty(T, N, dtype=DTYPES[case["y"]], device=dev)
    else:
        state["grad_y"] = normal(T, N, std=0.01)
        state["base"] = None if case["base"] == "none" else normal(T, H, std=0.01, dtype=torch.float32)
        state["grad_x"] = torch.empty(T, H, dtype=torch.float32, device=dev)
        state["grad_A"] = torch.empty(n, r, H, dtype=torch.float32, device=dev)
        state["grad_B"] = torch.empty(n, N, r, dtype=torch.float32, device=dev)
    return state


# ---------------------------------------------------------------- one pass

def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "verify":
        return _plain_verify(state)
    return _plain_lora_forward(state) if state["op"] == "lora_forward" else _plain_lora_backward(state)


def _run_own(s):
    import cross_entropy_tv_amd as lx
    if s["op"] == "verify":
        o = s["out"]
        lx.lx_draft_verify(s["target"], s["draft"], s["draft_tokens"], s["draft_start"], s["max_draft"],
                           s["temperature"], s["u_accept"], s["u_sample"], o["n_accepted"], o["tokens"],
                           o["logprobs"])
        return o
    if s["op"] == "lora_forward":
        lx.lx_lora_forward(s["x"], s["A"], s["B"], s["adapter"], s["req_start"], s["scale"], s["rank"], s["base"],
                           s["y"])
        return s["y"]
    lx.lx_lora_backward(s["grad_y"], s["x"], s["A"], s["B"], s["adapter"], s["req_start"], s["scale"], s["rank"],
                        s["base"], s["grad_x"], s["grad_A"], s["grad_B"])
    return {"grad_x": s["grad_x"], "grad_A": s["grad_A"], "grad_B": s["grad_B"]}


def _plain_verify(s):
    """In float64: a token is drawn by comparing a running sum over the vocabulary with a random number, and the
    sums' borders lie closer together than fp32 resolves."""
    target, draft, tokens, start, L = s["target"], s["draft"], s["draft_tokens"], s["draft_start"], s["max_draft"]
    S, N, V = start.shape[0] - 1, tokens.shape[0], target.shape[1]
    dev = target.device
    n = start[1:] - start[:-1]
    seq_t = torch.repeat_interleave(torch.arange(S, device=dev), n + 1, output_size=N + S)
    seq_d = torch.repeat_interleave(torch.arange(S, device=dev), n, output_size=N)
    temp = torch.ones(S, device=dev) if s["temperature"] is None else s["temperature"]
    greedy = temp == 0
    temp = torch.where(greedy, 1.0, temp.double())

    def softmax(rows, seq):
        z = rows.double()
        z = (z - z.amax(1, keepdim=True)) / temp[seq][:, None]
        e = torch.exp(z)
        return e / e.sum(1, keepdim=True)

    best = target.float().argmax(1)  # the first of equals
    onehot = torch.arange(V, device=dev)[None, :]
    p = softmax(target, seq_t)
    g = greedy[seq_t]
    p = torch.where(g[:, None], (onehot == best[:, None]).double(), p)
    # drafted token j of sequence i faces the target's row start[i] + i + j
    rows = torch.arange(N, device=dev) + seq_d
    pos = torch.arange(N, device=dev) - start[:-1][seq_d]
    ok_token = (tokens >= 0) & (tokens < V)
    x = torch.where(ok_token, tokens, 0)
    px = torch.where(ok_token, p[rows, x], 0.0)
    if draft is None:
        q = None
        qx = torch.ones(N, dtype=torch.float64, device=dev)
    else:
        q = softmax(draft, seq_d)
        qx = q[torch.arange(N, device=dev), x]
    r = s["u_accept"].double()
    accept = torch.where(g[rows], px > 0, r * qx < px)
    table = torch.zeros(S, L + 1, dtype=torch.bool, device=dev)
    table[seq_d, pos] = accept
    accepted = table.long().cumprod(1).sum(1)
    # the token behind the accepted ones: from what the target has beyond the draft, or from the target after the last
    row = start[:-1] + torch.arange(S, device=dev) + accepted
    rest = p[row]
    rejected = (accepted < n) & ~greedy
    if N:
        d = (start[:-1] + accepted).clamp(max=N - 1)
        beyond = (rest - q[d]).clamp(min=0) if q is not None else torch.where(
            (onehot == x[d][:, None]) & ok_token[d][:, None], 0.0, rest)
        rest = torch.where((rejected & (beyond.sum(1) > 0))[:, None], beyond, rest)
    run_sum = rest.cumsum(1)
    goal = s["u_sample"].double() * run_sum[:, -1]
    drawn = (run_sum <= goal[:, None]).sum(1)
    last = V - 1 - rest.flip(1).gt(0).to(torch.uint8).argmax(1)
    drawn = torch.minimum(drawn, last)
    out_tokens = torch.full((S, L + 1), -1, dtype=torch.int64, device=dev)
    out_logp = torch.zeros(S, L + 1, dtype=torch.float64, device=dev)
    keep = pos < accepted[seq_d]
    out_tokens[seq_d, pos] = torch.where(keep, tokens, -1)
    out_logp[seq_d, pos] = torch.where(keep, torch.log(px), 0.0)
    every = torch.arange(S, device=dev)
    out_tokens[every, accepted] = drawn
    out_logp[every, accepted] = torch.log(p[row, drawn])
    return {"n_accepted": accepted, "tokens": out_tokens, "logprobs": out_logp.float()}


def _columns(s):
    """The stacked adapters as one wide matrix and, for each row, the factor of each of its columns: the adapter's
    scale on the columns of the row's own adapter below its rank, 0 elsewhere."""
    A, B = s["A"], s["B"]
    n, r, H = A.shape
    T, dev = s["x"].shape[0], A.device
    lens = s["req_start"][1:] - s["req_start"][:-1]
    row_adapter = torch.repeat_interleave(s["adapter"], lens, output_size=T)
    mine = row_adapter[:, None] == torch.arange(n, device=dev)[None, :]
    factor = torch.where(mine, s["scale"][None, :], 0.0)
    factor = factor[:, :, None].expand(T, n, r)
    if s["rank"] is not None:
        factor = torch.where(torch.arange(r, device=dev)[None, :] < s["rank"][:, None], factor, 0.0)
    wide_A = A.float().reshape(n * r, H)
    wide_B = B.float().transpose(1, 2).reshape(n * r, B.shape[1])
    return wide_A, wide_B, factor.reshape(T, n * r)


def _plain_lora_forward(s):
    wide_A, wide_B, factor = _columns(s)
    y = ((s["x"].float() @ wide_A.t()) * factor) @ wide_B
    if s["base"] is not None:
        y = y + s["base"].float()
    return y.to(s["y"].dtype)


def _plain_lora_backward(s):
    wide_A, wide_B, factor = _columns(s)
    n, r, H = s["A"].shape
    N = s["B"].shape[1]
    x, dy = s["x"].float(), s["grad_y"].float()
    u = (x @ wide_A.t()) * factor
    v = (dy @ wide_B.t()) * factor
    grad_x = v @ wide_A
    if s["base"] is not None:
        grad_x = grad_x + s["base"]
    return {"grad_x": grad_x, "grad_A": (v.t() @ x).reshape(n, r, H),
            "grad_B": (u.t() @ dy).reshape(n, r, N).transpose(1, 2).contiguous()}


# ---------------------------------------------------------------- in 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_verify(case, s) if case["op"] == "verify" else _exact_lora(case, s)


def _exact_verify(case, s):
    S, L, V = case["S"], case["max_draft"], case["V"]
    lens, temps = _draft_lengths(case), _temperatures(case)
    n_accepted = torch.zeros(S, dtype=torch.int64)
    tokens = torch.full((S, L + 1), -1, dtype=torch.int64)
    logprobs = torch.zeros(S, L + 1, dtype=torch.float64)
    drafted, u_accept, u_sample = s["draft_tokens"].tolist(), s["u_accept"].tolist(), s["u_sample"].tolist()
    first = 0
    for i in range(S):
        def log_p(logits):
            z = logits.double()
            if temps[i] == 0.0:
                at = int((z == z.max()).nonzero()[0])
                lp = torch.full_like(z, -math.inf)
                lp[at] = 0.0
                return lp
            # the temperature as the fp32 number that the operator is given
            z = z / float(torch.tensor(temps[i], dtype=torch.float32))
            return z - torch.logsumexp(z, 0)

        j = 0
        while True:
            lp = log_p(s["target"][first + i + j])
            if j == lens[i]:
                mass = lp.exp()
                break
            x = drafted[first + j]
            if temps[i] == 0.0:
                ok, mass = float(lp[x]) == 0.0, lp.exp()
            elif s["draft"] is None:
                ok = u_accept[first + j] < math.exp(float(lp[x]))
                mass = lp.exp()
                mass[x] = 0.0
            else:
                lq = log_p(s["draft"][first + j])
                ok = u_accept[first + j] * math.exp(float(lq[x])) < math.exp(float(lp[x]))
                mass = (lp.exp() - lq.exp()).clamp(min=0.0)
            if not ok:
                break
            tokens[i, j] = x
            logprobs[i, j] = float(lp[x])
            j += 1
        if float(mass.sum()) <= 0.0:
            mass = lp.exp()
        sums = torch.cumsum(mass, 0)
        at = int(torch.searchsorted(sums, u_sample[i] * sums[-1], right=True))
        at = min(at, int(mass.nonzero()[-1]))
        n_accepted[i] = j
        tokens[i, j] = at
        logprobs[i, j] = float(lp[at])
        first += lens[i]
    return {"n_accepted": n_accepted, "tokens": tokens, "logprobs": logprobs}


def _exact_lora(case, s):
    start, adapter, rank = _requests(case)
    scale = s["scale"].double()
    x = s["x"].double()
    base = None if s["base"] is None else s["base"].double()
    spans = [(lo, hi, a) for lo, hi, a in zip(start, start[1:], adapter) if a >= 0 and hi > lo]
    if case["op"] == "lora_forward":
        y = torch.zeros(case["T"], case["N"], dtype=torch.float64, device=x.device) if base is None else base
        for lo, hi, a in spans:
            down = s["A"][a, :rank[a]].double()
            up = s["B"][a, :, :rank[a]].double()
            y[lo:hi] += scale[a] * (x[lo:hi] @ down.t() @ up.t())
        return y
    dy = s["grad_y"]
    grad_x = torch.zeros_like(x) if base is None else base
    grad_A = torch.zeros(s["A"].shape, dtype=torch.float64, device=x.device)
    grad_B = torch.zeros(s["B"].shape, dtype=torch.float64, device=x.device)
    for lo, hi, a in spans:
        down = s["A"][a, :rank[a]].double()
        up = s["B"][a, :, :rank[a]].double()
        d = dy[lo:hi].double()
        back = scale[a] * (d @ up)
        grad_x[lo:hi] += back @ down
        grad_A[a, :rank[a]] += back.t() @ x[lo:hi]
        grad_B[a, :, :rank[a]] += d.t() @ (scale[a] * (x[lo:hi] @ down.t()))
    return {"grad_x": grad_x, "grad_A": grad_A, "grad_B": grad_B}
