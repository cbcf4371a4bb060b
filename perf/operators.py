"""The prompt and single-token operators of a hybrid model's layers, as cases to time.

``run`` takes one pass through an operator on the state that ``prepare`` made: the
plain form (elementary torch operations in 32 bits, rounded once at the end) or,
with ``own`` set, the library's kernels through their public entry points.

Shapes: the linear-attention layer of the gated-delta-rule workloads (32 value
heads, 16 query/key heads, 128 x 128 states), the Mamba2-2.7B layer (80 heads, one
group, 64 x 128 states), and the hybrid model's attention layer (32 query heads, 8
key/value heads, head dim 128).
"""
import math

import torch

own = False

WORKSPACE_BYTES = 64 << 20           # scratch that a serving program keeps for its calls

LINEAR_HEADS = ((32, 16, 128), (80, 1, 64), (16, 16, 128), (8, 2, 64), (5, 5, 96))   # Hv, Hk, dv
ATTENTION_HEADS = ((32, 8), (16, 16), (8, 1), (12, 4), (64, 8))                      # Hq, Hkv


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # One long prompt through a linear-attention layer: few heads, a long axis.
        dict(name="linear_prompt_long", op="linear_prompt", lens="8192", heads_v=32, heads_k=16, dk=128, dv=128,
             dtype="bf16", skip=False, start=False),
        # A packed batch of prompts of very different lengths through a Mamba2 layer (decay
        # exp(dt A), write strength dt, skip D), each continuing from a cached state.
        dict(name="linear_prompt_packed", op="linear_prompt", lens="1,37,2048,500,129,64,1000,3,255,777,128,14",
             heads_v=80, heads_k=1, dk=128, dv=64, dtype="bf16", skip=True, start=True),
        # A short prompt in fp32, as a precision check of a small model runs it.
        dict(name="linear_prompt_fp32", op="linear_prompt", lens="96,33", heads_v=8, heads_k=4, dk=64, dv=32,
             dtype="f32", skip=True, start=True),
        # One new token of one sequence: the smallest call of a Mamba2 layer.
        dict(name="linear_step_single", op="linear_step", batch=1, heads_v=80, heads_k=1, dk=128, dv=64, dtype="bf16",
             skip=True),
        # One new token of each sequence of a serving batch.
        dict(name="linear_step_batch", op="linear_step", batch=64, heads_v=32, heads_k=16, dk=128, dv=128,
             dtype="bf16", skip=False),
        # One long prompt through the attention layer.
        dict(name="prompt_attention_long", op="prompt_attention", lens="8192", heads_q=32, heads_kv=8),
        # A packed batch of prompts of very different lengths.
        dict(name="prompt_attention_packed", op="prompt_attention", lens="1500,1,333,64,977,129,700,18,1025,256,90,511",
             heads_q=32, heads_kv=8),
        # One short prompt, where latency counts.
        dict(name="prompt_attention_short", op="prompt_attention", lens="37", heads_q=32, heads_kv=8),
        # One new token over one very long cache.
        dict(name="paged_attention_long", op="paged_attention", lens="131065", heads_q=32, heads_kv=8, page=64,
             cache="bf16"),
        # One new token of each sequence of a serving batch over an 8-bit cache in small
        # pages, lengths from one token (and one empty slot) up.
        dict(name="paged_attention_batch", op="paged_attention", lens="spread:64:4096", heads_q=32, heads_kv=8, page=16,
             cache="e4m3"),
        # A prompt's keys and values quantised into pages, and read back for the tree's attention.
        dict(name="cache_prompt_e4m3", op="cache", lens="5000,3001,191", heads_kv=8, page=64, cache="e4m3", read=True),
        # One new token of each sequence written into a bf16 cache.
        dict(name="cache_step_bf16", op="cache", lens="ones:64:512", heads_kv=8, page=16, cache="bf16", read=False),
    ]


def _split_total(rng, total, batch):
    batch = min(batch, total)
    cuts = sorted(rng.sample(range(1, total), batch - 1)) if batch > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _log_size(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("linear_prompt", "linear_step", "prompt_attention", "paged_attention", "cache"))
    if op == "linear_prompt":
        heads_v, heads_k, dv = rng.choice(LINEAR_HEADS)
        f32 = rng.random() < 0.25
        total = _log_size(rng, 2, 600 if f32 else 8192 if heads_v <= 32 else 4900)
        lens = _split_total(rng, total, rng.randint(1, 12))
        return dict(op=op, lens=",".join(map(str, lens)), heads_v=heads_v, heads_k=heads_k, dk=128, dv=dv,
                    dtype="f32" if f32 else "bf16", skip=rng.random() < 0.5, start=rng.random() < 0.5)
    if op == "linear_step":
        heads_v, heads_k, dv = rng.choice(LINEAR_HEADS)
        return dict(op=op, batch=_log_size(rng, 1, 64), heads_v=heads_v, heads_k=heads_k, dk=128, dv=dv,
                    dtype=rng.choice(("bf16", "bf16", "f32")), skip=rng.random() < 0.5)
    if op == "prompt_attention":
        heads_q, heads_kv = rng.choice(ATTENTION_HEADS)
        total = _log_size(rng, 2, 8192 if heads_q <= 32 else 5700)
        lens = _split_total(rng, total, rng.randint(1, 12))
        return dict(op=op, lens=",".join(map(str, lens)), heads_q=heads_q, heads_kv=heads_kv)
    if op == "paged_attention":
        heads_q, heads_kv = rng.choice(ATTENTION_HEADS)
        total = _log_size(rng, 2, (1 << 20) // heads_kv)
        batch = rng.randint(1, 48)
        lens = _split_total(rng, total, batch)
        return dict(op=op, lens=",".join(map(str, lens)), heads_q=heads_q, heads_kv=heads_kv,
                    page=rng.choice((8, 16, 32, 48, 64, 128)), cache=rng.choice(("bf16", "e4m3")))
    total = _log_size(rng, 2, 8192)
    lens = _split_total(rng, total, rng.randint(1, 12))
    return dict(op=op, lens=",".join(map(str, lens)), heads_kv=rng.choice((1, 4, 8)),
                page=rng.choice((8, 16, 32, 48, 64, 128)), cache=rng.choice(("bf16", "e4m3")), read=True)


def _lens(case):
    """The sequences' lengths: given, or a spread over a range with one empty slot, or ones."""
    text = case["lens"]
    if text.startswith("spread:"):
        n, top = map(int, text.split(":")[1:])
        return [0] + [max(1, round(top * ((i * 37) % n) / (n - 1))) for i in range(1, n)]
    if text.startswith("ones:"):
        return [1] * int(text.split(":")[1])
    return [int(t) for t in text.split(",")]


def _held(case):
    """Tokens that the cache holds before the write."""
    n, text = len(_lens(case)), case["lens"]
    if text.startswith("ones:"):
        top = int(text.split(":")[2])
        return [(i * 53) % (top - 1) for i in range(n)]
    return [(i * 29) % 100 for i in range(n)]


# ------------------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return _i32(at)


def _linear_inputs(case, rows, g):
    """Gates of a Mamba2 layer (dt = softplus(N(-2, 0.5)), decay exp(dt A), A in -[1, 16]);
    values ~ N(0, 1), keys and queries ~ N(0, 1) / sqrt(dk)."""
    t = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    hv, hk, dk, dv = case["heads_v"], case["heads_k"], case["dk"], case["dv"]
    normal = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    dt = torch.nn.functional.softplus(normal(rows, hv) * 0.5 - 2)
    decay = torch.exp(torch.rand(hv, generator=g, device="cuda") * math.log(16.0))
    return dict(q=(normal(rows, hk, dk) / math.sqrt(dk)).to(t), k=(normal(rows, hk, dk) / math.sqrt(dk)).to(t),
                v=normal(rows, hv, dv).to(t), alpha=torch.exp(-dt * decay), beta=dt,
                skip=normal(hv) if case["skip"] else None)


def _page_table(lens, page, g):
    """Pages handed out in random order, as a long-running server's free list gives them."""
    need = [-(-n // page) for n in lens]
    total = max(1, sum(need))
    order = torch.randperm(total + 3, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(lens), max(1, max(need))), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total + 3


def prepare(case, seed):
    g = _gen(seed)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    op = case["op"]
    s = dict(case=case, workspace=torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device="cuda"),
             err=torch.zeros(4, dtype=torch.int32, device="cuda"))
    if op in ("linear_prompt", "linear_step"):
        lens = _lens(case) if op == "linear_prompt" else [1] * case["batch"]
        s.update(_linear_inputs(case, sum(lens), g))
        state = (len(lens), case["heads_v"], case["dv"], case["dk"])
        given = op == "linear_step" or case["start"]
        s.update(S0=torch.randn(state, generator=g, device="cuda") * 0.1 if given else None,
                 offsets=_offsets(lens), o=torch.empty_like(s["v"]), S_new=torch.empty(state, device="cuda"))
        return s
    if op == "prompt_attention":
        lens = _lens(case)
        n = sum(lens)
        s.update(q=normal(n, case["heads_q"], 128), k=normal(n, case["heads_kv"], 128),
                 v=normal(n, case["heads_kv"], 128), offsets=_offsets(lens), scale=1.0 / math.sqrt(128))
        s["o"] = torch.empty_like(s["q"])
        return s
    hkv, page, lens = case["heads_kv"], case["page"], _lens(case)
    if op == "paged_attention":
        table, n_pages = _page_table(lens, page, g)
        s.update(q=normal(len(lens), case["heads_q"], 128), k_pages=normal(n_pages, hkv, page, 128),
                 v_pages=normal(n_pages, hkv, page, 128), k_scales=None, v_scales=None, table=table,
                 lens=_i32(lens), scale=1.0 / math.sqrt(128))
        s["o"] = torch.empty_like(s["q"])
        if case["cache"] == "e4m3":
            s["k_pages"], s["k_scales"] = _quantise(s["k_pages"])
            s["v_pages"], s["v_scales"] = _quantise(s["v_pages"])
        return s
    held = _held(case)
    ends = [a + b for a, b in zip(held, lens)]
    table, n_pages = _page_table(ends, page, g)
    # Keys carry a few strong channels, values are even: what a cache holds in earnest.
    strength = torch.exp(torch.randn(128, generator=g, device="cuda") * 0.7)
    s.update(k=(torch.randn((sum(lens), hkv, 128), generator=g, device="cuda") * strength).to(torch.bfloat16),
             v=normal(sum(lens), hkv, 128), offsets=_offsets(lens), start=_i32(held), ends=_i32(ends), table=table,
             k_pages=normal(n_pages, hkv, page, 128), v_pages=normal(n_pages, hkv, page, 128),
             k_scales=None, v_scales=None, k_ctx=None, v_ctx=None)
    if case["cache"] == "e4m3":
        s["k_pages"], s["k_scales"] = _quantise(s["k_pages"])
        s["v_pages"], s["v_scales"] = _quantise(s["v_pages"])
    if case["read"]:
        s["k_ctx"] = torch.zeros((len(lens), max(ends), hkv, 128), dtype=torch.bfloat16, device="cuda")
        s["v_ctx"] = torch.zeros_like(s["k_ctx"])
    return s


# ------------------------------------------------------------------------------ plain forms

def _rows_of(offsets, total):
    """The sequence of each packed row, and its position there."""
    at = torch.arange(total, device="cuda")
    seq = torch.searchsorted(offsets[1:].long(), at, right=True)
    return seq, at - offsets.long()[seq]


def _linear_prompt(s):
    """o_i = sum_{j <= i} (g_i / g_j) b_j (q_i . k_j) v_j + g_i S0 q_i + D v_i with g the running
    product of alpha; the exponents of the ratios are summed and subtracted in 64 bits."""
    total, hv = s["v"].shape[:2]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    rep = hv // q.shape[1]
    q, k, v = (t.transpose(0, 1) for t in (q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1), v))
    seq, _ = _rows_of(s["offsets"], total)
    logs = torch.log(s["alpha"].double()).cumsum(0)
    before = torch.cat((torch.zeros_like(logs[:1]), logs))
    first, last = before[s["offsets"][:-1].long()], before[s["offsets"][1:].long()]     # [b, Hv]
    logs_h = logs.T
    at = torch.arange(total, device="cuda")
    seen = (seq[:, None] == seq[None, :]) & (at[:, None] >= at[None, :])
    ratio = torch.exp((logs_h[:, :, None] - logs_h[:, None, :]).masked_fill_(~seen, -math.inf).float())
    o = torch.matmul(torch.matmul(q, k.transpose(1, 2)) * ratio * s["beta"].T[:, None, :], v)
    del ratio
    one_seq = (torch.arange(first.shape[0], device="cuda")[:, None] == seq[None, :])    # [b, total]
    weight = torch.exp(last[seq] - logs).float() * s["beta"]                           # [total, Hv]
    mine = one_seq[:, None, :, None] * (weight.T[:, :, None] * v)[None]                 # [b, Hv, total, dv]
    S = torch.matmul(mine.transpose(2, 3), k[None])
    if s["S0"] is not None:
        S = S + torch.exp(last - first).float()[:, :, None, None] * s["S0"]
        per_seq = torch.matmul(q[None], s["S0"].transpose(2, 3))                        # [b, Hv, total, dv]
        root = per_seq.permute(2, 0, 1, 3)[at, seq]                                     # [total, Hv, dv]
        o = o + (torch.exp(logs - first[seq]).float()[:, :, None] * root).transpose(0, 1)
    if s["skip"] is not None:
        o = o + s["skip"][:, None, None] * v
    return o.transpose(0, 1).to(s["v"].dtype).contiguous(), S


def _linear_step(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    rep = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    S = s["alpha"][:, :, None, None] * s["S0"] + (s["beta"][:, :, None] * v)[:, :, :, None] * k[:, :, None, :]
    o = torch.matmul(S, q[..., None])[..., 0]
    if s["skip"] is not None:
        o = o + s["skip"][:, None] * v
    return o.to(s["v"].dtype), S


def _prompt_attention(s):
    total, hq = s["q"].shape[:2]
    rep = hq // s["k"].shape[1]
    q = s["q"].float().transpose(0, 1)
    k, v = (t.float().repeat_interleave(rep, 1).transpose(0, 1) for t in (s["k"], s["v"]))
    seq, _ = _rows_of(s["offsets"], total)
    at = torch.arange(total, device="cuda")
    hidden = (seq[:, None] != seq[None, :]) | (at[:, None] < at[None, :])
    w = torch.matmul(q, k.transpose(1, 2)).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
    w = w.sub_(w.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(w, v) / w.sum(-1, keepdim=True)
    return o.transpose(0, 1).to(s["q"].dtype).contiguous()


def _power_of_two(biased):
    """2^(biased - 127) in 32 bits, exactly, by its exponent field (1 to 254)."""
    return (biased.to(torch.int32) << 23).view(torch.float32)


def _values(pages, scales):
    """The values that pages stand for, in 32 bits: 8-bit elements times 2^(scale - 127)."""
    x = pages.float()
    return x if scales is None else x * _power_of_two(scales)[..., None]


def _paged_attention(s):
    b, hq = s["q"].shape[:2]
    table = s["table"].long()
    hkv, page = s["k_pages"].shape[1:3]
    rep, cap = hq // hkv, table.shape[1] * page
    k, v = (_values(p[table], sc[table] if sc is not None else None).transpose(1, 2).reshape(b, hkv, cap, 128)
            for p, sc in ((s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"])))
    hidden = torch.arange(cap, device="cuda")[None, :] >= s["lens"][:, None]            # [b, cap]
    q = s["q"].float().reshape(b, hkv, rep, 128)
    w = (torch.matmul(q, k.transpose(2, 3)) * s["scale"]).masked_fill(hidden[:, None, None, :], -math.inf)
    top = w.amax(-1, keepdim=True)
    w = torch.exp(w - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, v.masked_fill(hidden[:, None, :, None], 0.0)) / torch.where(total == 0, torch.ones_like(total), total)
    return o.reshape(b, hq, 128).to(s["q"].dtype)


def _quantise(x):
    """bf16 rows of 128 -> (e4m3 rows, one power-of-two scale each, as its exponent plus 127):
    the least scale that brings the row's largest magnitude to 448 or below."""
    x = x.float()
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)                                  # top = m 2^e, m in [0.5, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8)                # 448 = 0.875 2^9
    e = torch.where(top == 0, torch.full_like(e, -118), e).clamp(-118, 119)
    return (x * _power_of_two(127 - e)[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _cache(s):
    page, hkv = s["k_pages"].shape[2], s["k_pages"].shape[1]
    seq, pos = _rows_of(s["offsets"], s["k"].shape[0])
    pos = pos + s["start"].long()[seq]
    where = s["table"].long()[seq, pos // page]
    for new, pages, scales in ((s["k"], s["k_pages"], s["k_scales"]), (s["v"], s["v_pages"], s["v_scales"])):
        if scales is None:
            pages[where, :, pos % page] = new
        else:
            x, e = _quantise(new)
            pages.view(torch.uint8)[where, :, pos % page] = x.view(torch.uint8)
            scales[where, :, pos % page] = e
    if s["k_ctx"] is None:
        return s["k_pages"], s["v_pages"]
    b, cap = s["k_ctx"].shape[:2]
    at = torch.arange(cap, device="cuda")
    valid = (at[None, :] < s["ends"][:, None])[:, :, None, None]
    src = s["table"].long()[:, (at // page).clamp(max=s["table"].shape[1] - 1)]         # [b, cap]
    for ctx, pages, scales in ((s["k_ctx"], s["k_pages"], s["k_scales"]), (s["v_ctx"], s["v_pages"], s["v_scales"])):
        got = _values(pages.view(torch.uint8).view(pages.dtype)[src, :, at % page],
                      None if scales is None else scales[src, :, at % page])
        ctx.copy_(torch.where(valid, got, ctx.float()))
    return s["k_ctx"], s["v_ctx"]


PLAIN = dict(linear_prompt=_linear_prompt, linear_step=_linear_step, prompt_attention=_prompt_attention,
             paged_attention=_paged_attention, cache=_cache)


def _run_own(s):
    from hybrid_packed_tree_b200 import stree
    op = s["case"]["op"]
    if op == "linear_prompt":
        stree.stree_linear_prompt(s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["offsets"], s["o"], S0=s["S0"],
                                  S_new=s["S_new"], skip=s["skip"], err_out=s["err"], workspace=s["workspace"])
        return s["o"], s["S_new"]
    if op == "linear_step":
        stree.stree_linear_step(s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["S0"], s["o"], s["S_new"],
                                skip=s["skip"])
        return s["o"], s["S_new"]
    if op == "prompt_attention":
        return stree.stree_prompt_attention(s["q"], s["k"], s["v"], s["offsets"], s["o"], s["scale"], err_out=s["err"])
    if op == "paged_attention":
        return stree.stree_paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["o"],
                                           s["scale"], k_scales=s["k_scales"], v_scales=s["v_scales"],
                                           err_out=s["err"], workspace=s["workspace"])
    stree.stree_cache_write(s["k"], s["v"], s["offsets"], s["start"], s["table"], s["k_pages"], s["v_pages"],
                            k_scales=s["k_scales"], v_scales=s["v_scales"], err_out=s["err"])
    if s["k_ctx"] is None:
        return s["k_pages"], s["v_pages"]
    stree.stree_cache_read(s["k_pages"], s["v_pages"], s["table"], s["ends"], s["k_ctx"], s["v_ctx"],
                           k_scales=s["k_scales"], v_scales=s["v_scales"], err_out=s["err"])
    return s["k_ctx"], s["v_ctx"]


def run(state):
    if own:
        return _run_own(state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------------------ what a pass has to do

def work(case):
    op = case["op"]
    if op in ("linear_prompt", "linear_step"):
        lens = _lens(case) if op == "linear_prompt" else [1] * case["batch"]
        n, b, size = sum(lens), len(lens), 2 if case["dtype"] == "bf16" else 4
        hv, hk, dk, dv = case["heads_v"], case["heads_k"], case["dk"], case["dv"]
        states = 2 if op == "linear_step" or case["start"] else 1
        return dict(bytes=size * n * (2 * hk * dk + 2 * hv * dv) + 8 * n * hv + states * 4 * b * hv * dv * dk
                    + (4 * hv if case["skip"] else 0), flops=4 * n * hv * dk * dv)
    if op == "prompt_attention":
        lens, hq, hkv = _lens(case), case["heads_q"], case["heads_kv"]
        return dict(bytes=2 * 128 * sum(lens) * (2 * hq + 2 * hkv),
                    flops=4 * 128 * hq * sum(n * (n + 1) // 2 for n in lens))
    lens, hkv = _lens(case), case["heads_kv"]
    row = 128 * 2 if case["cache"] == "bf16" else 128 + 1
    if op == "paged_attention":
        hq = case["heads_q"]
        return dict(bytes=2 * row * hkv * sum(lens) + 2 * 2 * 128 * hq * len(lens) + 4 * len(lens),
                    flops=4 * 128 * hq * sum(lens))
    ends = [a + b for a, b in zip(_held(case), lens)] if case["read"] else []
    return dict(bytes=2 * hkv * (sum(lens) * (256 + row) + sum(ends) * (256 + row)), flops=0)


# ------------------------------------------------------------------------------ the definitions in 64 bits

def _exact_linear(s, lens):
    """The recurrence token by token: S <- alpha S + beta v k^T, o = S q + D v."""
    b, (hv, dv), dk = len(lens), s["v"].shape[1:], s["k"].shape[2]
    S = torch.zeros((b, hv, dv, dk), dtype=torch.float64, device="cuda") if s["S0"] is None else s["S0"].double()
    o = torch.empty(s["v"].shape, dtype=torch.float64, device="cuda")
    group = torch.arange(hv, device="cuda") // (hv // s["k"].shape[1])
    begin = s["offsets"][:-1].long()
    order = sorted(range(b), key=lambda i: -lens[i])
    for t in range(max(lens)):
        live = torch.tensor([i for i in order if lens[i] > t], device="cuda") if b > 1 else torch.zeros(1, dtype=torch.long, device="cuda")
        rows = begin[live] + t
        v, q, k = s["v"][rows].double(), s["q"][rows].double()[:, group], s["k"][rows].double()[:, group]
        now = S[live] * s["alpha"][rows].double()[:, :, None, None]
        now += (s["beta"][rows].double()[:, :, None] * v)[..., None] * k[:, :, None, :]
        S[live] = now
        o[rows] = (now * q[:, :, None, :]).sum(-1) + (s["skip"].double()[:, None] * v if s["skip"] is not None else 0.0)
    return o, S


def _softmax_rows(scores):
    e = torch.exp(scores - scores.max(-1, keepdim=True).values)
    return e / e.sum(-1, keepdim=True)


def _exact_prompt(s, lens):
    o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    rep, at = s["q"].shape[1] // s["k"].shape[1], 0
    for n in lens:
        later = torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1)
        for h in range(s["q"].shape[1]):
            q, k, v = s["q"][at:at + n, h].double(), s["k"][at:at + n, h // rep].double(), s["v"][at:at + n, h // rep].double()
            o[at:at + n, h] = _softmax_rows((q @ k.T * s["scale"]).masked_fill_(later, -math.inf)) @ v
        at += n
    return o


def _two_to(e):
    """2^e in 64 bits, exactly (a power function may be off by a step)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _stands_for(pages, scales, ids, n):
    x = pages[ids].double()                                  # [pages, Hkv, page, 128]
    if scales is not None:
        x = x * _two_to(scales[ids].int() - 127)[..., None]
    return x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, 128)[:, :n]


def _exact_paged(s, lens):
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    page, hkv = s["k_pages"].shape[2], s["k_pages"].shape[1]
    for b, n in enumerate(lens):
        if n == 0:
            continue
        ids = s["table"][b, :-(-n // page)].long()
        k, v = _stands_for(s["k_pages"], s["k_scales"], ids, n), _stands_for(s["v_pages"], s["v_scales"], ids, n)
        q = s["q"][b].double().reshape(hkv, -1, 128)
        o[b] = (_softmax_rows(q @ k.transpose(1, 2) * s["scale"]) @ v).reshape(-1, 128)
    return o


def _exact_cached(x, cache):
    """What a row is after the cache: itself, or the nearest e4m3 values under its scale."""
    x = x.double()
    if cache == "bf16":
        return x
    top = x.abs().amax(-1, keepdim=True)
    scale = torch.full_like(top, 2.0 ** -118)
    for e in range(-117, 120):
        scale = torch.where(top > 448.0 * scale, torch.full_like(top, 2.0 ** e), scale)
    y = x / scale
    step = _two_to(torch.frexp(y.abs().clamp(min=2.0 ** -6)).exponent - 4)
    return torch.round(y / step) * step * scale              # torch.round: ties to even


def _exact_cache(s, case, lens):
    held, page = _held(case), case["page"]
    new = [_exact_cached(s[n], case["cache"]) for n in ("k", "v")]
    if not case["read"]:
        outs = [s["k_pages"].double(), s["v_pages"].double()]
        at = 0
        for b, n in enumerate(lens):
            for i in range(n):
                p = held[b] + i
                for out, x in zip(outs, new):
                    out[int(s["table"][b, p // page]), :, p % page] = x[at + i]
            at += n
        return outs
    outs, at = [s["k_ctx"].double(), s["v_ctx"].double()], 0
    for b, n in enumerate(lens):
        ids = s["table"][b, :-(-(held[b] + n) // page)].long()
        for out, x, name in zip(outs, new, ("k", "v")):
            old = _stands_for(s[name + "_pages"], s[name + "_scales"], ids, held[b])
            out[b, :held[b]] = old.transpose(0, 1)
            out[b, held[b]:held[b] + n] = x[at:at + n]
        at += n
    return outs


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("linear_prompt", "linear_step"):
        return _exact_linear(s, _lens(case) if op == "linear_prompt" else [1] * case["batch"])
    if op == "prompt_attention":
        return _exact_prompt(s, _lens(case))
    if op == "paged_attention":
        return _exact_paged(s, _lens(case))
    return _exact_cache(s, case, _lens(case))
