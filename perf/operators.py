"""Timed cases of the softmax-attention layer that a hybrid stack puts beside the Gated Delta
Rule-2 mixer: per-head norms and the position rotation of queries and keys (forward and
backward), the serving prologue that also writes keys and values into a paged 8-bit cache, and
attention over that cache.

Each case runs either in plain torch operations in 32 bits (`own` false) or through the
library's entry points (`own` true) on the same inputs.

The cache. Blocks of 64 tokens; for every block and key/value head
    k       [P, Hk, 64, d] e4m3, token-major
    v       [P, Hk, d, 64] e4m3, channel-major; token t of the block lies at column
            (t // 4 % 4) * 16 + (t // 16) * 4 + t % 4
    k_scale, v_scale [P, Hk] fp32, powers of two
and the value held is e4m3 * scale. block_table [N, MB] int32 names the blocks of each
sequence, seq_lens [N] int32 its tokens, the ones of the call included.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 64
EPS = 1e-6


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # training, one layer of the 1.3B-layer batch (8 sequences of 2048 tokens, 16 heads of
        # 128), queries and keys with as many heads
        dict(name="norm_rope_train_layer", op="rope_fwd", B=8, T=2048, Hq=16, Hk=16, d=128, rot=128,
             interleaved=False, dtype="bf16", far=0),
        # the fp32 check configuration of the library's tests: small, partial rotation,
        # neighbouring pairs, positions far into a long text
        dict(name="norm_rope_small_fp32", op="rope_fwd", B=1, T=255, Hq=2, Hk=2, d=64, rot=32,
             interleaved=True, dtype="fp32", far=1000000),
        # the gradient of the training layer, grouped heads
        dict(name="norm_rope_grad_layer", op="rope_bwd", B=8, T=2048, Hq=16, Hk=4, d=128, rot=128,
             interleaved=False, dtype="bf16", far=0),
        # gradient in fp32 of an odd batch
        dict(name="norm_rope_grad_odd_fp32", op="rope_bwd", B=3, T=411, Hq=6, Hk=3, d=64, rot=64,
             interleaved=True, dtype="fp32", far=0),
        # one decoded token of 256 sequences: norms, rotation, one row into each cache
        dict(name="prologue_decode_256", op="prologue", N=256, L=1, packed=False, ctx=4096, lens_seed=1,
             Hq=16, Hk=4, d=128, rot=128, interleaved=False),
        # prompts of 8 packed sequences of unequal lengths into an empty cache
        dict(name="prologue_prompt_packed", op="prologue", N=8, L=2048, packed=True, ctx=0, lens_seed=2,
             Hq=16, Hk=4, d=128, rot=128, interleaved=False),
        # one decoded token of one sequence over a short context: the latency of a call
        dict(name="attention_decode_1", op="attention", N=1, L=1, packed=False, ctx=1500, lens_seed=3,
             Hq=16, Hk=4, d=128, window=0),
        # one decoded token of 256 sequences at unequal lengths
        dict(name="attention_decode_256", op="attention", N=256, L=1, packed=False, ctx=4096, lens_seed=4,
             Hq=16, Hk=4, d=128, window=0),
        # verification of 4 draft tokens over 32K-token contexts
        dict(name="attention_verify_4_long", op="attention", N=4, L=4, packed=False, ctx=32768, lens_seed=5,
             Hq=16, Hk=2, d=128, window=0),
        # one decoded token of the sliding-window layer of a hybrid stack
        dict(name="attention_decode_window", op="attention", N=64, L=1, packed=False, ctx=8192, lens_seed=6,
             Hq=16, Hk=16, d=64, window=2048),
        # a whole prompt, causal
        dict(name="attention_prompt_8192", op="attention", N=1, L=8192, packed=False, ctx=0, lens_seed=7,
             Hq=16, Hk=4, d=128, window=0),
        # packed prompts of unequal lengths behind cached prefixes, sliding window
        dict(name="attention_prompt_packed_window", op="attention", N=6, L=1500, packed=True, ctx=1000, lens_seed=8,
             Hq=16, Hk=8, d=128, window=512),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope_fwd", "rope_bwd", "prologue", "attention", "attention"])
    d = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 3, 4, 8, 16])
    G = rng.choice([1, 2, 3, 4, 8])
    Hq = Hk * G if Hk * G <= 32 else Hk
    if op in ("rope_fwd", "rope_bwd"):
        B = log_int(1, 16)
        return dict(op=op, B=B, T=log_int(1, 16384 // B), Hq=Hq if Hq <= 16 else 16 // Hk * Hk, Hk=Hk, d=d,
                    rot=rng.choice([d, d // 2, d // 4 + 8]), interleaved=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), far=rng.choice([0, 0, 100000, 3000000]))
    if op == "prologue":
        prompt = rng.random() < 0.5
        N = log_int(1, 12 if prompt else 256)
        return dict(op=op, N=N, L=log_int(5, 16384 // N) if prompt else rng.choice([1, 1, 2, 4]),
                    packed=prompt and rng.random() < 0.6, ctx=log_int(1, 2000) if not prompt or rng.random() < 0.5 else 0,
                    lens_seed=rng.randrange(1 << 20), Hq=Hq if Hq <= 16 else 16 // Hk * Hk, Hk=Hk, d=d,
                    rot=rng.choice([d, d // 2]), interleaved=rng.random() < 0.5)
    window = rng.choice([0, 0, log_int(16, 4096)])
    if rng.random() < 0.6:  # single tokens and drafts
        N = log_int(1, 256)
        ctx = log_int(1, min(32768, 65536 * 8 // (N * max(1, Hk // 2))))
        return dict(op=op, N=N, L=rng.choice([1, 1, 1, 2, 4, 7]), packed=False, ctx=ctx, lens_seed=rng.randrange(1 << 20),
                    Hq=Hq, Hk=Hk, d=d, window=window)
    N = log_int(1, 8)
    L = log_int(17, 6000 // N)
    return dict(op=op, N=N, L=L, packed=rng.random() < 0.5, ctx=rng.choice([0, log_int(1, 2000)]),
                lens_seed=rng.randrange(1 << 20), Hq=Hq if Hq <= 16 else 16 // Hk * Hk, Hk=Hk, d=d, window=window)


def _lengths(case):
    """New tokens and all tokens of each sequence: host int64 arrays. Packed batches have new
    tokens between a quarter of L and L; contexts reach from half of ctx to ctx."""
    r = np.random.RandomState(case["lens_seed"])
    N, L, ctx = case["N"], case["L"], case["ctx"]
    new = r.randint(max(1, L // 4), L + 1, N) if case["packed"] else np.full(N, L)
    before = r.randint((ctx + 1) // 2, ctx + 1, N) if ctx else np.zeros(N, np.int64)
    return new.astype(np.int64), (before + new).astype(np.int64)


def _pairs(case):
    """Query-key pairs that the masks leave, and cached tokens that some query reads."""
    new, total = _lengths(case)
    w = case["window"] or 1 << 40
    pairs = read = 0
    for n, t in zip(new.tolist(), total.tolist()):
        p = np.arange(t - n, t)
        pairs += int(np.minimum(p + 1, w).sum())
        read += min(t, n - 1 + w)
    return pairs, read


def work(case):
    d, Hq, Hk = case["d"], case["Hq"], case["Hk"]
    if case["op"] in ("rope_fwd", "rope_bwd"):
        size = 4 if case["dtype"] == "fp32" else 2
        rows = case["B"] * case["T"] * (Hq + Hk)
        moves = 2 if case["op"] == "rope_fwd" else 3
        return {"bytes": rows * d * size * moves + case["B"] * case["T"] * 4, "flops": rows * d * (6 if moves == 2 else 14)}
    new, total = _lengths(case)
    tokens = int(new.sum())
    if case["op"] == "prologue":
        return {"bytes": tokens * d * (4 * Hq + 2 * 2 * Hk + 2 * Hk), "flops": tokens * d * (6 * Hq + 8 * Hk)}
    pairs, read = _pairs(case)
    return {"bytes": read * Hk * d * 2 + tokens * Hq * d * 4, "flops": 4 * pairs * Hq * d}


# ---------------------------------------------------------------------------- inputs

def _inv_freq(rot, dev):
    return (10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)).float()


def _columns(dev):
    """Column of token t in a block of the value cache."""
    t = torch.arange(BLOCK, device=dev)
    return (t // 4 % 4) * 16 + (t // 16) * 4 + t % 4


def _power_scale(amax):
    """The smallest power of two s >= 2^-64 with amax <= 448 s."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, -64)).clamp(min=-64)
    return torch.ldexp(torch.ones_like(amax), e)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    d, Hq, Hk = case["d"], case["Hq"], case["Hk"]
    s = dict(case=case)
    if case["op"] in ("rope_fwd", "rope_bwd"):
        dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
        B, T = case["B"], case["T"]
        s["q"], s["k"] = normal(B, T, Hq, d, dtype=dt), normal(B, T, Hk, d, dtype=dt)
        if case["op"] == "rope_bwd":
            s["dq"], s["dk"] = normal(B, T, Hq, d, dtype=dt), normal(B, T, Hk, d, dtype=dt)
        first = torch.randint(0, case["far"] + 1, (B, 1), generator=gen, device=dev)
        s["positions"] = (first + torch.arange(T, device=dev)).to(torch.int32)
        s["inv_freq"] = _inv_freq(case["rot"], dev)
        s["q_weight"] = 1 + 0.1 * normal(d, dtype=torch.float32)
        s["k_weight"] = 1 + 0.1 * normal(d, dtype=torch.float32)
        return s
    new, total = _lengths(case)
    N = case["N"]
    MB = int(-(-total.max() // BLOCK))
    P = int((-(-total // BLOCK)).sum()) + 3
    order = torch.randperm(P, generator=gen, device=dev).to(torch.int32)
    used = torch.from_numpy(-(-total // BLOCK)).to(dev)
    col = torch.arange(MB, device=dev)
    flat = (used.cumsum(0) - used)[:, None] + col
    s["block_table"] = torch.where(col < used[:, None], order[flat.clamp(max=P - 1)], torch.zeros_like(order[:1])).contiguous()
    s["seq_lens"] = torch.from_numpy(total).to(dev).to(torch.int32)
    s["cu_seqlens"] = None
    shape = (N, case["L"])
    if case["packed"]:
        s["cu_seqlens"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)])).to(dev).to(torch.int32)
        shape = (1, int(new.sum()))
    s["new_max"] = int(new.max())
    # cached keys are normed rows, so elements near 1; values of every block have a size of
    # their own
    k = normal(P, Hk, BLOCK, d, dtype=torch.float32)
    s["k_scale"] = _power_scale(k.abs().amax((2, 3)))
    s["k_cache"] = (k / s["k_scale"][:, :, None, None]).to(torch.float8_e4m3fn)
    k = normal(P, Hk, d, BLOCK, dtype=torch.float32) * torch.exp(0.5 * normal(P, Hk, 1, 1, dtype=torch.float32))
    s["v_scale"] = _power_scale(k.abs().amax((2, 3)))
    s["v_cache"] = (k / s["v_scale"][:, :, None, None]).to(torch.float8_e4m3fn)
    s["q"] = normal(*shape, Hq, d)
    if case["op"] == "prologue":
        s["k"], s["v"] = normal(*shape, Hk, d), normal(*shape, Hk, d)
        s["inv_freq"] = _inv_freq(case["rot"], dev)
        s["q_weight"] = 1 + 0.1 * normal(d, dtype=torch.float32)
        s["k_weight"] = 1 + 0.1 * normal(d, dtype=torch.float32)
    return s


# ---------------------------------------------------------------------------- passes

def run(s):
    op = s["case"]["op"]
    if own:
        import gated_delta_rule_36_amd as G
        c = s["case"]
        if op == "rope_fwd":
            return G.qk_norm_rope_fwd(s["q"], s["k"], s["inv_freq"], positions=s["positions"], q_weight=s["q_weight"],
                                      k_weight=s["k_weight"], eps=EPS, interleaved=c["interleaved"])
        if op == "rope_bwd":
            return G.qk_norm_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], s["inv_freq"], positions=s["positions"],
                                      q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=c["interleaved"])
        cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        if op == "prologue":
            q = G.attn_prologue(s["q"], s["k"], s["v"], cache, s["block_table"], s["seq_lens"], s["inv_freq"],
                                cu_seqlens=s["cu_seqlens"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                                interleaved=c["interleaved"])
            return (q, *cache)
        return G.cache_attention(s["q"], cache, s["block_table"], s["seq_lens"], cu_seqlens=s["cu_seqlens"],
                                 window=c["window"])
    return {"rope_fwd": _plain_rope_fwd, "rope_bwd": _plain_rope_bwd, "prologue": _plain_prologue,
            "attention": _plain_attention}[op](s)


def _angles(positions, inv_freq):
    """cos and sin of position * frequency, [..., 1, rot / 2] (the angle in 64 bits: far
    positions)."""
    a = positions.double()[..., None, None] * inv_freq.double()
    return a.cos().float(), a.sin().float()


def _halves(x, rot, interleaved):
    """The two members of every rotated pair, and what is not rotated."""
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]
    return x[..., : rot // 2], x[..., rot // 2 : rot], x[..., rot:]


def _joined(a, b, rest, interleaved):
    if interleaved:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _turned(x, weight, cos, sin, interleaved):
    n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    a, b, rest = _halves(n, 2 * cos.shape[-1], interleaved)
    return _joined(a * cos - b * sin, b * cos + a * sin, rest, interleaved)


def _plain_rope_fwd(s):
    cos, sin = _angles(s["positions"], s["inv_freq"])
    return tuple(_turned(s[x].float(), s[x + "_weight"], cos, sin, s["case"]["interleaved"]).to(s[x].dtype) for x in ("q", "k"))


def _plain_back(x, g, weight, cos, sin, interleaved):
    d = x.shape[-1]
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    a, b, rest = _halves(g, 2 * cos.shape[-1], interleaved)
    dn = _joined(a * cos + b * sin, b * cos - a * sin, rest, interleaved)
    dw = (dn * x * r).double().flatten(0, -2).sum(0).float()
    u = dn * weight
    return r * (u - x * (r * r / d) * (u * x).sum(-1, keepdim=True)), dw


def _plain_rope_bwd(s):
    cos, sin = _angles(s["positions"], s["inv_freq"])
    il = s["case"]["interleaved"]
    dq, dwq = _plain_back(s["q"].float(), s["dq"].float(), s["q_weight"], cos, sin, il)
    dk, dwk = _plain_back(s["k"].float(), s["dk"].float(), s["k_weight"], cos, sin, il)
    return dq.to(s["q"].dtype), dk.to(s["k"].dtype), dwq, dwk


def _token_places(s):
    """Sequence and position of every new token, [tokens]."""
    c = s["case"]
    lens = s["seq_lens"].long()
    if c["packed"]:
        cu = s["cu_seqlens"].long()
        t = torch.arange(s["q"].shape[1], device=lens.device)
        n = torch.searchsorted(cu[1:], t, right=True)
        return n, lens[n] - cu[n + 1] + t
    n = torch.arange(c["N"], device=lens.device).repeat_interleave(c["L"])
    return n, lens[n] - c["L"] + torch.arange(c["L"], device=lens.device).repeat(c["N"])


def _plain_prologue(s):
    c = s["case"]
    Hk, d = c["Hk"], c["d"]
    n, pos = _token_places(s)
    cos, sin = _angles(pos, s["inv_freq"])
    q = _turned(s["q"].float().flatten(0, 1), s["q_weight"], cos, sin, c["interleaved"]).to(s["q"].dtype).view_as(s["q"])
    k = _turned(s["k"].float().flatten(0, 1), s["k_weight"], cos, sin, c["interleaved"])
    v = s["v"].float().flatten(0, 1)
    # the touched blocks of every sequence as one padded grid [N, X, 64] of positions
    lens = s["seq_lens"].long()
    first = torch.full_like(lens, 1 << 40).scatter_reduce(0, n, pos, "amin")
    X = (s["new_max"] + BLOCK - 2) // BLOCK + 1
    blk = (first // BLOCK)[:, None] + torch.arange(X, device=lens.device)
    touched = blk * BLOCK < lens[:, None]
    slot = s["block_table"].long().gather(1, blk.clamp(max=s["block_table"].shape[1] - 1))
    place = blk[:, :, None] * BLOCK + torch.arange(BLOCK, device=lens.device)
    old = place < first[:, None, None]
    fresh = ~old & (place < lens[:, None, None])
    begun = ~old[:, :, :1]  # no older token in the block
    token = torch.zeros_like(place)
    token[n, pos // BLOCK - blk[n, 0], pos % BLOCK] = torch.arange(n.numel(), device=lens.device)
    out = []
    for x, cache, scale in ((k, s["k_cache"], s["k_scale"]), (v, s["v_cache"].view(torch.uint8)[..., _columns(lens.device)].view(torch.float8_e4m3fn).transpose(2, 3), s["v_scale"])):
        rows = x[token] * fresh[..., None, None]  # [N, X, 64, Hk, d]
        s_old = scale[slot]
        need = _power_scale(rows.abs().amax((2, 4)))
        s_new = torch.where(begun, need, torch.maximum(s_old, need))
        held = cache[slot].float().transpose(2, 3)  # [N, X, 64, Hk, d]
        again = (held * (s_old / s_new)[:, :, None, :, None]).to(torch.float8_e4m3fn).float()
        codes = (rows / s_new[:, :, None, :, None]).to(torch.float8_e4m3fn).float()
        rest = held if x is k else held * ~begun[..., None, None]
        codes = torch.where(old[..., None, None], again, torch.where(fresh[..., None, None], codes, rest))
        scale[slot[touched]] = s_new[touched]
        out.append(codes[touched].transpose(1, 2).to(torch.float8_e4m3fn))
    where = slot[touched]
    s["k_cache"].view(torch.uint8)[where] = out[0].view(torch.uint8)
    t = torch.argsort(_columns(lens.device))
    s["v_cache"].view(torch.uint8)[where] = out[1].view(torch.uint8).transpose(2, 3)[..., t]
    return q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _plain_attention(s):
    c = s["case"]
    N, Hq, Hk, d = c["N"], c["Hq"], c["Hk"], c["d"]
    dev = s["q"].device
    lens = s["seq_lens"].long()
    n, pos = _token_places(s)
    # queries padded to [N, L]: the token at position p of a sequence stands at L - (len - p)
    L = s["new_max"]
    at = L - lens[n] + pos
    q = torch.zeros(N, L, Hq, d, device=dev)
    q[n, at] = s["q"].float().flatten(0, 1)
    slot = s["block_table"].long()
    k = (s["k_cache"][slot].float() * s["k_scale"][slot][..., None, None]).transpose(1, 2).flatten(2, 3)  # [N, Hk, S, d]
    v = s["v_cache"].view(torch.uint8)[slot][..., _columns(dev)].view(torch.float8_e4m3fn).float()
    v = (v * s["v_scale"][slot][..., None, None]).permute(0, 2, 1, 4, 3).flatten(2, 3)
    q = q.view(N, L, Hk, Hq // Hk, d).permute(0, 2, 3, 1, 4).reshape(N, Hk, -1, d)
    x = torch.matmul(q, k.transpose(2, 3).contiguous()).view(N, Hk, Hq // Hk, L, -1) * (1 / math.sqrt(d))
    p = (lens[:, None] - L + torch.arange(L, device=dev))[:, :, None]
    j = torch.arange(x.shape[-1], device=dev)
    seen = (j <= p) & (j > p - (c["window"] or 1 << 40))
    x = x.masked_fill(~seen[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top == float("-inf"), torch.zeros_like(top), top))
    x = x / x.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(x.flatten(2, 3), v).view(N, Hq, L, d).transpose(1, 2)
    return o[n, at].to(s["q"].dtype).view_as(s["q"])


# ---------------------------------------------------------------------------- 64 bits

def _spun(x, positions, inv_freq, weight, interleaved):
    """Norm, then each pair as a complex number times exp(i angle)."""
    n = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()
    rot = 2 * inv_freq.numel()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), positions.double()[..., None] * inv_freq.double())
    head = n[..., :rot]
    pair = head.unflatten(-1, (-1, 2)) if interleaved else head.unflatten(-1, (2, -1)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn[..., None, :])
    z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, n[..., rot:]], -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope_fwd":
        return tuple(_spun(s[x].double(), s["positions"], s["inv_freq"], s[x + "_weight"], case["interleaved"]) for x in ("q", "k"))
    if op == "rope_bwd":
        grads = []
        for x in ("q", "k"):
            a = s[x].double().requires_grad_()
            w = s[x + "_weight"].double().requires_grad_()
            y = _spun(a, s["positions"], s["inv_freq"], w, case["interleaved"])
            grads.append(torch.autograd.grad(y, (a, w), s["d" + x].double()))
        return grads[0][0], grads[1][0], grads[0][1], grads[1][1]
    new, total = _lengths(case)
    begin = np.cumsum(new) - new
    flat = {x: s[x].flatten(0, 1) for x in ("q", "k", "v") if x in s}
    if op == "prologue":
        pos = torch.from_numpy(np.concatenate([np.arange(t - n, t) for n, t in zip(new, total)])).to(s["q"].device)
        q = _spun(flat["q"].double(), pos, s["inv_freq"], s["q_weight"], case["interleaved"])
        # what 8 bits hold has no value of its own in 64 bits
        return q.view(*s["q"].shape), None, None, None, None
    d, Hq, Hk = case["d"], case["Hq"], case["Hk"]
    out = torch.zeros(flat["q"].shape, dtype=torch.float64, device=s["q"].device)
    cols = _columns(out.device)
    for i, (n, t, b) in enumerate(zip(new.tolist(), total.tolist(), begin.tolist())):
        blocks = s["block_table"][i, : -(-t // BLOCK)].long()
        low = max(0, t - n + 1 - case["window"]) if case["window"] else 0
        p = torch.arange(t - n, t, device=out.device)[:, None]
        j = torch.arange(low, t, device=out.device)
        hide = j > p
        if case["window"]:
            hide |= p - j >= case["window"]
        for h in range(Hk):
            k = (s["k_cache"][blocks, h].double() * s["k_scale"][blocks, h].double()[:, None, None]).reshape(-1, d)[low:t]
            v = (s["v_cache"][blocks, h].double() * s["v_scale"][blocks, h].double()[:, None, None])[..., cols]
            v = v.transpose(1, 2).reshape(-1, d)[low:t]
            for g in range(h * (Hq // Hk), (h + 1) * (Hq // Hk)):
                x = flat["q"][b : b + n, g].double() @ k.t() / math.sqrt(d)
                out[b : b + n, g] = torch.softmax(x.masked_fill(hide, float("-inf")), -1) @ v
    return out.view(*s["q"].shape)
