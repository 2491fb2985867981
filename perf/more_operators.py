"""Measured cases of the rotating slot write and of attention over a shared latent vector a token, in their
plain form and through the library's calls.

Rotation at position p, over the first n dimensions of a head, by the float32 table row cos_sin[p] (n / 2
cosines, then n / 2 sines): (a, b) becomes (a c - b s, b c + a s) for the pairs (x_i, x_(i + n/2)), or
(x_2i, x_(2i+1)) with `pairs`.  What is written to a cache is rounded to the inputs' type first.

A latent cache holds, for every token, a latent vector of R numbers (normalised by its root mean square and a
weight on the way in) and a rotated key part of 64 that all heads share.  The absorbed form attends over these
R + 64 numbers with queries of that size and takes the latent itself as the value; the expanded form attends
over keys and values of each head's own, computed from the latents, beside the shared key part.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
ROPE = 64     # the shared key part
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.bfloat16}  # of q, k, v, by the cache's


# ---------------------------------------------------------------- cases

def _rope(name, tokens, heads, kv_heads, head_size, rope=None, pairs=False, cache="bf16", scattered=False):
    c = dict(kind="rope", tokens=tokens, heads=heads, kv_heads=kv_heads, head_size=head_size, rope=rope or head_size,
             pairs=pairs, cache=cache, scattered=scattered)
    return dict(c, name=name) if name else c


def _store(name, tokens, heads, latent, pairs=False, norm=True, read=False, cache="bf16", scattered=False):
    c = dict(kind="store", tokens=tokens, heads=heads, latent=latent, pairs=pairs, norm=norm, read=read, cache=cache,
             scattered=scattered)
    return dict(c, name=name) if name else c


def _absorbed(name, heads, latent, requests, ctx_lo, ctx_hi, q_lo=1, q_hi=1, dist="uniform", lens=1):
    c = dict(kind="absorbed", heads=heads, latent=latent, requests=requests, ctx_lo=ctx_lo, ctx_hi=ctx_hi, q_lo=q_lo,
             q_hi=q_hi, dist=dist, lens=lens)
    return dict(c, name=name) if name else c


def _expanded(name, heads, size, requests, q_lo, q_hi, ctx_lo, ctx_hi, lens=1):
    c = dict(kind="expanded", heads=heads, size=size, requests=requests, q_lo=q_lo, q_hi=q_hi, ctx_lo=ctx_lo,
             ctx_hi=ctx_hi, dist="uniform", lens=lens)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the new tokens of a four-request decode step: a call whose latency counts, not its bytes
        _rope("rope_4_tokens", 4, 4, 2, 64, scattered=True),
        # a 2048-token chunk into an FP8 cache, a part of each head rotated, neighbours paired
        _rope("rope_chunk_fp8", 2048, 32, 8, 128, rope=64, pairs=True, cache="fp8"),
        # a long prompt, Llama-3-8B heads
        _rope("rope_long_prompt", 32768, 32, 8, 128),
        # the new tokens of a 256-request decode step over latents
        _store("latent_256_tokens", 256, 32, 512, pairs=True, scattered=True),
        # a long prompt's latents written, and read back for the expanded form
        _store("latent_long_prompt", 16384, 32, 512, pairs=True, read=True),
        # a decode step of four short requests
        _absorbed("absorbed_tiny", 4, 256, 4, 1, 64),
        # decode, batch 256, contexts lognormal (median 1024, sigma 0.8) up to 8192
        _absorbed("absorbed_decode", 32, 512, 256, 1024, 8192, dist="lognormal"),
        # long-context decode, batch 16
        _absorbed("absorbed_long", 16, 512, 16, 32768, 131072),
        # drafted tokens verified: two to eight per request
        _absorbed("absorbed_verify", 32, 512, 48, 256, 4096, q_lo=2, q_hi=8),
        # ragged short prompts
        _expanded("expanded_short", 16, 64, 3, 17, 201, 0, 0),
        # a step's prompts of ordinary length
        _expanded("expanded_prompts", 32, 128, 6, 300, 2048, 0, 0),
        # a 2048-token chunk of a long prompt
        _expanded("expanded_chunk", 32, 128, 1, 2048, 2048, 6144, 6144),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "store", "decode", "decode", "few", "expanded", "expanded"])
    if kind == "rope":
        d, kv, group = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
        return _rope(None, _log_int(rng, 1, 32768 if kv * group <= 32 else 16384), kv * group, kv, d,
                     rope=rng.choice([d, d, d // 2, 48]), pairs=rng.random() < 0.5,
                     cache=rng.choice(["bf16", "bf16", "f32", "fp8"]), scattered=rng.random() < 0.5)
    heads, lens = _log_int(rng, 1, 128), rng.randrange(1, 1 << 20)
    latent = rng.choice([256, 512, 512])
    if kind == "store":
        return _store(None, _log_int(rng, 1, min(16384, (1 << 19) // heads)), heads, latent, pairs=rng.random() < 0.5,
                      norm=rng.random() < 0.7, read=rng.random() < 0.5, cache=rng.choice(["bf16", "bf16", "f32"]),
                      scattered=rng.random() < 0.5)
    if kind == "decode":
        n = _log_int(rng, 1, 256)
        hi = _log_int(rng, 16, min(131072, (1 << 20) // n, (1 << 24) // (n * heads)))
        return _absorbed(None, heads, latent, n, max(1, hi // rng.choice([1, 2, 8, 16])), hi, lens=lens)
    if kind == "few":
        q_hi = rng.randrange(2, 17)
        n = _log_int(rng, 1, 64)
        hi = _log_int(rng, 16, max(17, min(8192, (1 << 24) // (n * heads * q_hi))))
        return _absorbed(None, heads, latent, n, max(1, hi // rng.choice([1, 4, 16])), hi, q_lo=rng.randrange(1, q_hi + 1),
                         q_hi=q_hi, lens=lens)
    heads = min(heads, 64)
    n = _log_int(rng, 1, 8)
    q_hi = _log_int(rng, 1, min(2048, (1 << 15) // n, (1 << 17) // (n * heads)))
    ctx = rng.choice([0, 0, _log_int(rng, 16, max(17, min(6144, (1 << 18) // (n * heads))))])
    return _expanded(None, heads, rng.choice([64, 128, 128]), n, max(1, q_hi // rng.choice([1, 2, 4])), q_hi, 0, ctx, lens=lens)


def _lengths(case):
    """(q_lens, seq_lens) of a case's requests."""
    rng = np.random.default_rng(case["lens"])
    n = case["requests"]
    if case["dist"] == "lognormal":
        ctx = np.clip(np.rint(case["ctx_lo"] * np.exp(0.8 * rng.standard_normal(n))), 1, case["ctx_hi"]).astype(np.int64)
    else:
        ctx = rng.integers(case["ctx_lo"], case["ctx_hi"], size=n, endpoint=True)
    q = rng.integers(case["q_lo"], case["q_hi"], size=n, endpoint=True)
    # the context of a decode counts its own token; the tokens of a chunk come on top of it
    return q, (ctx if case["kind"] == "absorbed" and case["q_hi"] == 1 else ctx + q).astype(np.int64)


def work(case):
    if case["kind"] == "rope":
        t, e = case["tokens"], TYPES[case["cache"]].itemsize
        ec = 1 if case["cache"] == "fp8" else e
        d, hq, hkv = case["head_size"], case["heads"], case["kv_heads"]
        return {"bytes": t * (2 * hq * d * e + 2 * hkv * d * (e + ec) + 4 * case["rope"] + 16),
                "flops": 3 * t * (hq + hkv) * case["rope"]}
    if case["kind"] == "store":
        t, e, row = case["tokens"], TYPES[case["cache"]].itemsize, case["latent"] + ROPE
        total = t * (2 * row * e + 2 * case["heads"] * ROPE * e + 4 * ROPE + 16) + (case["latent"] * e if case["norm"] else 0)
        return {"bytes": total + (t * (2 * row * e + 8) if case["read"] else 0),
                "flops": t * (3 * (case["heads"] + 1) * ROPE + (4 * case["latent"] if case["norm"] else 0))}
    q, s = _lengths(case)
    t, h = int(q.sum()), case["heads"]
    pairs = int((q * s - q * (q - 1) // 2).sum())  # (query, visible key)
    if case["kind"] == "absorbed":
        r = case["latent"]
        return {"bytes": int(s.sum()) * (r + ROPE) * 2 + t * h * (2 * r + ROPE) * 2 + 4 * int((-(-s // BLOCK)).sum()) + 8 * len(s),
                "flops": 2 * h * (2 * r + ROPE) * pairs}
    d = case["size"]
    return {"bytes": int(s.sum()) * (2 * h * d + ROPE) * 2 + t * h * (2 * d + ROPE) * 2 + 8 * len(s),
            "flops": 2 * h * (2 * d + ROPE) * pairs}


# ---------------------------------------------------------------- the plain form

def _rotated(x, table, positions, pairs):
    """float32 [T, H, D]: x with its first n = table.shape[1] dimensions rotated."""
    n = table.shape[1]
    row = table[positions][:, None]
    c, s = row[..., :n // 2], row[..., n // 2:]
    y = x.float()
    if pairs:
        a, b = y[..., 0:n:2], y[..., 1:n:2]
        return torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), y[..., n:]], -1)
    a, b = y[..., :n // 2], y[..., n // 2:n]
    return torch.cat([a * c - b * s, b * c + a * s, y[..., n:]], -1)


def _put(cache, slots, rows):
    cache.flatten(0, 1)[slots] = rows


def _codes(x, scale):
    """FP8 (E4M3) codes of x / scale, saturating."""
    return (x.float() / torch.tensor(scale, device=x.device)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_rope(st):
    q_out = _rotated(st["q"], st["table"], st["positions"], st["pairs"]).to(st["q"].dtype)
    k = _rotated(st["k"], st["table"], st["positions"], st["pairs"]).to(st["k"].dtype)
    v = st["v"]
    if st["cache"] == "fp8":
        k, v = _codes(k, st["k_scale"]), _codes(v, st["v_scale"])
    _put(st["k_cache"], st["slots"], k)
    _put(st["v_cache"], st["slots"], v)
    return _held(st, q_out)


def _held(st, q_out):
    if st["cache"] == "fp8":  # (scales of one: a code is the value it stands for)
        return q_out, st["k_cache"].view(torch.float8_e4m3fn), st["v_cache"].view(torch.float8_e4m3fn)
    return q_out, st["k_cache"], st["v_cache"]


def _plain_store(st):
    dtype = st["c"].dtype
    q_out = _rotated(st["q"], st["table"], st["positions"], st["pairs"]).to(dtype)
    c = st["c"].float()
    if st["weight"] is not None:
        c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * st["weight"].float()
    k = _rotated(st["k"][:, None], st["table"], st["positions"], st["pairs"])[:, 0]
    _put(st["latents"], st["slots"], torch.cat([c, k], -1).to(dtype))
    if not st["read"]:
        return q_out, st["latents"]
    rows = st["latents"].flatten(0, 1)[st["slots"]]
    return q_out, st["latents"], rows[:, :c.shape[-1]].contiguous(), rows[:, c.shape[-1]:].contiguous()


def _padded(st):
    """Rows of the flattened step by request, [n, longest query]: their index, and whether they exist."""
    first, last = st["starts"][:-1].long(), st["starts"][1:].long()
    j = torch.arange(st["max_query"], device=first.device)
    at = first[:, None] + j
    return at.clamp(max=len(st["q"]) - 1), at < last[:, None], j


def _weights(scores, seen):
    p = torch.exp(scores.masked_fill(~seen, -math.inf) - scores.masked_fill(~seen, -math.inf).amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _plain_absorbed(st):
    r = st["latents"].shape[-1] - ROPE
    at, real, j = _padded(st)
    length = st["seq_lens"].long()
    rows = (st["starts"][1:] - st["starts"][:-1]).long()
    keys = st["latents"][st["tables"].long().clamp(min=0)].flatten(1, 2).float()  # [n, keys, R + 64]
    key = torch.arange(keys.shape[1], device=keys.device)
    keys = keys.masked_fill((key >= length[:, None])[..., None], 0.0)  # slots that nothing was written to
    q = st["q"][at].float()  # [n, queries, heads, R + 64]
    scores = torch.matmul(q.flatten(1, 2), keys.transpose(-1, -2)).unflatten(1, q.shape[1:3]) * st["scale"]
    seen = key <= (length - rows)[:, None, None] + j[:, None]  # [n, queries, keys]
    p = _weights(scores, seen[:, :, None])
    del scores
    o = torch.matmul(p.flatten(1, 2), keys[..., :r]).unflatten(1, q.shape[1:3])
    return o[real].to(st["q"].dtype)


def _plain_expanded(st):
    at, real, j = _padded(st)
    first, length = st["kv_starts"][:-1].long(), (st["kv_starts"][1:] - st["kv_starts"][:-1]).long()
    rows = (st["starts"][1:] - st["starts"][:-1]).long()
    key = torch.arange(st["max_kv"], device=first.device)
    kv_at = (first[:, None] + key).clamp(max=len(st["k_rope"]) - 1)
    q = st["q"][at].float().transpose(1, 2)  # [n, heads, queries, D + 64]
    d = q.shape[-1] - ROPE
    k = st["k_nope"][kv_at].float().permute(0, 2, 3, 1)  # [n, heads, D, keys]
    scores = torch.matmul(q[..., :d], k)
    scores += torch.matmul(q[..., d:], st["k_rope"][kv_at].float().transpose(1, 2)[:, None])
    seen = key <= (length - rows)[:, None, None] + j[:, None]
    p = _weights(scores * st["scale"], seen[:, None])
    del scores, k
    v = st["v"][kv_at].float().transpose(1, 2)
    return torch.matmul(p, v).transpose(1, 2)[real].to(st["q"].dtype)


# ---------------------------------------------------------------- states and runs

def _normal(shape, gen, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _table(positions, n):
    """cos and sin of the angles p / 10000^(2 i / n), formed in 64 bits."""
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * torch.pow(
        torch.tensor(10000.0, device="cuda", dtype=torch.float64), -torch.arange(0, n, 2, device="cuda", dtype=torch.float64) / n)
    return torch.cat([angle.cos(), angle.sin()], -1).float()


def _places(tokens, scattered, gen):
    """(blocks, slots): where the tokens go, whole blocks in any order, or any slots."""
    blocks = -(-tokens // BLOCK) + 8
    perm = torch.randperm(blocks, generator=gen, device="cuda")
    slots = (perm[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")).flatten()
    if scattered:
        slots = slots[torch.randperm(len(slots), generator=gen, device="cuda")]
    return blocks, slots[:tokens].contiguous()


def _positions(tokens, scattered, gen):
    """A prompt's positions, or those of decodes (anywhere in 131072), and the table's rows."""
    if scattered:
        return torch.randint(0, 131072, (tokens,), generator=gen, device="cuda"), 131072
    return torch.arange(tokens, device="cuda") + 1000, tokens + 1000


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    if case["kind"] == "rope":
        t, hq, hkv, d, dtype = case["tokens"], case["heads"], case["kv_heads"], case["head_size"], TYPES[case["cache"]]
        blocks, slots = _places(t, case["scattered"], gen)
        positions, rows = _positions(t, case["scattered"], gen)
        qkv = _normal((t, (hq + 2 * hkv) * d), gen, dtype)  # one projection's rows
        q, k, v = (x.unflatten(-1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], -1))
        held = _normal((2, blocks, BLOCK, hkv, d), gen, dtype)  # what the caches held before
        if case["cache"] == "fp8":
            held = _codes(held, 1.0)
        return dict(kind="rope", cache=case["cache"], pairs=case["pairs"], q=q, k=k, v=v, slots=slots, positions=positions,
                    table=_table(rows, case["rope"]), k_cache=held[0].clone(), v_cache=held[1].clone(), k_scale=1.0, v_scale=1.0,
                    q_out=torch.empty(t, hq, d, dtype=dtype, device="cuda"))
    if case["kind"] == "store":
        t, h, r, dtype = case["tokens"], case["heads"], case["latent"], TYPES[case["cache"]]
        blocks, slots = _places(t, case["scattered"], gen)
        positions, rows = _positions(t, case["scattered"], gen)
        row = _normal((t, r + ROPE), gen, dtype)  # the projection to the latent and the key part
        q = _normal((t, h, 128 + ROPE), gen, dtype)  # queries whose last 64 dimensions are rotated
        return dict(kind="store", pairs=case["pairs"], read=case["read"], c=row[:, :r], k=row[:, r:], q=q[..., 128:],
                    weight=(1 + 0.1 * _normal((r,), gen, torch.float32)).to(dtype) if case["norm"] else None,
                    slots=slots, positions=positions, table=_table(rows, ROPE), heads=h,
                    latents=_normal((blocks, BLOCK, r + ROPE), gen, dtype),
                    q_out=torch.zeros(t, h, r + ROPE, dtype=dtype, device="cuda")[..., r:],  # beside the absorbed part
                    c_out=torch.empty(t, r, dtype=dtype, device="cuda"), k_out=torch.empty(t, ROPE, dtype=dtype, device="cuda"))
    q, s = _lengths(case)
    starts = np.concatenate([[0], np.cumsum(q)])
    t, h = int(starts[-1]), case["heads"]
    to32 = lambda x: torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).cuda()  # noqa: E731
    st = dict(kind=case["kind"], heads=h, starts=to32(starts), max_query=int(q.max()), max_kv=int(s.max()))
    if case["kind"] == "expanded":
        d, tk = case["size"], int(s.sum())
        kv = _normal((tk, h, 2 * d), gen)  # one projection of the latents: each head's key and value
        rest = _normal((tk, 2 * ROPE), gen)
        st.update(q=_normal((t, h, d + ROPE), gen), k_nope=kv[..., :d], v=kv[..., d:], k_rope=rest[:, ROPE:],
                  kv_starts=to32(np.concatenate([[0], np.cumsum(s)])), scale=1.0 / math.sqrt(d + ROPE),
                  out=torch.empty(t, h, d, dtype=torch.bfloat16, device="cuda"))
        return st
    r = case["latent"]
    nb = -(-s // BLOCK)
    blocks = int(nb.sum()) * 9 // 8 + 1
    first = np.concatenate([[0], np.cumsum(nb)])
    perm = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    place = first[:-1, None] + np.arange(int(nb.max()))
    table = perm[torch.from_numpy(np.minimum(place, blocks - 1)).cuda()]
    table[torch.from_numpy(np.arange(int(nb.max())) >= nb[:, None]).cuda()] = -1
    # slots that hold no request's token are NaN
    length = np.zeros(blocks, np.int64)
    owner = np.repeat(np.arange(len(q)), nb)
    length[:len(owner)] = s[owner] - (np.arange(len(owner)) - first[owner]) * BLOCK
    written = torch.zeros(blocks, BLOCK, dtype=torch.bool, device="cuda")
    written[perm.long()] = torch.from_numpy(np.arange(BLOCK) < length[:, None]).cuda()
    latents = torch.empty(blocks, BLOCK, r + ROPE, dtype=torch.bfloat16, device="cuda")
    step = 1 << 14
    for b in range(0, blocks, step):
        n = min(step, blocks - b)
        latents[b:b + n] = _normal((n, BLOCK, r + ROPE), gen).masked_fill_(~written[b:b + n, :, None], math.nan)
    st.update(q=_normal((t, h, r + ROPE), gen), latents=latents, tables=table.contiguous(), seq_lens=to32(s),
              scale=1.0 / math.sqrt(128 + ROPE), out=torch.empty(t, h, r, dtype=torch.bfloat16, device="cuda"))
    return st


def _library(st):
    """The library, and the layout and workspace that a program keeps beside its caches."""
    import paged_kv_attention_04_gb300 as P
    if "layout" not in st:
        if st["kind"] == "rope":
            st["layout"] = P.layout_of(st["k_cache"], st["q"].shape[1], k_scale=st["k_scale"], v_scale=st["v_scale"])
        elif st["kind"] != "expanded":
            st["layout"] = P.latent_layout_of(st["latents"], st["heads"])
            if st["kind"] == "absorbed":
                st["workspace"] = P.alloc_latent_workspace(st["layout"], len(st["seq_lens"]), len(st["q"]), st["max_query"],
                                                           st["max_kv"])
    return P, st.get("layout")


def _own_run(st):
    P, lay = _library(st)
    if st["kind"] == "rope":
        P.pa_rope_cache_write(st["q"], st["k"], st["v"], st["positions"], st["table"], st["slots"], st["q_out"], st["k_cache"],
                              st["v_cache"], lay, pairs=st["pairs"])
        return _held(st, st["q_out"])
    if st["kind"] == "store":
        P.pa_latent_write(st["c"], st["k"], st["q"], st["positions"], st["table"], st["slots"], st["q_out"], st["latents"], lay,
                          norm_weight=st["weight"], eps=EPS, pairs=st["pairs"])
        if not st["read"]:
            return st["q_out"], st["latents"]
        P.pa_latent_read(st["latents"], st["slots"], st["c_out"], st["k_out"], lay)
        return st["q_out"], st["latents"], st["c_out"], st["k_out"]
    if st["kind"] == "absorbed":
        P.pa_latent_forward(st["q"], st["latents"], st["tables"], st["seq_lens"], st["starts"], st["max_query"], st["max_kv"],
                            st["scale"], st["out"], st["workspace"], lay)
    else:
        P.pa_expanded_forward(st["q"], st["k_nope"], st["k_rope"], st["v"], st["starts"], st["kv_starts"], st["max_query"],
                              st["max_kv"], st["scale"], st["out"])
    return st["out"]


def run(state):
    """One pass: a rotating write, a latent write (and its read-back), or attention in the absorbed or the expanded form."""
    if own:
        return _own_run(state)
    return {"rope": _plain_rope, "store": _plain_store, "absorbed": _plain_absorbed, "expanded": _plain_expanded}[state["kind"]](state)


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_turn(x, table, positions, pairs):
    """Rotation as a product with exp(i angle), the first n dimensions taken as complex numbers."""
    n = table.shape[1]
    w = torch.complex(table[positions, :n // 2].double(), table[positions, n // 2:].double())[:, None]
    y = x.double().clone()
    re, im = (slice(0, n, 2), slice(1, n, 2)) if pairs else (slice(0, n // 2), slice(n // 2, n))
    z = torch.complex(y[..., re], y[..., im]) * w
    y[..., re], y[..., im] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "rope":
        dtype = st["k"].dtype
        q, k = (_exact_turn(st[x], st["table"], st["positions"], case["pairs"]) for x in "qk")
        caches = []
        for new, held in ((k, st["k_cache"]), (st["v"].double(), st["v_cache"])):
            fp8 = case["cache"] == "fp8"
            whole = (held.view(torch.float8_e4m3fn) if fp8 else held).double()
            if fp8:  # the nearest E4M3 number of the rounded key: steps of 2^-3 of its power of two, 2^-9 below 2^-6
                y = new.to(dtype).double().clamp(-448, 448)
                step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
                new = torch.round(y / step) * step
            whole.view(-1, *whole.shape[2:])[st["slots"]] = new
            caches.append(whole)
        return (q, *caches)
    if case["kind"] == "store":
        q = _exact_turn(st["q"], st["table"], st["positions"], case["pairs"])
        k = _exact_turn(st["k"][:, None], st["table"], st["positions"], case["pairs"])[:, 0]
        c = st["c"].double()
        if case["norm"]:
            c = c / torch.sqrt((c * c).sum(-1, keepdim=True) / case["latent"] + EPS) * st["weight"].double()
        whole = st["latents"].double()
        whole.view(-1, whole.shape[-1])[st["slots"]] = torch.cat([c, k], -1)
        return (q, whole, c, k) if case["read"] else (q, whole)
    q_lens, seq_lens = _lengths(case)
    if work(case)["flops"] > 1e12:
        return None
    out = torch.empty(st["out"].shape, dtype=torch.float64, device="cuda")
    a = b = 0
    for i, (n, s) in enumerate(zip(q_lens.tolist(), seq_lens.tolist())):
        pos = torch.arange(s, device="cuda")
        hidden = pos[None, :] > torch.arange(s - n, s, device="cuda")[:, None]
        q = st["q"][a:a + n].double()
        if case["kind"] == "absorbed":
            rows = st["latents"].flatten(0, 1)[st["tables"][i].long()[pos // BLOCK] * BLOCK + pos % BLOCK].double()
            logits = torch.einsum("ihd,kd->hik", q, rows) * st["scale"]
            w = torch.softmax(logits.masked_fill(hidden, -math.inf), -1)
            out[a:a + n] = torch.einsum("hik,kd->ihd", w, rows[:, :case["latent"]])
        else:
            kr = st["k_rope"][b:b + s].double()
            for h in range(case["heads"]):
                kh = torch.cat([st["k_nope"][b:b + s, h].double(), kr], -1)
                w = torch.softmax((q[:, h] @ kh.T * st["scale"]).masked_fill(hidden, -math.inf), -1)
                out[a:a + n, h] = w @ st["v"][b:b + s, h].double()
        a, b = a + n, b + s
    return out
