"""Measured cases of the 4-bit KV cache: the quantising slot write, the read-back and
attention over the cache, in their plain form and through the library's calls.

A 4-bit cache holds, for every token, kv head and group of 32 head dimensions, 32 codes of
4 bits and an f16 scale s and zero z; a code c stands for (c * s + z) * tensor_scale.  For a
group x (bf16) the write takes y = x / tensor_scale, saturated at +-16384, z = f16(min y),
s = f16((max y - min y) / 15) and c = round((y - z) / s) in 0 .. 15 (0 where s is 0), in
float32, ties to even; a group that holds a NaN reads back as NaN.

A cache is a byte tensor [num_blocks][num_kv_heads][10 * head_size]: a page per 16-token block
and kv head.  In 16-bit units, D = head_size, t the token's row in the block, a unit holding four
codes (nibble n, lowest first):
  K page  codes   [16 t][4 c][D/32 g][2 u], unit (t, c, g, u): dims 32 g + 8 c + 4 u + n
          params  [16 t][s of the D/32 groups, then their z]
  V page  codes   [2 h][8 e][4 p][D/32 i][2 b], unit of token 8 h + 2 p + b: dims e D/8 + 4 i + n
          params  [D/32 groups][4 p][s, z][2 h][2 b]
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
GROUP = 32
LIMIT = 16384.0


# ---------------------------------------------------------------- cases

def _attend(name, heads, kv_heads, head_size, decodes=0, ctx_lo=1, ctx_hi=1, chunks=0, q_lo=0, q_hi=0, prior_lo=0,
            prior_hi=0, dist="uniform", write=False, k_scale=1.0, v_scale=1.0, lens=1):
    c = dict(kind="attend", heads=heads, kv_heads=kv_heads, head_size=head_size, decodes=decodes, ctx_lo=ctx_lo,
             ctx_hi=ctx_hi, chunks=chunks, q_lo=q_lo, q_hi=q_hi, prior_lo=prior_lo, prior_hi=prior_hi, dist=dist,
             write=write, k_scale=k_scale, v_scale=v_scale, lens=lens)
    return dict(c, name=name) if name else c


def _copy(name, kind, tokens, kv_heads, head_size, scattered=False, k_scale=1.0, v_scale=1.0):
    c = dict(kind=kind, tokens=tokens, kv_heads=kv_heads, head_size=head_size, scattered=scattered, k_scale=k_scale,
             v_scale=v_scale)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the new tokens of a four-request decode step: a call whose latency counts, not its bytes
        _copy("store_4_tokens", "store", 4, 2, 64, scattered=True),
        # the new tokens of a 2048-token prefill chunk, Llama-3-8B heads, consecutive slots
        _copy("store_chunk", "store", 2048, 8, 128),
        # a long prompt's KV taken over from another instance, with per-tensor scales
        _copy("store_long_prompt", "store", 32768, 8, 128, k_scale=0.5, v_scale=2.0),
        # KV of several short requests read back for a bf16 instance: scattered slots, an odd count
        _copy("load_scattered", "load", 5003, 4, 64, scattered=True, k_scale=0.5, v_scale=2.0),
        # one 131072-token request read back
        _copy("load_long", "load", 131072, 8, 128),
        # a decode step of four short requests
        _attend("decode_tiny", 4, 2, 64, decodes=4, ctx_hi=64),
        # TinyLlama-1.1B decode, batch 64
        _attend("decode_tinyllama", 32, 4, 64, decodes=64, ctx_lo=128, ctx_hi=2048),
        # Llama-3-8B decode, batch 256, contexts lognormal (median 1024, sigma 0.8) up to 8192
        _attend("decode_llama3_8b", 32, 8, 128, decodes=256, ctx_lo=1024, ctx_hi=8192, dist="lognormal"),
        # long-context decode, batch 16
        _attend("decode_long", 32, 8, 128, decodes=16, ctx_lo=32768, ctx_hi=131072),
        # drafted tokens verified: two to eight per request
        _attend("verify", 32, 8, 128, chunks=48, q_lo=2, q_hi=8, prior_lo=256, prior_hi=4096),
        # a 2048-token chunk of a long prompt
        _attend("chunk_long", 32, 8, 128, chunks=1, q_lo=2048, q_hi=2048, prior_lo=6144, prior_hi=6144),
        # a whole mixed step: the write, attention of 64 decodes and two ragged chunks, and the new tokens read back
        _attend("step_mixed", 32, 8, 128, decodes=64, ctx_lo=256, ctx_hi=4096, chunks=2, q_lo=300, q_hi=512,
                prior_hi=1536, write=True, k_scale=0.5, v_scale=2.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice([64, 128])
    scales = rng.choice([dict(), dict(k_scale=0.5, v_scale=2.0), dict(k_scale=1.25, v_scale=0.375)])
    kind = rng.choice(["store", "load", "decode", "decode", "verify", "chunk", "chunk", "step"])
    if kind in ("store", "load"):
        return _copy(None, kind, _log_int(rng, 1, 32768 if kind == "store" else 131072), rng.choice([1, 2, 4, 8]), d,
                     scattered=rng.random() < 0.5, **scales)
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 8])
    heads = dict(heads=kv * group, kv_heads=kv, head_size=d, lens=rng.randrange(1, 1 << 20), **scales)
    if kind == "decode":
        batch = _log_int(rng, 1, 256)
        hi = _log_int(rng, 16, min(131072, (1 << 21) // batch))
        return _attend(None, decodes=batch, ctx_lo=max(1, hi // rng.choice([1, 2, 8, 16])), ctx_hi=hi, **heads)
    if kind == "verify":
        q_hi = rng.randrange(2, 16)
        return _attend(None, chunks=_log_int(rng, 1, 64), q_lo=rng.randrange(1, q_hi + 1), q_hi=q_hi,
                       prior_hi=_log_int(rng, 16, 8192), **heads)
    q_hi = _log_int(rng, 16, 2048)
    chunks = dict(chunks=rng.randrange(1, 4), q_lo=max(1, q_hi // rng.choice([1, 2, 4])), q_hi=q_hi,
                  prior_hi=_log_int(rng, 16, 6144 if kv * group <= 16 else 1536))
    if kind == "chunk":
        return _attend(None, **chunks, **heads)
    return _attend(None, decodes=_log_int(rng, 1, 64), ctx_hi=_log_int(rng, 16, 4096), write=True, **chunks, **heads)


def _lengths(case):
    """(q_lens, seq_lens) of a case's requests, the decodes first."""
    rng = np.random.default_rng(case["lens"])
    if case["dist"] == "lognormal":
        z = rng.standard_normal(case["decodes"])
        dec = np.clip(np.rint(case["ctx_lo"] * np.exp(0.8 * z)), 1, case["ctx_hi"]).astype(np.int64)
    else:
        dec = rng.integers(case["ctx_lo"], case["ctx_hi"], size=case["decodes"], endpoint=True)
    q = rng.integers(case["q_lo"], case["q_hi"], size=case["chunks"], endpoint=True)
    prior = rng.integers(case["prior_lo"], case["prior_hi"], size=case["chunks"], endpoint=True)
    return (np.concatenate([np.ones(case["decodes"], np.int64), q]),
            np.concatenate([dec, prior + q]).astype(np.int64))


def work(case):
    kv, d = case["kv_heads"], case["head_size"]
    row4, row16 = kv * d * 5 // 8, kv * d * 2  # a token's K (or V) in 4 bits, in bf16
    if case["kind"] == "store":
        t = case["tokens"]
        return {"bytes": t * (2 * 2 * (row16 + row4) + 8), "flops": 0}
    if case["kind"] == "load":
        t = case["tokens"]
        return {"bytes": t * (2 * (row16 + row4) + 8), "flops": 0}
    q, s = _lengths(case)
    t = int(q.sum())
    pairs = int((q * s - q * (q - 1) // 2).sum())  # (query, visible key)
    total = 2 * int(s.sum()) * row4 + 2 * t * case["heads"] * d * 2 + 4 * int((-(-s // BLOCK)).sum()) + 8 * len(s)
    if case["write"]:
        total += t * (2 * 2 * row16 + 2 * row4 + 8)  # new K and V in, read back out; their codes written
    return {"bytes": total, "flops": 4 * d * case["heads"] * pairs}


# ---------------------------------------------------------------- the 4-bit form, in torch operations

def _quantise(x, scale):
    """Codes (int16 [..., D]), s and z (f16 [..., D/32]) of x."""
    full = lambda v: torch.full((), v, dtype=torch.float32, device=x.device)  # noqa: E731
    y = (x.float() / full(scale)).clamp(-LIMIT, LIMIT).unflatten(-1, (-1, GROUP))
    lo, hi = y.amin(-1), y.amax(-1)
    s, z = ((hi - lo) / full(15.0)).half(), lo.half()
    c = torch.round((y - z.float().unsqueeze(-1)) / s.float().unsqueeze(-1)).clamp(0, 15)
    c = torch.where((s > 0).unsqueeze(-1), c, torch.zeros_like(c))
    return c.flatten(-2).to(torch.int16), s, z


def _units(codes):
    """Four codes a 16-bit unit: [..., 4] -> [...]."""
    return codes[..., 0] | (codes[..., 1] << 4) | (codes[..., 2] << 8) | (codes[..., 3] << 12)


def _k_units(codes, s, z):
    """A token's 16-bit units of a K page, in the page's order: [..., D] codes -> [..., 5 D / 16]."""
    u = _units(codes.unflatten(-1, (-1, 4, 2, 4))).transpose(-3, -2).flatten(-3)
    return torch.cat([u, torch.cat([s, z], -1).view(torch.int16)], -1)


def _v_units(codes, s, z):
    u = _units(codes.unflatten(-1, (8, -1, 4))).flatten(-2)
    return torch.cat([u, torch.stack([s, z], -1).flatten(-2).view(torch.int16)], -1)


def _unit_maps(d, device):
    """The units of a page that hold each of its 16 tokens, in the page's order: of K and of V, [16, 5 D / 16]."""
    i, j = torch.arange(4 * d, device=device), torch.arange(d, device=device)
    k = torch.cat([i // (d // 4), j // (d // 16)])
    v = torch.cat([i // (2 * d) * 8 + i // (d // 16) % 4 * 2 + i % 2, j // 2 % 2 * 8 + j // 8 % 4 * 2 + j % 2])
    return [torch.argsort(m, stable=True).view(BLOCK, 5 * d // 16) for m in (k, v)]


def _nibbles(u):
    return torch.stack([u & 15, (u >> 4) & 15, (u >> 8) & 15, (u >> 12) & 15], -1)


def _values(codes, s, z, scale):
    """float32 values of codes [..., D/32, 32] with s and z [..., D/32]."""
    return ((codes.float() * s.float().unsqueeze(-1) + z.float().unsqueeze(-1)) * scale).flatten(-2)


def _k_values(units, scale):
    """float32 [..., D] of tokens' units [..., 5 D / 16]."""
    n = units.shape[-1] // 5 * 4
    c = _nibbles(units[..., :n].unflatten(-1, (4, -1, 2))).transpose(-4, -3).flatten(-3)
    s, z = units[..., n:].contiguous().view(torch.float16).unflatten(-1, (2, -1)).unbind(-2)
    return _values(c, s, z, scale)


def _v_values(units, scale):
    n = units.shape[-1] // 5 * 4
    c = _nibbles(units[..., :n]).flatten(-2).unflatten(-1, (-1, GROUP))
    s, z = units[..., n:].contiguous().view(torch.float16).unflatten(-1, (-1, 2)).unbind(-1)
    return _values(c, s, z, scale)


def _rows(cache, units, slots):
    """Index of the slots' units in a cache [NB, H, 5 D] of 16-bit units."""
    heads = torch.arange(cache.shape[1], device=cache.device)
    return (slots // BLOCK)[:, None, None], heads[None, :, None], units[slots % BLOCK][:, None, :]


def _plain_store(st):
    """The quantising write of k and v into their slots of the caches, in place."""
    kc, vc = st["k_cache"].view(torch.int16), st["v_cache"].view(torch.int16)
    mk, mv = _unit_maps(st["k"].shape[-1], kc.device)
    kc[_rows(kc, mk, st["slots"])] = _k_units(*_quantise(st["k"], st["k_scale"]))
    vc[_rows(vc, mv, st["slots"])] = _v_units(*_quantise(st["v"], st["v_scale"]))


def _plain_load(st):
    kc, vc = st["k_cache"].view(torch.int16), st["v_cache"].view(torch.int16)
    mk, mv = _unit_maps(kc.shape[-1] // 5, kc.device)
    return (_k_values(kc[_rows(kc, mk, st["slots"])], st["k_scale"]).to(torch.bfloat16),
            _v_values(vc[_rows(vc, mv, st["slots"])], st["v_scale"]).to(torch.bfloat16))


def _plain_attend(st, r0, r1, q_len, seq_len):
    """Attention of requests r0 .. r1 - 1, padded to q_len rows and seq_len keys: float32 [r1 - r0, q_len, Hq, D]."""
    dev = st["q"].device
    n, (_, hq, d), hkv = r1 - r0, st["q"].shape, st["k_cache"].shape[1]
    first, length = st["starts"][r0:r1].long(), st["seq_lens"][r0:r1].long()
    rows = st["starts"][r0 + 1:r1 + 1].long() - first
    j = torch.arange(q_len, device=dev)
    q = st["q"][(first[:, None] + j).clamp(max=len(st["q"]) - 1)].float()
    q = q.view(n, q_len, hkv, hq // hkv, d).transpose(1, 2).flatten(2, 3)  # [n, Hkv, rows x group, D]
    blocks = -(-seq_len // BLOCK)
    table = st["tables"][r0:r1, :blocks].long().clamp(min=0)
    mk, mv = _unit_maps(d, dev)
    key = torch.arange(blocks * BLOCK, device=dev)
    k = _k_values(st["k_cache"].view(torch.int16)[table][..., mk], st["k_scale"])  # [n, blocks, Hkv, 16, D]
    k = k.transpose(1, 2).flatten(2, 3)
    scores = torch.matmul(q, k.transpose(-1, -2)).unflatten(2, (q_len, -1)) * st["scale"]
    del k
    seen = key <= (length - rows)[:, None, None] + j[:, None]  # [n, q_len, keys]
    scores = scores.masked_fill(~seen[:, None, :, None, :], -math.inf)
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).flatten(2, 3)
    del scores
    v = _v_values(st["v_cache"].view(torch.int16)[table][..., mv], st["v_scale"]).transpose(1, 2).flatten(2, 3)
    v = v.masked_fill((key >= length[:, None])[:, None, :, None], 0.0)  # slots that nothing was written to
    return torch.matmul(p, v).view(n, hkv, q_len, hq // hkv, d).transpose(1, 2).flatten(2, 3)


def _plain_forward(st):
    """Attention of the whole step: the decodes, then the chunks."""
    parts = []
    n = st["decodes"]
    if n:
        parts.append(_plain_attend(st, 0, n, 1, st["max_decode"]).flatten(0, 1))
    if st["chunks"]:
        o = _plain_attend(st, n, n + st["chunks"], st["max_chunk"], st["max_chunk_seq"])
        parts.append(o[st["chunk_rows"]])
    return torch.cat(parts).to(torch.bfloat16)


# ---------------------------------------------------------------- states and runs

def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _pool(blocks, heads, d, scale, spread, gen, written, units, unit_map):
    """A cache of `blocks` blocks whose written slots hold quantised N(0, spread) data, the others NaN."""
    cache = torch.empty(blocks, heads, 5 * d, dtype=torch.int16, device="cuda")
    step = max(1, (1 << 27) // (BLOCK * heads * d))
    for b in range(0, blocks, step):
        n = min(step, blocks - b)
        x = _normal((n, heads, BLOCK, d), gen) * spread
        x.masked_fill_(~written[b:b + n, None, :, None], math.nan)
        cache[b:b + n, :, unit_map.flatten()] = units(*_quantise(x, scale)).flatten(-2)
    return cache.view(torch.uint8)


def _pools(case, blocks, written, gen):
    h, d = case["kv_heads"], case["head_size"]
    mk, mv = _unit_maps(d, "cuda")
    ks, vs = case["k_scale"], case["v_scale"]
    return {"k_cache": _pool(blocks, h, d, ks, 1.0, gen, written, _k_units, mk),
            "v_cache": _pool(blocks, h, d, vs, 1.0, gen, written, _v_units, mv), "k_scale": ks, "v_scale": vs}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    h, d = case["kv_heads"], case["head_size"]
    if case["kind"] != "attend":
        t = case["tokens"]
        blocks = -(-t // BLOCK) + 8
        perm = torch.randperm(blocks, generator=gen, device="cuda")
        slots = (perm[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")).flatten()
        if case["scattered"]:
            slots = slots[torch.randperm(len(slots), generator=gen, device="cuda")]
        slots = slots[:t].contiguous()
        written = torch.zeros(blocks * BLOCK, dtype=torch.bool, device="cuda")
        if case["kind"] == "load":
            written[slots] = True
        st = _pools(case, blocks, written.view(blocks, BLOCK), gen)
        st.update(kind=case["kind"], slots=slots, heads=h)
        if case["kind"] == "store":
            st["k"], st["v"] = _normal((t, h, d), gen), _normal((t, h, d), gen)
        st["k_out"], st["v_out"] = (torch.empty(t, h, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return st
    q, s = _lengths(case)
    nb = -(-s // BLOCK)
    blocks = int(nb.sum()) * 9 // 8 + 1
    first = np.concatenate([[0], np.cumsum(nb)])
    starts = np.concatenate([[0], np.cumsum(q)])
    t = int(starts[-1])
    perm = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    place = first[:-1, None] + np.arange(int(nb.max()))
    table = perm[torch.from_numpy(np.minimum(place, blocks - 1)).cuda()]
    table[torch.from_numpy(np.arange(int(nb.max())) >= nb[:, None]).cuda()] = -1
    req = np.repeat(np.arange(len(q)), q)
    off = np.arange(t) - starts[req]
    pos = s[req] - q[req] + off
    slots = perm[torch.from_numpy(first[req] + pos // BLOCK).cuda()].long() * BLOCK + torch.from_numpy(pos % BLOCK).cuda()
    # the slots that hold data: every request's keys, less this step's where the run writes them
    length = np.zeros(blocks, np.int64)
    owner = np.repeat(np.arange(len(q)), nb)
    held = s - q if case["write"] else s
    length[:len(owner)] = held[owner] - (np.arange(len(owner)) - first[owner]) * BLOCK
    written = torch.zeros(blocks, BLOCK, dtype=torch.bool, device="cuda")
    written[perm.long()] = torch.from_numpy(np.arange(BLOCK) < length[:, None]).cuda()
    st = _pools(case, blocks, written, gen)
    n = case["decodes"]
    st.update(kind="attend", write=case["write"], heads=case["heads"], decodes=n, chunks=case["chunks"],
              scale=1.0 / math.sqrt(d), slots=slots, tables=table.contiguous(),
              seq_lens=torch.from_numpy(s.astype(np.int32)).cuda(), starts=torch.from_numpy(starts.astype(np.int32)).cuda(),
              max_query=int(q.max()), max_seq=int(s.max()), max_decode=int(s[:n].max()) if n else 0,
              max_chunk=int(q[n:].max()) if case["chunks"] else 0, max_chunk_seq=int(s[n:].max()) if case["chunks"] else 0)
    st["chunk_rows"] = (torch.from_numpy(req[starts[n]:] - n).cuda(), torch.from_numpy(off[starts[n]:]).cuda())
    st["q"] = _normal((t, case["heads"], d), gen)
    st["out"] = torch.empty_like(st["q"])
    if case["write"]:
        st["k"], st["v"] = _normal((t, h, d), gen), _normal((t, h, d), gen)
        st["k_out"], st["v_out"] = torch.empty_like(st["k"]), torch.empty_like(st["v"])
    return st


def _library(st):
    """The library, and the layout and workspace that a program keeps beside its caches."""
    import paged_kv_attention_04_gb300 as P
    if "layout" not in st:
        st["layout"] = P.layout_of(st["k_cache"], st["heads"], k_scale=st["k_scale"], v_scale=st["v_scale"])
        if st["kind"] == "attend":
            st["workspace"] = P.alloc_workspace(st["layout"], len(st["seq_lens"]), len(st["q"]), st["max_seq"])
    return P, st["layout"]


def _own_run(st):
    P, lay = _library(st)
    kc, vc = st["k_cache"], st["v_cache"]
    if st["kind"] == "store" or st.get("write"):
        P.pa_cache_write(st["k"], st["v"], st["slots"], kc, vc, lay)
    if st["kind"] == "attend":
        P.pa_forward(st["q"], kc, vc, st["tables"], st["seq_lens"], st["starts"], st["max_query"], st["max_seq"],
                     st["scale"], st["out"], st["workspace"], lay)
        if not st["write"]:
            return st["out"]
    P.pa_cache_read(kc, vc, st["slots"], st["k_out"], st["v_out"], lay)
    return (st["out"], st["k_out"], st["v_out"]) if st["kind"] == "attend" else (st["k_out"], st["v_out"])


def _plain_run(st):
    if st["kind"] == "store" or st.get("write"):
        _plain_store(st)
    if st["kind"] != "attend":
        return _plain_load(st)
    out = _plain_forward(st)
    return (out, *_plain_load(st)) if st["write"] else out


def run(state):
    """One pass: a write and its read-back, a read-back, attention, or a whole step (write, attention, read-back)."""
    return _own_run(state) if own else _plain_run(state)


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_new(x, scale):
    """float64 values that the cache holds for new rows x [T, H, D]."""
    y = (x.double() / scale).clamp(-LIMIT, LIMIT)
    y = y.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    z = y.min(-1, keepdim=True).values.half().double()
    s = ((y.max(-1, keepdim=True).values - y.min(-1, keepdim=True).values) / 15).half().double()
    c = torch.where(s > 0, ((y - z) / torch.where(s > 0, s, 1.0)).round().clamp(0, 15), 0.0)
    return ((c * s + z) * scale).reshape(x.shape)


def _exact_held(cache, slots, is_v, scale):
    """float64 [T, H, D] of slots of a cache, by each dimension's byte and nibble."""
    d = cache.shape[-1] // 10
    dim, t = torch.arange(d, device=cache.device)[None], (slots % BLOCK)[:, None]
    g = dim // GROUP
    if is_v:
        e, r = dim // (d // 8), dim % (d // 8)
        byte = t // 8 * 4 * d + e * (d // 2) + t % 8 // 2 * (d // 8) + r // 4 * 4 + t % 2 * 2 + r % 4 // 2
        s_at = 8 * d + g * 64 + t % 8 // 2 * 16 + t // 8 * 4 + t % 2 * 2
        z_at = s_at + 8
    else:
        byte = t * (d // 2) + dim % GROUP // 8 * (d // 8) + g * 4 + dim % 8 // 2
        s_at = 8 * d + t * (d // 8) + g * 2
        z_at = s_at + d // GROUP * 2
    rows = cache[slots // BLOCK].transpose(0, 1)  # [H, T, bytes]
    pick = lambda at: rows.gather(-1, at[None].expand(rows.shape[0], -1, -1))  # noqa: E731
    c = (pick(byte) >> (dim % 2 * 4).to(torch.uint8)) & 15
    f16 = lambda at: torch.stack([pick(at), pick(at + 1)], -1).contiguous().view(torch.float16)[..., 0].double()  # noqa: E731
    return ((c.double() * f16(s_at) + f16(z_at)) * scale).transpose(0, 1)


def exact(case, seed):
    st = prepare(case, seed)
    ks, vs = st["k_scale"], st["v_scale"]
    if case["kind"] == "store":
        return _exact_new(st["k"], ks), _exact_new(st["v"], vs)
    if case["kind"] == "load":
        return _exact_held(st["k_cache"], st["slots"], False, ks), _exact_held(st["v_cache"], st["slots"], True, vs)
    new = (_exact_new(st["k"], ks), _exact_new(st["v"], vs)) if case["write"] else None
    q_lens, seq_lens = _lengths(case)
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    a = 0
    for r, (n, s) in enumerate(zip(q_lens.tolist(), seq_lens.tolist())):
        pos = torch.arange(s, device="cuda")
        slots = st["tables"][r].long()[pos // BLOCK] * BLOCK + pos % BLOCK
        k = _exact_held(st["k_cache"], slots, False, ks)
        v = _exact_held(st["v_cache"], slots, True, vs)
        if new is not None:
            k[s - n:], v[s - n:] = new[0][a:a + n], new[1][a:a + n]
        group = st["q"].shape[1] // k.shape[1]
        for g in range(k.shape[1]):
            q = st["q"][a:a + n, g * group:(g + 1) * group].double()
            logits = torch.einsum("ihd,kd->ihk", q, k[:, g]) * st["scale"]
            hidden = pos[None, :] > torch.arange(s - n, s, device="cuda")[:, None]
            w = torch.softmax(logits.masked_fill(hidden[:, None, :], -math.inf), -1)
            out[a:a + n, g * group:(g + 1) * group] = torch.einsum("ihk,kd->ihd", w, v[:, g])
        a += n
    return (out, *new) if new is not None else out
