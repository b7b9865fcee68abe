"""The operators around the 4-bit cache and the rotary positions, as cases that can be timed and compared.

Each case is one call sequence of a serving program:

  rope_append     rotate the queries and keys of new tokens by their positions and append K and V to the paged cache
                  (E4M3, fp16 or E2M1 pools); Q, K and V are slices of one packed projection
  append          append K and V to the E2M1 cache and read the rows back as fp16
  decode          attention of decode / verify queries over the E2M1 cache, dense or over top-k token lists
  prefill         attention of packed prompt chunks over the E2M1 cache

`run` computes them with elementary torch operations in 32 bits, or, where `own` is true, with the library's calls.

E2M1 pools are [pages][kv heads][9 * D / 4] bytes. A page of one kv head holds the codes of its 4 tokens, D / 2 bytes each
(channel 2i in the low nibble of byte i), then its block scales as [D / 16 blocks][4 tokens] E4M3 bytes. A channel's value is
E2M1(code) * E4M3(block scale) * the layer's scale.
"""
import math

import torch

own = False

PAGE = 4
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # one decode step of 64 sequences: the call is launch and latency
        dict(name="rope_e4m3_decode", op="rope_append", pool="e4m3", tokens=64, q_heads=32, kv_heads=4, head_dim=128, rot=128,
             interleaved=False, first=4000),
        # a prefill chunk appended to the E4M3 cache
        dict(name="rope_e4m3_chunk", op="rope_append", pool="e4m3", tokens=8192, q_heads=32, kv_heads=4, head_dim=128, rot=128,
             interleaved=False, first=0),
        # interleaved pairs, a quarter of the head rotated, fp16 pools, an odd number of tokens
        dict(name="rope_fp16_part", op="rope_append", pool="fp16", tokens=1021, q_heads=8, kv_heads=2, head_dim=64, rot=16,
             interleaved=True, first=77),
        # a chunk and 48 decode tokens appended to the E2M1 cache, half of the head rotated
        dict(name="rope_e2m1_chunk", op="rope_append", pool="e2m1", tokens=8240, q_heads=32, kv_heads=4, head_dim=128, rot=64,
             interleaved=False, first=100000),
        # one decode step's rows into the E2M1 cache
        dict(name="append_e2m1_decode", op="append", tokens=48, kv_heads=4, head_dim=128),
        # a prompt's rows into the E2M1 cache
        dict(name="append_e2m1_chunk", op="append", tokens=4096, kv_heads=8, head_dim=128),
        # two short contexts at head_dim 64: the smallest call
        dict(name="decode_tiny", op="decode", batch=2, q_len=1, lens="list:37,100", q_heads=8, kv_heads=2, head_dim=64, topk=0),
        # the ordinary decode step
        dict(name="decode_4k", op="decode", batch=32, q_len=1, lens="fixed:4096", q_heads=32, kv_heads=4, head_dim=128, topk=0),
        # a verify step over contexts of very different lengths
        dict(name="verify_ragged", op="decode", batch=64, q_len=4, lens="log:1024:32768", q_heads=32, kv_heads=4, head_dim=128, topk=0),
        # long contexts, few sequences; the last one attends over a list of tokens
        dict(name="decode_long", op="decode", batch=4, q_len=1, lens="fixed:262144", q_heads=32, kv_heads=4, head_dim=128, topk=2048),
        # several prompts' chunks with history, odd lengths
        dict(name="prefill_ragged", op="prefill", chunks="700,37,1,1290", history="513,0,2000,64", q_heads=16, kv_heads=2, head_dim=128),
        # one long chunk over its own tokens
        dict(name="prefill_8k", op="prefill", chunks="8192", history="0", q_heads=32, kv_heads=4, head_dim=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rope_append", "append", "decode", "decode", "prefill"])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8])
    if op == "rope_append":
        head_dim = rng.choice([64, 128])
        return dict(op=op, pool=rng.choice(["e4m3", "fp16", "e2m1"]), tokens=_log_int(rng, 1, 4096), q_heads=kv_heads * min(group, 4),
                    kv_heads=kv_heads, head_dim=head_dim, rot=16 * rng.randint(1, head_dim // 16), interleaved=rng.random() < 0.5,
                    first=_log_int(rng, 1, 200000))
    if op == "append":
        return dict(op=op, tokens=_log_int(rng, 1, 8192), kv_heads=kv_heads, head_dim=rng.choice([64, 128]))
    if op == "decode":
        q_len = rng.choice([1, 1, 1, 2, 3, 4])
        batch = _log_int(rng, 1, 64)
        longest = _log_int(rng, max(4, q_len), 380000 // batch)
        lens = "fixed:%d" % longest if rng.random() < 0.3 else "log:%d:%d" % (max(q_len, longest // 20), longest)
        return dict(op=op, batch=batch, q_len=q_len, lens=lens, q_heads=kv_heads * group, kv_heads=kv_heads,
                    head_dim=rng.choice([64, 128]), topk=_log_int(rng, 1, 3000) if rng.random() < 0.3 else 0)
    n = rng.randint(1, 5)
    chunks = [_log_int(rng, 1, 1400) for _ in range(n)]
    history = [rng.choice([0, _log_int(rng, 1, 4000)]) for _ in range(n)]
    return dict(op=op, chunks=",".join(map(str, chunks)), history=",".join(map(str, history)), q_heads=kv_heads * min(group, 4),
                kv_heads=kv_heads, head_dim=128)


def _context_lens(case):
    kind, _, rest = case["lens"].partition(":")
    if kind == "fixed":
        return [int(rest)] * case["batch"]
    if kind == "list":
        return [int(x) for x in rest.split(",")]
    lo, hi = (int(x) for x in rest.split(":"))
    # lengths evenly spread over their logarithm, in an order that mixes them
    n = case["batch"]
    at = [math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * (i + 0.5) / n) for i in range(n)]
    return [max(lo, min(hi, int(at[(7 * i + 3) % n if math.gcd(7, n) == 1 else i]))) for i in range(n)]


# ---------------------------------------------------------------------------
# E2M1 pools in elementary operations

def _quantize(x, scale):
    """x [..., D] -> codes [..., D] (0..15), block scales [..., D / 16] (E4M3); scale: a tensor of one value."""
    blocks = x.unflatten(-1, (-1, 16))
    a = blocks.abs().amax(-1)
    b = (a / (scale * 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = b.float() * scale
    r = torch.where(d > 0, 1.0 / d, torch.zeros_like(d))
    y = blocks * r[..., None]
    m = y.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = code + 8 * (torch.signbit(y)).to(torch.uint8)
    return code.flatten(-2), b


def _views(pool, head_dim):
    codes = pool[..., :2 * head_dim].unflatten(-1, (PAGE, head_dim // 2))
    scales = pool[..., 2 * head_dim:].unflatten(-1, (head_dim // 16, PAGE))
    return codes, scales


def _values(codes, scales, pairs, scale):
    """Bytes [..., D / 2] and block scale bytes [..., D / 16] -> values [..., D] in 32 bits."""
    v = pairs[codes.long()].flatten(-2).unflatten(-1, (-1, 16))
    return ((v * scales.contiguous().view(torch.float8_e4m3fn).float()[..., None]) * scale).flatten(-2)


def _pairs(device):
    one = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=device)
    i = torch.arange(256, device=device)
    return torch.stack((one[i & 15], one[i >> 4]), -1)


def _pool_from(x, scale):
    """x [pages, kv heads, 4, D] -> an E2M1 pool."""
    code, b = _quantize(x, scale)
    codes = code[..., 0::2] | (code[..., 1::2] << 4)
    return torch.cat((codes.flatten(-2), b.view(torch.uint8).transpose(-1, -2).flatten(-2)), -1)


# ---------------------------------------------------------------------------
# what a program has in hand before the call

def _table(max_positions, rot, device):
    """cos | sin of position * 10000^(-2j / rot), from angles in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    angle = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * f
    return torch.cat((angle.cos(), angle.sin()), -1).float()


def _scale(x, most):
    """The layer's scale: the largest magnitude of a calibration draw over the largest value the type holds."""
    return torch.tensor(x.float().abs().max().item() / most, dtype=torch.float32).item()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed * 7919 + 13)
    rand = lambda *shape: torch.randn(*shape, device=dev, generator=g)  # noqa: E731
    op, Hkv = case["op"], case["kv_heads"]
    D = case["head_dim"]
    s = dict(op=op, case=case, pairs=_pairs(dev))
    # a few channels are far larger than the others, as keys and values have them
    gain = 1.0 + 5.0 * (torch.rand(Hkv, D, device=dev, generator=g) > 0.97).float()
    if op in ("rope_append", "append"):
        T = case["tokens"]
        pages = max(8, (T + 3) // 4 + T // 32)
        s["slots"] = torch.randperm(pages * PAGE, device=dev, generator=g)[:T].to(torch.int32)
        pool = case.get("pool", "e2m1")
        if op == "rope_append":
            Hq = case["q_heads"]
            packed = rand(T, Hq + 2 * Hkv, D)
            packed[:, Hq:Hq + Hkv] *= gain
            packed = packed.half()
            s["q"], s["k"], s["v"] = packed[:, :Hq], packed[:, Hq:Hq + Hkv], packed[:, Hq + Hkv:]
            s["q_out"] = torch.empty(T, Hq, D, dtype=torch.float16, device=dev)
            s["positions"] = (case["first"] + torch.randperm(T, device=dev, generator=g)).to(torch.int32)
            s["table"] = _table(case["first"] + T, case["rot"], dev)
        else:
            s["k"], s["v"] = (rand(T, Hkv, D) * gain).half(), rand(T, Hkv, D).half()
        if pool == "e2m1":
            shape, kind, most = (pages, Hkv, 9 * D // 4), torch.uint8, 2688.0
            s["k_out"] = torch.empty(T, Hkv, D, dtype=torch.float16, device=dev)
            s["v_out"] = torch.empty_like(s["k_out"])
        else:
            shape, kind, most = (pages, Hkv, PAGE, D), (torch.uint8 if pool == "e4m3" else torch.float16), 448.0
        s["k_cache"] = torch.zeros(shape, dtype=kind, device=dev)
        s["v_cache"] = torch.zeros(shape, dtype=kind, device=dev)
        s["pool"], s["ks"], s["vs"] = pool, _scale(s["k"], most), _scale(s["v"], most)
    else:
        if op == "decode":
            lens = _context_lens(case)
        else:
            chunks = [int(x) for x in case["chunks"].split(",")]
            lens = [n + int(h) for n, h in zip(chunks, case["history"].split(","))]
        B, most = len(lens), max((n + 3) // 4 for n in lens)
        used = sum((n + 3) // 4 for n in lens)
        pages = used + used // 16 + 1
        order = torch.randperm(pages, device=dev, generator=g).to(torch.int32)
        table = torch.zeros(B, most, dtype=torch.int32)
        at = 0
        order = order.cpu()
        for b, n in enumerate(lens):
            table[b, :(n + 3) // 4] = order[at:at + (n + 3) // 4]
            at += (n + 3) // 4
        s["block_tables"] = table.to(dev)
        s["context_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        for name in ("k", "v"):
            draw_ = rand(64, Hkv, PAGE, D) * (gain[:, None] if name == "k" else 1.0)
            s[name + "s"] = _scale(draw_, 2688.0)
            scale = torch.tensor(s[name + "s"], device=dev)
            pool = torch.empty(pages, Hkv, 9 * D // 4, dtype=torch.uint8, device=dev)
            step = max(1, (1 << 25) // (Hkv * PAGE * D))
            for p in range(0, pages, step):
                n = min(step, pages - p)
                x = rand(n, Hkv, PAGE, D)
                pool[p:p + n] = _pool_from(x * gain[:, None] if name == "k" else x, scale)
            s[name + "_cache"] = pool
        if op == "decode":
            s["q"] = rand(B, case["q_len"], case["q_heads"], D).half()
            # split partials: 32-bit rows of D + 2 values for every query row and split, as many splits as fill the card
            splits = min(1024, 2048 // (B * Hkv) + 1)
            s["workspace"] = torch.empty(B * case["q_len"] * case["q_heads"] * splits * (D + 2) + 256, device=dev)
            if case["topk"]:
                K = case["topk"]
                idx = torch.zeros(B, Hkv, K, dtype=torch.int32, device=dev)
                counts = torch.zeros(B, dtype=torch.int32)
                for b in range(B - 1, -1, -4):   # one sequence in four attends over a list
                    n = min(K, lens[b])
                    counts[b] = n
                    for h in range(Hkv):
                        idx[b, h, :n] = torch.randperm(lens[b], device=dev, generator=g)[:n].sort().values.to(torch.int32)
                s["topk_idx"], s["topk_lens"] = idx, counts.to(dev)
        else:
            start = [0]
            for n in chunks:
                start.append(start[-1] + n)
            s["q_start"] = torch.tensor(start, dtype=torch.int32, device=dev)
            s["max_q_len"] = max(chunks)
            # the attended keys and values as fp16 tiles of 128 tokens, with a mask of 16 bytes each
            s["workspace"] = torch.empty(B * Hkv * ((most * PAGE + 127) // 128) * (2 * 128 * D * 2 + 16), dtype=torch.uint8, device=dev)
            s["q"] = rand(start[-1], case["q_heads"], D).half()
        s["out"] = torch.empty_like(s["q"])
    for name in ("ks", "vs"):
        s[name + "_t"] = torch.tensor(s[name], dtype=torch.float32, device=dev)
    return s


# ---------------------------------------------------------------------------
# one pass

def _rotate(x, table, positions, rot, interleaved):
    row = table[positions.long()][:, None]
    c, n = row[..., :rot // 2], row[..., rot // 2:]
    x = x.float()
    a = x[..., 0:rot:2] if interleaved else x[..., :rot // 2]
    b = x[..., 1:rot:2] if interleaved else x[..., rot // 2:rot]
    y1, y2 = a * c - b * n, b * c + a * n
    y = torch.stack((y1, y2), -1).flatten(-2) if interleaved else torch.cat((y1, y2), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _append_plain(s, k, v):
    slot = s["slots"].long()
    page, at = slot // PAGE, slot % PAGE
    for x, pool, scale in ((k, s["k_cache"], s["ks_t"]), (v, s["v_cache"], s["vs_t"])):
        if s["pool"] == "fp16":
            pool[page, :, at] = x.half()
        elif s["pool"] == "e4m3":
            pool[page, :, at] = (x / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            code, b = _quantize(x, scale)
            codes, scales = _views(pool, x.shape[-1])
            codes[page, :, at] = code[..., 0::2] | (code[..., 1::2] << 4)
            scales[page, :, :, at] = b.view(torch.uint8)


def _read_plain(s, head_dim):
    slot = s["slots"].long()
    page, at = slot // PAGE, slot % PAGE
    got = []
    for pool, scale in ((s["k_cache"], s["ks_t"]), (s["v_cache"], s["vs_t"])):
        codes, scales = _views(pool, head_dim)
        got.append(_values(codes[page, :, at], scales[page, :, :, at], s["pairs"], scale).half())
    return got


def _pages_plain(s, pool, scale, head_dim):
    """The sequences' rows [B, kv heads, tokens, D] in 32 bits."""
    codes, scales = _views(pool[s["block_tables"].long()], head_dim)
    v = _values(codes, scales.transpose(-1, -2), s["pairs"], scale)      # [B, pages, kv heads, 4, D]
    return v.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _softmax_plain(score, mask, v):
    score = score.masked_fill(~mask, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (score - top).exp()
    return (p @ v) / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _decode_plain(s, case):
    q, lens = s["q"].float(), s["context_lens"].long()
    B, n, Hq, D = q.shape
    Hkv = case["kv_heads"]
    G = Hq // Hkv
    k = _pages_plain(s, s["k_cache"], s["ks_t"], D)
    v = _pages_plain(s, s["v_cache"], s["vs_t"], D)
    rows = q.unflatten(2, (Hkv, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)            # [B, kv heads, n * G, D]
    pos = torch.arange(k.shape[2], device=q.device)
    last = lens[:, None] - n + torch.arange(n, device=q.device)                      # [B, n]
    mask = (pos <= last[..., None]).repeat_interleave(G, 1)[:, None]                  # [B, 1, n * G, tokens]
    if "topk_idx" in s:
        K = s["topk_idx"].shape[2]
        live = torch.arange(K, device=q.device) < s["topk_lens"][:, None, None]
        hit = torch.zeros(B, Hkv, k.shape[2] + 1, dtype=torch.bool, device=q.device)
        hit.scatter_(2, torch.where(live, s["topk_idx"], k.shape[2]).long(), True)
        mask = mask & (hit[..., :-1] | (s["topk_lens"] == 0)[:, None, None])[:, :, None]
    o = _softmax_plain((rows @ k.transpose(-1, -2)) * (1.0 / math.sqrt(D)), mask, v)
    return o.unflatten(2, (n, G)).permute(0, 2, 1, 3, 4).flatten(2, 3).half()


def _prefill_plain(s, case):
    q, lens, start = s["q"].float(), s["context_lens"].long(), s["q_start"].long()
    total, Hq, D = q.shape
    Hkv, most = case["kv_heads"], s["max_q_len"]
    G = Hq // Hkv
    n = start[1:] - start[:-1]
    k = _pages_plain(s, s["k_cache"], s["ks_t"], D)
    v = _pages_plain(s, s["v_cache"], s["vs_t"], D)
    i = torch.arange(most, device=q.device)
    row = (start[:-1, None] + i).clamp(max=total - 1)                                 # [B, most]
    rows = q[row].unflatten(2, (Hkv, G)).permute(0, 2, 3, 1, 4).flatten(2, 3)         # [B, kv heads, G * most, D]
    last = (lens - n)[:, None] + i
    mask = (torch.arange(k.shape[2], device=q.device) <= last[..., None])[:, None].repeat(1, 1, G, 1)
    o = _softmax_plain((rows @ k.transpose(-1, -2)) * (1.0 / math.sqrt(D)), mask, v)
    o = o.unflatten(2, (G, most)).permute(0, 3, 1, 2, 4).flatten(2, 3)                # [B, most, Hq, D]
    token = torch.arange(total, device=q.device)
    b = torch.searchsorted(start[1:], token, right=True)
    return o[b, token - start[b]].half()


def _outputs(s, q_out, rows):
    """Pools as the values they hold (E4M3 codes in units of the layer's scale), E2M1 rows read back."""
    got = {} if q_out is None else {"q": q_out}
    if s["pool"] == "e2m1":
        got["k"], got["v"] = rows
    else:
        kind = torch.float8_e4m3fn if s["pool"] == "e4m3" else torch.float16
        got["k"], got["v"] = s["k_cache"].view(kind), s["v_cache"].view(kind)
    return got


def run(s):
    case, op = s["case"], s["op"]
    if own:
        return _run_own(s, case, op)
    if op == "rope_append":
        q, k = (_rotate(s[n], s["table"], s["positions"], case["rot"], case["interleaved"]) for n in ("q", "k"))
        s["q_out"].copy_(q)
        _append_plain(s, k, s["v"].float())
        return _outputs(s, s["q_out"], _read_plain(s, case["head_dim"]) if s["pool"] == "e2m1" else None)
    if op == "append":
        _append_plain(s, s["k"].float(), s["v"].float())
        return _outputs(s, None, _read_plain(s, case["head_dim"]))
    return (_decode_plain if op == "decode" else _prefill_plain)(s, case)


def _run_own(s, case, op):
    from fp8_paged_kv_e4m3_gb300 import kvq
    if op == "rope_append":
        args = (s["q"], s["k"], s["v"], s["positions"], s["table"], s["slots"], s["k_cache"], s["v_cache"])
        if s["pool"] == "fp16":
            kvq.kv_append_rope_fp16(*args, q_out=s["q_out"], interleaved=case["interleaved"])
        else:
            call = kvq.kv_append_rope_e4m3 if s["pool"] == "e4m3" else kvq.kv_append_rope_e2m1
            call(*args, s["ks"], s["vs"], q_out=s["q_out"], interleaved=case["interleaved"])
    elif op == "append":
        kvq.kv_append_e2m1(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["ks"], s["vs"])
    if op in ("rope_append", "append"):
        rows = None
        if s["pool"] == "e2m1":
            rows = kvq.kv_gather_e2m1(s["k_cache"], s["v_cache"], s["slots"], s["ks"], s["vs"], s["k_out"], s["v_out"])
        return _outputs(s, s.get("q_out"), rows)
    if op == "decode":
        idx, counts = s.get("topk_idx"), s.get("topk_lens")
        return kvq.paged_decode_attn_e2m1(s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"], s["ks"], s["vs"],
                                          s["workspace"], s["out"], idx, counts)
    return kvq.paged_prefill_attn_e2m1(s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"], s["q_start"], s["ks"],
                                       s["vs"], s["workspace"], s["out"], max_q_len=s["max_q_len"])


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    op, Hkv, D = case["op"], case["kv_heads"], case["head_dim"]
    row = 9 * D // 16                                      # bytes of one E2M1 row of one kv head
    if op in ("rope_append", "append"):
        T, pool = case["tokens"], case.get("pool", "e2m1")
        held = {"e4m3": D, "fp16": 2 * D, "e2m1": row}[pool]
        size = T * Hkv * 2 * (2 * D + held) + 4 * T
        if pool == "e2m1":
            size += T * Hkv * 2 * (held + 2 * D)           # read back as fp16
        flops = 4 * T * Hkv * D
        if op == "rope_append":
            size += T * case["q_heads"] * 4 * D + T * (4 + 4 * case["rot"])
            flops += 3 * T * (case["q_heads"] + Hkv) * case["rot"]
        return {"bytes": size, "flops": flops}
    Hq = case["q_heads"]
    if op == "decode":
        lens, n = _context_lens(case), case["q_len"]
        listed_ = set(range(len(lens) - 1, -1, -4)) if case["topk"] else set()
        size = 4 * len(lens) * n * Hq * D
        flops = 0
        for b, L in enumerate(lens):
            seen = min(case["topk"], L) if b in listed_ else L
            size += seen * Hkv * 2 * row + (seen * Hkv * 4 if b in listed_ else 0) + min(seen, (L + 3) // 4) * 4
            flops += 4 * D * Hq * n * seen
        return {"bytes": size, "flops": flops}
    size = flops = 0
    for n, h in zip(case["chunks"].split(","), case["history"].split(",")):
        n, L = int(n), int(n) + int(h)
        size += 4 * n * Hq * D + L * Hkv * 2 * row + L
        flops += 4 * D * Hq * (n * (L - n) + n * (n + 1) // 2)
    return {"bytes": size, "flops": flops}


# ---------------------------------------------------------------------------
# the operators from their definitions, in 64 bits

def _round_to(x, mantissa, smallest, largest):
    """x to the nearest value with `mantissa` bits below the leading one, steps no finer than 2^smallest, ties to even."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1 - mantissa).clamp(min=smallest).to(x.dtype))
    return ((x / step).round() * step).clamp(-largest, largest)


def _f32(x):
    """A 64-bit result rounded to 32 bits: the caches' quotients and products are defined in binary32."""
    return x.float().double()


def _cache_values(x, scale, pool):
    """What the pool holds of x: E4M3 in units of the scale, E2M1 as values, fp16 as it is."""
    if pool == "fp16":
        return x
    if pool == "e4m3":
        return _round_to(_f32(x / scale), 3, -9, 448.0)
    blocks = x.reshape(*x.shape[:-1], -1, 16)
    six = torch.tensor(6.0 * scale, dtype=torch.float64, device=x.device)
    b = _round_to(_f32(blocks.abs().amax(-1, keepdim=True) / _f32(six)), 3, -9, 448.0)
    y = _f32(blocks * _f32(1.0 / _f32(torch.where(b > 0, b * scale, 1.0))))
    return (torch.where(b > 0, _round_to(y, 1, -1, 6.0), 0.0) * b * scale).reshape(x.shape)


def _decoded(pool, scale, head_dim):
    """An E2M1 pool as [pages, kv heads, 4, D] in 64 bits, from the bits."""
    raw = pool[..., :2 * head_dim].reshape(*pool.shape[:2], PAGE, head_dim // 2).to(torch.int32)
    code = torch.stack((raw % 16, raw // 16), -1).reshape(*pool.shape[:2], PAGE, head_dim)
    e, m = (code // 2) % 4, (code % 2).double()
    size = torch.where(e == 0, m / 2, (1 + m / 2) * torch.pow(2.0, (e - 1).double()))
    size = torch.where(code >= 8, -size, size)
    raw = pool[..., 2 * head_dim:].reshape(*pool.shape[:2], head_dim // 16, PAGE).to(torch.int32)
    e, m = (raw // 8) % 16, (raw % 8).double()
    b = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.pow(2.0, (e - 10).double()))
    return size * b.transpose(-1, -2).repeat_interleave(16, -1) * scale


def _rows64(s, b, length, name, head_dim):
    pages = s["block_tables"][b, :(length + 3) // 4].long()
    v = _decoded(s[name + "_cache"][pages], float(s[name + "s"]), head_dim)
    return v.permute(1, 0, 2, 3).reshape(v.shape[1], -1, head_dim)[:, :length]


def _attend64(q, k, v, mask):
    """q [n, D], k and v [tokens, D], mask [n, tokens]."""
    w = torch.softmax((q @ k.T / math.sqrt(q.shape[-1])).masked_fill(~mask, -math.inf), -1)
    return torch.nan_to_num(w) @ v


def exact(case, seed):
    s = prepare(case, seed)
    op, D, Hkv = case["op"], case["head_dim"], case["kv_heads"]
    if op in ("rope_append", "append"):
        got, k = {}, s["k"].double()
        if op == "rope_append":
            rot = case["rot"]
            row = s["table"].double()[s["positions"].long()][:, None]
            turn = torch.complex(row[..., :rot // 2], row[..., rot // 2:])
            rotated = []
            for x in (s["q"].double(), k):
                part = x[..., :rot].reshape(*x.shape[:-1], *((-1, 2) if case["interleaved"] else (2, -1)))
                z = (torch.complex(part[..., 0], part[..., 1]) if case["interleaved"] else
                     torch.complex(part[..., 0, :], part[..., 1, :])) * turn
                y = torch.stack((z.real, z.imag), -1 if case["interleaved"] else -2)
                rotated.append(torch.cat((y.reshape(*x.shape[:-1], rot), x[..., rot:]), -1))
            got["q"], k = rotated
        for name, x in (("k", k), ("v", s["v"].double())):
            held = _cache_values(x, float(s[name + "s"]), s["pool"])
            if s["pool"] == "e2m1":
                got[name] = held
            else:
                pool = torch.zeros(s["k_cache"].shape, dtype=torch.float64, device=x.device)
                pool.permute(0, 2, 1, 3)[s["slots"].long() // PAGE, s["slots"].long() % PAGE] = held
                got[name] = pool
        return got
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    G = case["q_heads"] // Hkv
    for b, L in enumerate(s["context_lens"].tolist()):
        k, v = (_rows64(s, b, L, name, D) for name in ("k", "v"))
        if op == "decode":
            rows, to, n = s["q"][b].double(), out[b], case["q_len"]
        else:
            lo, hi = s["q_start"][b].item(), s["q_start"][b + 1].item()
            rows, to, n = s["q"][lo:hi].double(), out[lo:hi], hi - lo
        seen = torch.arange(L, device=k.device) <= torch.arange(L - n, L, device=k.device)[:, None]
        for h in range(case["q_heads"]):
            mask = seen
            if "topk_idx" in s and s["topk_lens"][b] > 0:
                chosen = torch.zeros(L, dtype=torch.bool, device=k.device)
                chosen[s["topk_idx"][b, h // G, :s["topk_lens"][b]].long()] = True
                mask = seen & chosen
            to[:, h] = _attend64(rows[:, h], k[h // G], v[h // G], mask)
    return out
