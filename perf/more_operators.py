"""What an attention layer runs between its projections and its output when sequences live in
the paged cache, with plain forms: norms and rotary positions of queries and keys, the same
on the way into the cache, and attention of the new tokens over the cache.

With ``own`` set, run() makes the calls a user makes of the library; otherwise it computes
the same from elementary torch operations.  A case's ``op`` is

  "rope"    gdn_qk_norm_rope        RMS norms of the heads of q and k, and their rotation
  "append"  gdn_kv_append_rope      the same; k and v go to the cache's pages
  "extend"  gdn_attn_prefill_paged  new tokens of each sequence over its cached rows, all of
                                    them or a window and the first few

and its lengths are texts of comma-separated numbers, one for each sequence.
"""
import itertools
import math

import torch

own = False

EPS = 1e-6


def listed():
    return [
        # one decoding step of 64 sequences, a quarter of each head rotated: launch latency
        dict(name="rope_step_b64", op="rope", tokens=64, h_q=16, h_kv=2, dim=256, rotary=64,
             theta=1e7, far=262144, norm=True, pairs=False, sections="", mixed=False),
        # a batch of long prompts, whole heads rotated
        dict(name="rope_t32768", op="rope", tokens=32768, h_q=32, h_kv=8, dim=128, rotary=128,
             theta=1e6, far=131072, norm=True, pairs=False, sections="", mixed=False),
        # pictures and text: positions in time, height and width, an odd number of tokens
        dict(name="rope_video_t9001", op="rope", tokens=9001, h_q=16, h_kv=4, dim=128, rotary=128,
             theta=5e6, far=30000, norm=True, pairs=False, sections="24,20,20", mixed=True),
        # one decoding step of 256 sequences into 8-bit pages
        dict(name="append_step_b256", op="append", new=",".join(["1"] * 256),
             start=",".join(str((i * 37) % 500) for i in range(256)), h_q=16, h_kv=2, dim=256,
             rotary=64, theta=1e7, norm=True, pairs=False, page=64, pages=8, bits=8),
        # a ragged batch of pieces into bf16 pages of 16, neighbouring dimensions rotated
        dict(name="append_ragged", op="append", new="16384,4095,17,2048,1,5000,333",
             start="70000,0,31,777,8191,100,5", h_q=32, h_kv=8, dim=128, rotary=128, theta=5e5,
             norm=False, pairs=True, page=16, pages=5400, bits=16),
        # drafted tokens of eight sequences checked at once: latency, a few rows each
        dict(name="extend_verify_b8", op="extend", new="4,5,2,4,3,1,4,5",
             length="517,1203,64,2500,3001,900,1777,4090", h_q=16, h_kv=2, dim=256, page=64,
             bits=16, window=0, sinks=0),
        # a few tokens over a very long 8-bit cache
        dict(name="extend_verify_l131072", op="extend", new="5,3", length="131072,60001", h_q=16,
             h_kv=2, dim=256, page=64, bits=8, window=0, sinks=0),
        # a piece of a long prompt over the rows cached before it
        dict(name="extend_piece", op="extend", new="2048", length="16000", h_q=16, h_kv=2, dim=256,
             page=64, bits=16, window=0, sinks=0),
        # the same over an 8-bit cache in smaller pages, heads of 128
        dict(name="extend_piece_e4m3_d128", op="extend", new="2000", length="11011", h_q=32,
             h_kv=8, dim=128, page=16, bits=8, window=0, sinks=0),
        # a step of a server that mixes a piece of a prompt with sequences that decode
        dict(name="extend_mixed", op="extend", new="512" + ",1" * 24,
             length="6000," + ",".join(str(1 + (i * i * 331) % 7001) for i in range(24)), h_q=32,
             h_kv=8, dim=128, page=32, bits=16, window=0, sinks=0),
        # a long prompt's piece in a layer that sees a window and the first four tokens
        dict(name="extend_window", op="extend", new="4000", length="20000", h_q=16, h_kv=2,
             dim=256, page=128, bits=16, window=4096, sinks=4),
        # a decoding step of such a layer
        dict(name="extend_window_step_b64", op="extend", new=",".join(["1"] * 64),
             length=",".join(str(500 + (i * 997) % 9001) for i in range(64)), h_q=16, h_kv=2,
             dim=256, page=64, bits=8, window=2048, sinks=4),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "extend", "extend"])
    dim = rng.choice([128, 256])
    h_kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    text = lambda xs: ",".join(str(x) for x in xs)  # noqa: E731
    turn = dict(rotary=rng.choice([32, 64, 96, 128, dim]), theta=rng.choice([1e4, 5e5, 1e6, 1e7]),
                norm=rng.random() < 0.7, pairs=rng.random() < 0.3)
    if op == "rope":
        tokens = _spread(rng, 1, 32768 * 40 * 128 // (h_kv * (group + 1) * dim))
        sections = ""
        if rng.random() < 0.4:
            a = rng.randrange(4, turn["rotary"] // 2 - 8)
            b = rng.randrange(2, turn["rotary"] // 2 - a - 1)
            sections = text([a, b, turn["rotary"] // 2 - a - b])
        return dict(op=op, tokens=min(tokens, 65536), h_q=h_kv * group, h_kv=h_kv, dim=dim,
                    far=_spread(rng, 100, 2 ** 21), sections=sections, mixed=rng.random() < 0.5,
                    **turn)
    n = _spread(rng, 1, 48)
    page = rng.choice([8, 16, 32, 64, 128, 256])
    bits = rng.choice([8, 16])
    if op == "append":
        new = [_spread(rng, 1, 16384 // n) for _ in range(n)]
        start = [_spread(rng, 1, 4096) - 1 for _ in range(n)]
        pages = max(-(-(s + x) // page) for s, x in zip(start, new)) + rng.randrange(3)
        return dict(op=op, new=text(new), start=text(start), h_q=h_kv * group, h_kv=h_kv, dim=dim,
                    page=page, pages=pages, bits=bits, **turn)
    most = _spread(rng, 1, 2048)
    new = [_spread(rng, 1, max(1, most // n)) if n > 1 else most for _ in range(n)]
    length = [x + _spread(rng, 1, 131072 // (n * h_kv)) - 1 for x in new]
    # so that the score matrix stays below the largest listed case's
    while sum(new) * sum(length) * h_kv * group > 2 ** 30 and (len(new) > 1 or new[0] > 1):
        if len(new) > 1:
            new.pop()
            length.pop()
        else:
            length = [length[0] - new[0] + (new[0] + 1) // 2]
            new = [(new[0] + 1) // 2]
    window = rng.choice([0, 0, _spread(rng, 1, 4096)])
    return dict(op=op, new=text(new), length=text(length), h_q=h_kv * group, h_kv=h_kv, dim=dim,
                page=page, bits=bits, window=window, sinks=rng.choice([0, 1, 4, 130]) if window else 0)


def _numbers(text):
    return [int(x) for x in text.split(",") if x]


def _offsets(lengths):
    return [0, *itertools.accumulate(lengths)]


def _normal(gen, shape, spread=1.0, loud=0):
    """bf16 N(0, spread^2); the first `loud` channels of a row four times that, as
    the keys of a trained model have a few channels that stand out."""
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    x *= spread
    if loud:
        x[..., :loud] *= 4
    return x


def _pool(gen, counts, h_kv, page, dim, bits, loud):
    """Pages holding rows of an earlier use, in the cache's own form, three more than needed."""
    rows = _normal(gen, (sum(counts) + 3, h_kv, page, dim), loud=loud)
    return (rows, None) if bits == 16 else _quantise(rows)


def _tables(gen, counts, width):
    """A page table [sequences][width]: every page used once, in no order; the
    entries that a sequence does not need hold -1."""
    order = torch.randperm(sum(counts) + 3, generator=gen, device="cuda").to(torch.int32)
    used = torch.nn.utils.rnn.pad_sequence(order[:sum(counts)].split(counts), batch_first=True,
                                           padding_value=-1)
    return torch.nn.functional.pad(used, (0, width - used.shape[1]), value=-1).contiguous()


def _axes(case):
    """Which axis each frequency's angle goes by: a section after the other, or in turn
    while the sections last (and by the first axis after that); none without sections."""
    sections = _numbers(case.get("sections", ""))
    if not sections:
        return None
    if not case["mixed"]:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    return [i % 3 if i < 3 * sections[i % 3] else 0 for i in range(case["rotary"] // 2)]


def _grid(gen, tokens, far):
    """Positions of text and pictures in turn: in text all axes alike, in a picture of
    24 x 32 patches time stands still while height and width go over its grid."""
    t = torch.arange(tokens, device="cuda")
    block, at = t // 1000, t % 1000
    picture = at < 768
    first = torch.randint(0, max(1, far - 1000), (tokens // 1000 + 1,), generator=gen,
                          device="cuda").sort().values[block]
    height = first + torch.where(picture, at // 32, at - 768 + 32)
    width = first + torch.where(picture, at % 32, at - 768 + 32)
    return torch.stack([first + torch.where(picture, 0 * at, at - 768 + 32), height, width])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, dim, h_q, h_kv = case["op"], case["dim"], case["h_q"], case["h_kv"]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    state = dict(op=op)
    if op != "extend":
        half = case["rotary"] // 2
        place = torch.arange(half, device="cuda", dtype=torch.float64)
        state.update(inv_freq=(case["theta"] ** (-place / half)).float(), pairs=case["pairs"],
                     eps=EPS if case["norm"] else None, q_weight=None, k_weight=None, axes=None,
                     axis=None)
        if case["norm"]:
            for name in ("q_weight", "k_weight"):
                state[name] = 1 + 0.3 * torch.randn(dim, generator=gen, device="cuda")
        tokens = case["tokens"] if op == "rope" else sum(_numbers(case["new"]))
        # q, k and v side by side, as one projection leaves them
        qkv = torch.cat([_normal(gen, (tokens, h_q, dim), 1.5),
                         _normal(gen, (tokens, h_kv, dim), loud=4),
                         _normal(gen, (tokens, h_kv, dim))], dim=1)
        state.update(q=qkv[:, :h_q], k=qkv[:, h_q:h_q + h_kv], v=qkv[:, h_q + h_kv:])
    if op == "rope":
        axes = _axes(case)
        if axes is None:
            at = torch.randint(0, case["far"], (tokens,), generator=gen, device="cuda")
        else:
            at = _grid(gen, tokens, case["far"])
            state.update(axes=bytes(axes), axis=torch.tensor(axes, device="cuda"))
        return dict(state, positions=at.to(torch.int32))
    new, page, bits = _numbers(case["new"]), case["page"], case["bits"]
    if op == "append":
        start = _numbers(case["start"])
        length = [s + x for s, x in zip(start, new)]
        counts = [-(-x // page) for x in length]
        width = case["pages"]
        state.update(start=i32(start))
    else:
        length = _numbers(case["length"])
        counts = [-(-x // page) for x in length]
        width = max(counts)
        state.update(q=_normal(gen, (sum(new), h_q, dim), 1.5), length=i32(length),
                     window=case["window"], sinks=case["sinks"], scale=dim ** -0.5,
                     rows=sum(length))
    k_pages, k_exp = _pool(gen, counts, h_kv, page, dim, bits, 4)
    v_pages, v_exp = _pool(gen, counts, h_kv, page, dim, bits, 0)
    return dict(state, k_pages=k_pages, v_pages=v_pages, k_exp=k_exp, v_exp=v_exp,
                table=_tables(gen, counts, width), cu=i32(_offsets(new)))


# ------------------------------------------------------------------ plain forms
def _places(cu, total):
    """The sequence of each of the packed tokens, and its place in it."""
    t = torch.arange(total, device=cu.device)
    n = torch.searchsorted(cu[1:].long(), t, right=True)
    return n, t - cu.long()[n]


def _normed(x, weight, eps):
    x = x.float()
    if eps is None:
        return x
    return x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + eps) * weight


def _turned(s, x, weight, positions):
    """A head's norm and rotation, in bf16.  The angles are products in 64 bits: with 32 a
    position of 100,000 is off by a hundredth of a radian."""
    x = _normed(x, weight, s["eps"])
    freq = s["inv_freq"].double()
    at = positions.double()
    angle = at[s["axis"]].T * freq if s["axis"] is not None else at[:, None] * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    r = 2 * freq.shape[0]
    a, b = (x[..., :r:2], x[..., 1:r:2]) if s["pairs"] else (x[..., :r // 2], x[..., r // 2:r])
    a, b = a * cos - b * sin, b * cos + a * sin
    both = torch.stack([a, b], dim=-1).flatten(-2) if s["pairs"] else torch.cat([a, b], dim=-1)
    return torch.cat([both, x[..., r:]], dim=-1).to(torch.bfloat16)


def _power(byte):
    """2^(byte - 127) for an exponent byte, by its bits."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _quantise(x):
    """e4m3 codes of the last dimension's rows, and their exponent bytes: the
    smallest power of two that brings a row's largest finite value to 448 or less."""
    x = x.float()
    finite = torch.isfinite(x)
    amax = torch.where(finite, x.abs(), torch.zeros_like(x)).amax(dim=-1)
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1); 448 = 7/8 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)
    e = torch.where(amax > 0, e, torch.zeros_like(e))
    y = x * _power(127 - e)[..., None]
    codes = torch.where(finite, y, torch.full_like(y, math.nan)).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def _plain_append(s):
    total, page = s["k"].shape[0], s["k_pages"].shape[2]
    n, place = _places(s["cu"], total)
    pos = place + s["start"].long()[n]
    at, slot = s["table"].long()[n, pos // page], pos % page
    q, k = _turned(s, s["q"], s["q_weight"], pos), _turned(s, s["k"], s["k_weight"], pos)
    if s["k_exp"] is None:
        s["k_pages"][at, :, slot] = k
        s["v_pages"][at, :, slot] = s["v"]
        return q
    # the 8-bit types have no indexed assignment: their bytes are moved
    kc, ke = _quantise(k)
    vc, ve = _quantise(s["v"])
    s["k_pages"].view(torch.uint8)[at, :, slot] = kc.view(torch.uint8)
    s["v_pages"].view(torch.uint8)[at, :, slot] = vc.view(torch.uint8)
    s["k_exp"][at, :, slot] = ke
    s["v_exp"][at, :, slot] = ve
    return q


def _plain_extend(s):
    q = s["q"].float()
    tq, h_q, dim = q.shape
    h_kv, page = s["k_pages"].shape[1:3]
    group, length = h_q // h_kv, s["length"].long()
    # the cached rows of all sequences side by side: [h_kv][rows][dim]
    ends = length.cumsum(0)
    nk, pk = _places(torch.nn.functional.pad(ends, (1, 0)), s["rows"])
    at, slot = s["table"].long()[nk, pk // page], pk % page

    def rows(pages, exps):
        if exps is None:
            return pages[at, :, slot].float().transpose(0, 1)
        x = pages.view(torch.uint8)[at, :, slot].view(torch.float8_e4m3fn).float()
        return (x * _power(exps[at, :, slot])[..., None]).transpose(0, 1)

    k, v = rows(s["k_pages"], s["k_exp"]), rows(s["v_pages"], s["v_exp"])
    # a sequence's queries are the last of its positions
    nq, pq = _places(s["cu"], tq)
    pq = pq + (length - (s["cu"][1:] - s["cu"][:-1]).long())[nq]
    seen = (nq[:, None] == nk[None, :]) & (pk[None, :] <= pq[:, None])
    if s["window"]:
        seen &= (pk[None, :] > pq[:, None] - s["window"]) | (pk[None, :] < s["sinks"])
    qh = q.view(tq, h_kv, group, dim).permute(1, 2, 0, 3).reshape(h_kv, group * tq, dim)
    w = torch.bmm(qh * s["scale"], k.transpose(1, 2)).view(h_kv, group, tq, -1)
    w.masked_fill_(~seen, -math.inf)
    top = w.amax(dim=-1, keepdim=True).clamp_(min=torch.finfo(w.dtype).min)
    w.sub_(top).exp_()
    total = w.sum(dim=-1, keepdim=True)
    o = torch.bmm(w.view(h_kv, group * tq, -1), v).view(h_kv, group, tq, dim)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.permute(2, 0, 1, 3).reshape(tq, h_q, dim).to(torch.bfloat16)


# ------------------------------------------------------------------ the library's calls
def _own_rope(s):
    import gated_deltanet_linear_recurrence_gb300 as gdn
    return gdn.gdn_qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"],
                                q_weight=s["q_weight"], k_weight=s["k_weight"], norm_eps=s["eps"],
                                axes=s["axes"], interleaved=s["pairs"])


def _own_append(s):
    import gated_deltanet_linear_recurrence_gb300 as gdn
    return gdn.gdn_kv_append_rope(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"],
                                  s["cu"], s["start"], s["inv_freq"], q_weight=s["q_weight"],
                                  k_weight=s["k_weight"], norm_eps=s["eps"],
                                  interleaved=s["pairs"], k_exp=s["k_exp"], v_exp=s["v_exp"])


def _own_extend(s):
    import gated_deltanet_linear_recurrence_gb300 as gdn
    return gdn.gdn_attn_prefill_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["cu"],
                                      s["length"], k_exp=s["k_exp"], v_exp=s["v_exp"],
                                      window=s["window"] or None, sinks=s["sinks"],
                                      scale=s["scale"])


def run(state):
    op = state["op"]
    if op == "rope":
        if own:
            q, k = _own_rope(state)
        else:
            q = _turned(state, state["q"], state["q_weight"], state["positions"])
            k = _turned(state, state["k"], state["k_weight"], state["positions"])
        return {"q": q, "k": k}
    if op == "append":
        out = {"q": _own_append(state) if own else _plain_append(state),
               "k_pages": state["k_pages"], "v_pages": state["v_pages"]}
        if state["k_exp"] is not None:  # the bytes as the powers of two that they stand for
            out.update(k_unit=state["k_exp"].view(torch.float8_e8m0fnu),
                       v_unit=state["v_exp"].view(torch.float8_e8m0fnu))
        return out
    return {"o": _own_extend(state) if own else _plain_extend(state)}


def _seen(a, b, window, sinks):
    """Keys that the last a of b positions see, in all."""
    if not window:
        return a * (b - a) + a * (a + 1) // 2
    return sum(p + 1 - max(0, p + 1 - window) + min(sinks, max(0, p + 1 - window))
               for p in range(max(0, b - a), b))


def work(case):
    dim, h_q, h_kv = case["dim"], case["h_q"], case["h_kv"]
    if case["op"] == "rope":
        axes = len(_numbers(case["sections"])) or 1
        values = case["tokens"] * (h_q + h_kv) * dim
        return {"bytes": 4 * values + 4 * axes * case["tokens"] + 2 * case["rotary"] + 8 * dim,
                "flops": 8 * values}
    new, page = _numbers(case["new"]), case["page"]
    row = dim * 2 if case["bits"] == 16 else dim + 1
    if case["op"] == "append":
        tokens = sum(new)
        touched = sum(-(-(s + x) // page) - s // page for s, x in zip(_numbers(case["start"]), new))
        return {"bytes": tokens * (4 * h_q * dim + 2 * h_kv * (2 * dim + row)) + 4 * touched
                + 8 * len(new) + 2 * case["rotary"] + 8 * dim,
                "flops": tokens * (8 * h_q + 9 * h_kv) * dim}
    length, window, sinks = _numbers(case["length"]), case["window"], case["sinks"]
    rows = [b - max(0, b - a - window + 1) + min(sinks, max(0, b - a - window + 1)) if window else b
            for a, b in zip(new, length)]
    return {"bytes": 2 * sum(rows) * h_kv * row + 4 * sum(new) * h_q * dim
            + sum(4 * -(-x // page) + 8 for x in rows),
            "flops": 4 * dim * h_q * sum(_seen(a, b, window, sinks) for a, b in zip(new, length))}


# ------------------------------------------------------------------ 64 bits, from the definitions
def _rotate64(x, weight, eps, place, inv_freq, axis, pairs):
    """x [T][heads][dim] as complex numbers turned by place * inv_freq."""
    x = x.double()
    if eps is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + eps).sqrt() * weight.double()
    n = inv_freq.numel()
    where = place.double()
    where = where.expand(n, -1) if axis is None else torch.stack([where[a] for a in axis])
    spin = torch.exp(1j * (where * inv_freq.double()[:, None]).T)[:, None]  # [T][1][n]
    first = torch.arange(n, device=x.device) * (2 if pairs else 1)
    second = first + (1 if pairs else n)
    z = torch.complex(x[..., first], x[..., second]) * spin
    x[..., first], x[..., second] = z.real, z.imag
    return x


def _unit64(x):
    """The powers of two in which an 8-bit cache keeps the rows of x."""
    amax = x.abs().amax(dim=-1, keepdim=True)
    unit = torch.exp2(torch.ceil(torch.log2(amax / 448)))
    unit = torch.where(amax > 448 * unit, unit * 2, unit)
    unit = torch.where(amax <= 448 * unit / 2, unit / 2, unit).clamp(min=2.0 ** -126)
    return torch.where(amax > 0, unit, torch.ones_like(unit))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        turn = lambda x, w: _rotate64(x, w, s["eps"], s["positions"], s["inv_freq"],  # noqa: E731
                                      _axes(case), s["pairs"])
        return {"q": turn(s["q"], s["q_weight"]), "k": turn(s["k"], s["k_weight"])}
    page = case["page"]
    if case["op"] == "append":
        place, at = [], []
        for n, (a, x) in enumerate(zip(_numbers(case["start"]), _numbers(case["new"]))):
            p = torch.arange(a, a + x, device="cuda")
            place.append(p)
            at.append(s["table"][n].long()[p.div(page, rounding_mode="floor")] * page + p % page)
        place, at = torch.cat(place), torch.cat(at)
        turn = lambda x, w: _rotate64(x, w, s["eps"], place, s["inv_freq"], None,  # noqa: E731
                                      s["pairs"])

        def put(pages, rows):  # rows [T][h_kv][...] into pages [P][h_kv][page][...]
            flat = pages.transpose(1, 2).flatten(0, 1).clone()
            flat[at] = rows
            return flat.unflatten(0, (-1, page)).transpose(1, 2)

        k, v = turn(s["k"], s["k_weight"]), s["v"].double()
        out = {"q": turn(s["q"], s["q_weight"])}
        for name, x in (("k", k), ("v", v)):
            old = s[name + "_pages"].float().double()
            if case["bits"] == 8:  # the quotients that its codes stand for
                x = x / _unit64(x.to(torch.bfloat16).double())
                out[name + "_unit"] = None
            out[name + "_pages"] = put(old, x)
        return out
    group, window, sinks = case["h_q"] // case["h_kv"], case["window"], case["sinks"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    first = 0
    for n, (a, b) in enumerate(zip(_numbers(case["new"]), _numbers(case["length"]))):
        at = s["table"][n, :-(-b // page)].long()
        rows = []
        for pages, exps in ((s["k_pages"], s["k_exp"]), (s["v_pages"], s["v_exp"])):
            if exps is None:
                x = pages[at].double()
            else:
                x = pages.view(torch.uint8)[at].view(torch.float8_e4m3fn).double()
                x = x * torch.exp2(exps[at].double() - 127)[..., None]
            rows.append(x.transpose(0, 1).reshape(case["h_kv"], -1, case["dim"])[:, :b])
        keys = torch.arange(b, device="cuda")
        for i in range(0, a, 512):
            j = min(a, i + 512)
            place = torch.arange(b - a + i, b - a + j, device="cuda")[:, None]
            hidden = keys > place
            if window:
                hidden |= (keys <= place - window) & (keys >= sinks)
            for h in range(case["h_q"]):
                w = s["q"][first + i:first + j, h].double() @ rows[0][h // group].T * s["scale"]
                w = torch.softmax(w.masked_fill(hidden, -math.inf), dim=1)
                o[first + i:first + j, h] = w @ rows[1][h // group]
        first += a
    return {"o": o}
