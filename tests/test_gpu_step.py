"""Rotary positions, the rotating append, the 4-bit cache, reading slots back and the adjustment of logits on the GPU,
through the binding, against plain 64-bit forms (step_reference.py, paged_reference.py).  Tolerances are the bounds
derived there; what is held in 4 or 8 bits has to be equal."""
from __future__ import annotations

import random

import pytest
import torch

import paged_reference as ref
import step_reference as sref
from step_reference import E2, Batch4

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import geometric_map_reduce_amd as gm

BF, FP, F32, E4, E8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def say(msg):
    print(msg, flush=True)


def put(t):
    return None if t is None else t.cuda()


def close(got, want, tol, what):
    got, want = got.double(), want.double()
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~(same | ((got - want).abs() <= tol))
    if bool(bad.any()):
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {got[i].item()} for "
                             f"{want[i].item()}, tolerance {tol[i].item() if torch.is_tensor(tol) else tol}")


def pools(b):
    """(pages, scales) of keys and values on the GPU, as a call takes them."""
    k, v = put(b.k), put(b.v)
    if isinstance(b, Batch4):
        return k.view(E2), v.view(E2), put(b.k_scale).view(E8), put(b.v_scale).view(E8)
    return k, v, put(b.k_scale), put(b.v_scale)


def raw(t):
    return t.cpu().view(torch.uint8)


# ---- rotary positions

ROTARY = [
    # tokens, heads, dim, rotated columns
    (1, 1, 2, 2), (1, 40, 128, 128), (7, 3, 128, 64), (33, 5, 96, 96), (5, 2, 80, 40), (64, 1, 64, 2), (3, 2, 6, 4), (9, 3, 7, 6),
    (4, 2, 256, 0), (300, 8, 256, 256), (2, 1, 4096, 4096), (1100, 2, 64, 48), (2500, 3, 32, 24), (1, 1, 1, 0),
]


@pytest.mark.parametrize("tokens,heads,dim,rot", ROTARY)
@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary(tokens, heads, dim, rot, dtype, interleaved):
    say(f"rotary {tokens} x {heads} x {dim}, {rot} turn, {dtype}, interleaved {interleaved}")
    g = torch.Generator().manual_seed(tokens * 7 + dim)
    x = torch.randn((tokens, heads, dim), generator=g).to(dtype)
    at = torch.randint(-(1 << 20), 1 << 20, (tokens,), generator=g).to(torch.int32)
    at[0] = 0 if tokens > 1 else 2 ** 31 - 1
    at[-1] = -2 ** 31 if tokens > 2 else at[-1]
    freqs = gm.keops_rotary_frequencies(rot, 500000.0) if rot else torch.zeros(0, dtype=torch.float64)
    for factor, inverse in ((1.0, False), (-1.3, True)):
        y = gm.keops_rotary(put(x), put(at), put(freqs), interleaved=interleaved, factor=factor, inverse=inverse)
        want = sref.rotate(x, at, freqs, interleaved, factor, inverse)
        close(y.cpu(), want, sref.rotate_bound(x, want, freqs, dtype, factor), "rotary")
        assert torch.equal(y[..., rot:].cpu(), x[..., rot:])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rotary_in_place_and_in_wider_rows(dtype, interleaved):
    """Queries and keys of one product's rows, in place; values beside them and guards stay."""
    for dim, rot in ((64, 64), (64, 20), (36, 36), (10, 6)):
        say(f"rotary in place, {dim} {rot} {dtype} {interleaved}")
        g = torch.Generator().manual_seed(dim)
        wide = torch.randn((50, 3, 4, dim), generator=g).to(dtype)
        at = torch.arange(50, dtype=torch.int32)
        freqs = gm.keops_rotary_frequencies(rot)
        dev = put(wide)
        x = dev[:, 1]
        want = gm.keops_rotary(x, put(at), put(freqs), interleaved=interleaved)
        assert gm.keops_rotary(x, put(at), put(freqs), interleaved=interleaved, out=x) is x
        assert torch.equal(x, want)
        ref64 = sref.rotate(wide[:, 1], at, freqs, interleaved)
        close(want.cpu(), ref64, sref.rotate_bound(wide[:, 1], ref64, freqs, dtype), "rotary")
        assert torch.equal(dev[:, 0].cpu(), wide[:, 0]) and torch.equal(dev[:, 2].cpu(), wide[:, 2])
        # from a place that 16 bytes do not divide
        flat = torch.randn(50 * 4 * dim + 1, generator=g).to(dtype)
        x = flat[1:].view(50, 4, dim)
        got = gm.keops_rotary(put(flat)[1:].view(50, 4, dim), put(at), put(freqs), interleaved=interleaved)
        ref64 = sref.rotate(x, at, freqs, interleaved)
        close(got.cpu(), ref64, sref.rotate_bound(x, ref64, freqs, dtype), "rotary")


def test_rotary_gradient():
    """The inverse rotation is the gradient: against the plain form's by autograd and against differences."""
    say("rotary gradient")
    g = torch.Generator().manual_seed(3)
    x = torch.randn((20, 3, 24), generator=g)
    dy = torch.randn((20, 3, 24), generator=g)
    at = torch.randint(0, 5000, (20,), generator=g).to(torch.int32)
    freqs = gm.keops_rotary_frequencies(16)
    for interleaved in (False, True):
        leaf = x.double().requires_grad_()
        sref.rotate(leaf, at, freqs, interleaved, 1.7).backward(dy.double())
        args = put(at), put(freqs), interleaved, 1.7
        got = gm.keops_rotary(put(dy), *args, inverse=True).cpu()
        close(got, leaf.grad, sref.rotate_bound(dy, leaf.grad, freqs, F32, 1.7), "gradient")
        # the map is linear: a difference along any direction is its value there
        h = torch.randn(x.shape, generator=g)
        step = (gm.keops_rotary(put(x + h), *args).double() - gm.keops_rotary(put(x - h), *args).double()).cpu() / 2
        # of some 1,440 products of size up to 1.7 * 4 * 4, each rounded a few times
        assert abs((step * dy).sum() - (got.double() * h).sum()) <= 1440 * 30 * 16 * ref.U32


def test_rotary_far_angles_and_non_finite():
    say("rotary far angles")
    at = torch.tensor([2 ** 31 - 1, 2 ** 30 + 7, -2 ** 31, 999999999], dtype=torch.int32)
    freqs = torch.tensor([1.0, 3.1415926535897931, 0.3, 1234.5678], dtype=torch.float64)
    x = torch.tensor([1.0, 0.5, 0.0, -2.0, 0.0, 1.0, 1.0, 3.0])[None, None].repeat(4, 1, 1)
    y = gm.keops_rotary(put(x), put(at), put(freqs))
    want = sref.rotate(x, at, freqs)
    close(y.cpu(), want, sref.rotate_bound(x, want, freqs, F32), "far angles")
    x[1, 0, 2] = float("nan")
    x[2, 0, 1] = float("inf")
    y = gm.keops_rotary(put(x), put(at), put(freqs)).cpu()
    for t, c in ((1, 2), (2, 1)):
        assert not bool(y[t, 0, [c, c + 4]].isfinite().any())
        others = [i for i in range(8) if i % 4 != c % 4]
        close(y[t, 0, others], want[t, 0, others], sref.rotate_bound(x[t:t + 1].nan_to_num(0, 0, 0), want[t:t + 1], freqs, F32)[0, 0, others], "others")


# ---- the rotating append

APPEND = [
    # lens, new, query heads, key/value heads, dim, page, rotated columns
    ([1], [1], 1, 1, 64, 16, 64), ([40, 0, 300, 7], [3, 0, 300, 1], 4, 2, 96, 20, 96), ([129] * 70, [1] * 70, 8, 4, 128, 32, 64),
    ([50, 2], [5, 4], 0, 3, 256, 1, 256), ([77], [60], 6, 2, 128, 24, 40), ([30, 900], [2, 5], 2, 1, 64, 7, 6), ([5000], [5000], 2, 1, 64, 64, 64),
]


def append_batch(lens, new, heads, kv, dim, page, dtype, cache, seed=31):
    if cache == E2:
        b = Batch4(seed, lens, new, max(heads, 1), kv, dim, page, dtype, junk=0.0)
    else:
        b = ref.Batch(seed, lens, new, max(heads, 1), kv, dim, page, dtype, cache, junk=0.0)
    wide = (torch.randn((b.T, heads + 2 * kv, dim), generator=b.gen) * 2).to(dtype)
    return b, wide


def check_append(b, wide, heads, freqs, positions, interleaved, factor, weights=None, own=False):
    """Pools, weights and queries after a call; `own`: through keops_cache_append, without a rotation."""
    kv = b.kv
    k, v, ks, vs = pools(b)
    w, dev = put(weights), put(wide)
    where = torch.tensor([0] * b.T, dtype=torch.int32)
    for t, _, j, _, _ in sref.places(b):
        where[t] = j
    at = where if positions is None else positions
    args = (k, v, put(b.table), put(b.lens_t()), put(b.starts))
    if own:
        gm.keops_cache_append(dev[:, heads:heads + kv], dev[:, heads + kv:], *args, weights=w, k_scale=ks, v_scale=vs)
        key = wide[:, heads:heads + kv]
    else:
        q = gm.keops_cache_append_rotary(dev[:, :heads], dev[:, heads:heads + kv], dev[:, heads + kv:], *args, put(freqs),
                                         positions=put(positions), interleaved=interleaved, factor=factor, weights=w, k_scale=ks, v_scale=vs)
        want = sref.rotate(wide[:, :heads], at, freqs, interleaved, factor)
        tol = sref.rotate_bound(wide[:, :heads], want, freqs, b.dtype, factor)
        close(q.cpu(), want, tol, "queries")
        key = sref.rotate(wide[:, heads:heads + kv], at, freqs, interleaved, factor)
    val = wide[:, heads + kv:]
    torch.cuda.synchronize()
    if isinstance(b, Batch4):
        for name, got, w4 in zip(("keys", "values", "powers of keys", "powers of values"), (k, v, ks, vs), sref.append_4bit(b, key, val)):
            assert torch.equal(raw(got), w4), name
    else:
        for name, got, pool, x, scale in (("keys", k, b.k, key, b.k_scale), ("values", v, b.v, val, b.v_scale)):
            got = got.cpu()
            seen = torch.zeros(pool.shape[:2], dtype=torch.bool)
            for t, s, j, pg, row in sref.places(b):
                if pg < 0:
                    continue
                seen[pg, row] = True
                if scale is None:
                    r = x[t].double()
                    tol = sref.rotate_bound(wide[t:t + 1, heads:heads + kv], r[None], freqs, b.dtype, factor)[0] if name == "keys" and not own else 0.0
                    close(got[pg, row], r, tol, name)
                elif name == "keys":
                    assert torch.equal(got[pg, row].float(), nearest_8bit(x[t].double() / scale.double()[:, None])), (name, t)
                else:
                    assert torch.equal(got[pg, row].float(), (x[t].float() / scale[:, None]).clamp(-448, 448).to(E4).float()), (name, t)
            assert torch.equal(raw(got)[~seen], raw(pool)[~seen]), name
    if weights is not None:
        want = weights.clone()
        for t, s, j, pg, row in sref.places(b):
            if pg >= 0:
                want[pg, :, row] = 0.0
        assert torch.equal(w.cpu(), want)


def nearest_8bit(x):
    """e4m3 values nearest to x in 64 bits, halfway to the even code, cut to +-448."""
    level = torch.arange(127, dtype=torch.uint8).view(E4).double()
    away = (x.abs()[..., None] - level).abs()
    code = away.argmin(-1)
    tie = (away == away.amin(-1, keepdim=True)).sum(-1) > 1
    code = torch.where(tie & (code % 2 == 1), code + 1, code)
    return torch.copysign(level[code], x).float()


@pytest.mark.parametrize("lens,new,heads,kv,dim,page,rot", APPEND)
@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FP, FP), (BF, E4), (FP, E4), (BF, E2), (FP, E2)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_rotary(lens, new, heads, kv, dim, page, rot, dtype, cache, interleaved):
    say(f"rotating append {len(lens)} sequences, {heads}/{kv} x {dim}, page {page}, {rot} turn, {dtype} {cache}, interleaved {interleaved}")
    b, wide = append_batch(lens, new, heads, kv, dim, page, dtype, cache)
    if len(lens) == 4:
        b.table[0, 0] = b.P + 5
    freqs = gm.keops_rotary_frequencies(rot, 10000.0)
    given = None
    if interleaved:
        given = torch.randint(-100000, 1 << 20, (b.T,), generator=b.gen).to(torch.int32)
    weights = torch.rand((b.P, kv, page), generator=b.gen) + 1 if kv != 4 else None
    check_append(b, wide, heads, freqs, given, interleaved, 1.0 if rot == dim else 1.25, weights)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(128, 128), (64, 24), (96, 96), (96, 40), (256, 256)])
def test_append_rotary_is_rotary(dim, rot, interleaved, dtype):
    """Queries, and keys of a 16-bit cache, have the bits that keops_rotary gives them."""
    say(f"append rotary and rotary {dim} {rot} {interleaved} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(dim + rot)
    n, page = [900, 1, 411], 64
    T = sum(n)
    q, k, v = (torch.randn((T, h, dim), generator=g, device="cuda").to(dtype) for h in (6, 2, 2))
    kp, vp = (torch.zeros((24, page, 2, dim), dtype=dtype, device="cuda") for _ in range(2))
    table = torch.randperm(24, generator=torch.Generator().manual_seed(1))[:24].int().view(1, 24).repeat(3, 1).cuda()
    table[1], table[2, :7] = table[0, 15], table[0, 16:23]
    lens = torch.tensor(n, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 900, 901, T], dtype=torch.int32, device="cuda")
    freqs = gm.keops_rotary_frequencies(rot, device="cuda")
    at = torch.cat([torch.arange(x) for x in n]).int().cuda()
    for positions, p in ((None, at), (at * 1000 - 5, at * 1000 - 5)):
        turned = gm.keops_cache_append_rotary(q, k, v, kp, vp, table, lens, starts, freqs, positions=positions, interleaved=interleaved,
                                              factor=1.25)
        assert torch.equal(turned, gm.keops_rotary(q, p, freqs, interleaved=interleaved, factor=1.25))
        kr, vr = gm.keops_cache_read(kp, vp, table, lens, starts, T)
        assert torch.equal(kr, gm.keops_rotary(k, p, freqs, interleaved=interleaved, factor=1.25)) and torch.equal(vr, v)


@pytest.mark.parametrize("cache", [E2, E4, BF])
def test_append_rotary_at_position_zero_is_the_append(cache):
    """Where nothing turns, keys come out as those of keops_cache_append, ties of every kind included."""
    say(f"rotating append at position 0, {cache}")
    b, _ = append_batch([2048], [2048], 0, 1, 64, 64, BF, cache)
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF).reshape(1024, 1, 64).repeat(2, 1, 1)
    x = torch.where(x.isnan(), torch.ones_like(x), x)
    x[1024:] = torch.randn((1024, 1, 64), generator=b.gen).to(BF).mul(4).round().div(4)         # small whole quarters: many ties
    if cache == E4:
        b.k_scale, b.v_scale = torch.tensor([0.75]), torch.tensor([0.75])
    freqs = gm.keops_rotary_frequencies(64)
    got = []
    for own in (True, False):
        k, v, ks, vs = pools(b)
        args = (put(x), put(x), k, v, put(b.table), put(b.lens_t()), put(b.starts))
        if own:
            gm.keops_cache_append(*args, k_scale=ks, v_scale=vs)
        else:
            gm.keops_cache_append_rotary(put(x)[:, :0], *args, put(freqs), positions=torch.zeros(2048, dtype=torch.int32).cuda(),
                                         k_scale=ks, v_scale=vs)
        got.append([k.cpu(), v.cpu()] + ([raw(ks), raw(vs)] if cache == E2 else []))
    for name, p, q in zip("kvxy", *got):
        if cache == BF and name == "k":
            p, q = p.float(), q.float()              # 0 (-inf) is NaN under a rotation, and -0 may be 0
            fine = p.isfinite()
            other = torch.cat([fine[..., 32:], fine[..., :32]], -1)
            assert torch.equal(p[fine & other], q[fine & other])
        elif cache == BF:
            assert torch.equal(p, q)
        elif cache == E4 and name == "k":
            # an infinity beside a value: 0 times it is NaN; a quotient rounded to 32 bits first may meet a tie
            p, q = p.float(), q.float()
            fine = p.isfinite() & q.isfinite() & (p.abs() < 448)
            assert torch.equal(p[fine], q[fine]) and fine.double().mean() > 0.7
        elif cache == E2 and name in "kx":
            # blocks next to an infinity's: 0 times it is NaN
            if name == "k":
                fine = (got[1][2] != 255).permute(0, 2, 1, 3).repeat_interleave(16, -1)
                a, c = raw(p), raw(q)
                # the sign of a zero does not count
                zero = lambda t: t & ~(((t & 0x07) == 0).byte() * 0x08) & ~(((t & 0x70) == 0).byte() * 0x80)  # noqa: E731
                assert torch.equal(zero(a)[fine], zero(c)[fine])
            else:
                assert torch.equal(p[q != 255], q[q != 255])
        else:
            assert torch.equal(raw(p), raw(q))


def test_append_rotary_extreme_scales():
    """An e4m3 cache's quotients by infinite, zero, subnormal and huge scales are the append's."""
    say("append rotary, extreme scales")
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn((40, 4, 64), generator=g, device="cuda").bfloat16() for _ in range(2))
    k[3] = 0
    scale = torch.tensor([float("inf"), 0.0, 2.0 ** -140, 3e38]).cuda()
    table = torch.arange(3, dtype=torch.int32, device="cuda").view(1, 3)
    lens, starts = torch.tensor([40], dtype=torch.int32).cuda(), torch.tensor([0, 40], dtype=torch.int32).cuda()
    held = []
    for turn in (False, True):
        kp, vp = (torch.zeros((3, 16, 4, 64), dtype=torch.uint8, device="cuda").view(E4) for _ in range(2))
        if turn:
            gm.keops_cache_append_rotary(k[:, :0], k, v, kp, vp, table, lens, starts, gm.keops_rotary_frequencies(64, device="cuda"),
                                         positions=torch.zeros(40, dtype=torch.int32, device="cuda"), k_scale=scale, v_scale=scale)
        else:
            gm.keops_cache_append(k, v, kp, vp, table, lens, starts, k_scale=scale, v_scale=scale)
        held.append((raw(kp), raw(vp)))
    assert bool((held[0][0][:, :, 0] & 0x7f == 0).all())
    for x, y in zip(*held):
        none = (x & 0x7f == 0x7f) & (y & 0x7f == 0x7f)
        assert bool((none | (x == y)).all())


def test_append_4bit_every_16_bit_value():
    """Every bf16 and fp16 value, in blocks of one magnitude and in blocks of all: least powers, subnormals, infinities."""
    for dtype in (BF, FP):
        for order in ("rows", "columns"):
            say(f"append in 4 bits, every {dtype}, {order}")
            x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
            x = x.reshape(1024, 1, 64) if order == "rows" else x.reshape(64, 1, 1024).permute(2, 1, 0).contiguous()
            b = Batch4(37, [1024], [1024], 1, 1, 64, 64, dtype, junk=0.0)
            wide = torch.cat([x, x], 1)
            check_append(b, wide, 0, None, None, False, 1.0, own=True)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("lens,new,heads,kv,dim,page,rot", APPEND)
def test_append_4bit(lens, new, heads, kv, dim, page, rot, dtype):
    say(f"append in 4 bits {len(lens)} sequences, {kv} x {dim}, page {page}, {dtype}")
    b, wide = append_batch(lens, new, heads, kv, dim, page, dtype, E2)
    if len(lens) == 4:
        b.table[0, 0] = -7
    wide[0, -1, 3] = float("nan")
    check_append(b, wide, heads, None, None, False, 1.0, torch.rand((b.P, kv, page), generator=b.gen) + 1, own=True)


def test_append_rotary_rows_of_no_sequence_stay():
    say("rotating append, rows behind the last sequence")
    b, wide = append_batch([20, 9], [3, 2], 4, 2, 64, 16, BF, BF)
    wide = torch.cat([wide, torch.randn((4, 8, 64), generator=b.gen).to(BF)])
    k, v, _, _ = pools(b)
    dev, out = put(wide), torch.full((9, 4, 64), 7.0, dtype=BF, device="cuda")
    freqs = gm.keops_rotary_frequencies(64).cuda()
    gm.keops_cache_append_rotary(dev[:, :4], dev[:, 4:6], dev[:, 6:], k, v, put(b.table), put(b.lens_t()), put(b.starts), freqs, out=out)
    assert bool((out[5:] == 7).all()) and not bool((out[:5] == 7).any())
    # fewer slots than new tokens: a token before the first slot has its query turned to its place before it
    lens = torch.tensor([1, 9], dtype=torch.int32)
    out2 = gm.keops_cache_append_rotary(dev[:5, :4], dev[:5, 4:6], dev[:5, 6:], k, v, put(b.table), lens.cuda(), put(b.starts), freqs)
    at = torch.tensor([-2, -1, 0, 7, 8], dtype=torch.int32)
    want = sref.rotate(wide[:5, :4], at, freqs.cpu())
    close(out2.cpu(), want, sref.rotate_bound(wide[:5, :4], want, freqs.cpu(), BF), "queries")


# ---- attention over 4 bits

def run_attention(b, decay=0.0, max_len=None, **kw):
    w = put(b.weights)
    k, v, ks, vs = pools(b)
    out, lse = gm.keops_paged_attention(put(b.q), k, v, put(b.table), put(b.lens_t()), put(b.starts), max(b.new + [0]),
                                        max(b.lens + [0]) if max_len is None else max_len, scale=b.scale, window=b.window, weights=w,
                                        decay=decay, k_scale=ks, v_scale=vs, **kw)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu(), None if w is None else w.cpu()


def check_attention(b, decay=0.0, **kw):
    out, lse, w = run_attention(b, decay, **kw)
    o, z, ww, ot, zt, wt = ref.attention(b, decay)
    close(lse, z, zt, "lse")
    close(out, o, ot, "out")
    if w is not None:
        close(w, ww, wt, "weights")


ATTEND = [
    # lens, new, query heads, key/value heads, dim, page, type, window
    ([1], [1], 1, 1, 64, 16, BF, 0), ([1], [1], 8, 2, 128, 16, FP, 0), ([33], [1], 4, 1, 128, 16, BF, 0),
    ([1000], [1], 32, 8, 128, 16, BF, 0), ([1000, 1, 77, 513], [1, 1, 1, 1], 8, 2, 64, 20, FP, 0),
    ([300, 129, 4000], [4, 2, 3], 8, 2, 128, 32, BF, 0), ([300, 0, 40], [4, 0, 3], 10, 2, 96, 24, FP, 0),
    ([700, 64], [9, 1], 14, 2, 96, 7, BF, 0), ([500, 31], [3, 2], 7, 1, 256, 64, BF, 100), ([260], [1], 5, 1, 256, 128, FP, 33),
    ([200, 90], [4, 3], 8, 1, 256, 16, FP, 0), ([64, 65, 63], [64, 65, 63], 4, 2, 64, 16, BF, 0),
    ([130, 257], [130, 200], 4, 1, 128, 24, FP, 0), ([300], [150], 2, 1, 96, 128, BF, 0), ([333, 80], [40, 80], 8, 2, 256, 20, BF, 0),
    ([222], [60], 8, 1, 256, 16, FP, 17), ([2000], [12], 8, 1, 128, 64, BF, 0), ([777, 400, 100], [300, 10, 100], 8, 4, 64, 24, FP, 128),
    ([1500], [5], 8, 8, 128, 1, BF, 64), ([1500], [3], 4, 2, 96, 64, BF, 0), ([27000, 300], [2, 1], 5, 1, 64, 64, BF, 0),
    # widened to 16 bits first
    ([500, 90, 0, 70], [270, 90, 0, 1], 8, 2, 64, 24, FP, 0), ([400], [130], 8, 1, 128, 16, BF, 0), ([300, 290], [140, 1], 8, 1, 96, 7, BF, 50),
    ([290], [260], 8, 2, 256, 64, FP, 130), ([1100, 300], [130, 128], 8, 1, 64, 1, BF, 65),
]


@pytest.mark.parametrize("lens,new,heads,kv,dim,page,dtype,window", ATTEND)
@pytest.mark.parametrize("weights", [False, True])
def test_attention(lens, new, heads, kv, dim, page, dtype, window, weights):
    say(f"attention in 4 bits {lens} {new} {heads}/{kv} {dim} page {page} {dtype} window {window} weights {weights}")
    b = Batch4(sum(lens) + dim, lens, new, heads, kv, dim, page, dtype)
    b.window = window
    if weights:
        b.weights = torch.rand((b.P, kv, page), generator=b.gen)
    check_attention(b, decay=0.5 if weights and len(lens) > 1 else 0.0)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("new,weights", [(1, False), (2, True), (7, False), (6, True)])
def test_attention_past_the_caches(dtype, dim, new, weights):
    say(f"attention in 4 bits past the caches, {dtype}, dim {dim}, {new} new, weights {weights}")
    b = Batch4(73, [300, 77, 40], [new, 1, 0], 8, 2, dim, 24, dtype)
    if weights:
        b.weights = torch.zeros((b.P, 2, 24))
    check_attention(b, max_len=1 << 21)                     # 2 x 3 x 2 x 2^21 rows of 34 bytes: 428 MB and more


@pytest.mark.parametrize("dim,kv,dtype", [(64, 4, BF), (64, 2, FP), (64, 3, BF), (96, 4, FP), (96, 8, BF), (96, 1, BF), (128, 8, BF), (128, 6, FP),
                                          (128, 5, BF), (256, 2, BF), (64, 12, BF), (128, 2, FP)])
@pytest.mark.parametrize("new,group,window,weights", [(1, 4, 0, False), (3, 2, 0, False), (2, 9, 70, False), (1, 1, 0, True)])
def test_attention_heads_together(dim, kv, dtype, new, group, window, weights):
    """Bounds under which one, two or four neighbouring heads go together, in runs over several sequences."""
    say(f"neighbouring heads, {kv} x {dim}, {dtype}, {new} new, group {group}, window {window}, weights {weights}")
    lens = [700, 0, 333, 90, 1025]
    b = Batch4(61 + dim + kv, lens, [min(new, n) for n in lens], kv * group, kv, dim, 24, dtype)
    b.window = window
    b.table[0, 3] = -1
    if weights:
        b.weights = torch.rand((b.P, kv, 24), generator=b.gen)
    check_attention(b, max_len=30000)


@pytest.mark.parametrize("dim,new,dtype,kv", [(64, 3, BF, 2), (128, 3, FP, 2), (96, 3, BF, 2), (256, 3, BF, 2), (64, 40, BF, 2), (128, 40, FP, 2),
                                              (256, 40, BF, 2), (96, 40, FP, 2), (128, 3, BF, 2), (128, 40, BF, 2), (64, 3, BF, 4), (96, 3, FP, 8),
                                              (128, 3, BF, 6), (64, 100, BF, 2), (128, 100, FP, 2), (256, 100, BF, 4), (96, 90, BF, 2)])
@pytest.mark.parametrize("max_len", [None, 30000])
def test_hidden_values_reach_no_row(dim, new, dtype, kv, max_len):
    """NaN blocks and blocks past the type's largest number, in the key and value of a later token and below the window,
    change nothing for the rows that do not see them; the rows that see them get what the formula gives."""
    say(f"hidden non-finite blocks, {kv} x {dim}, {new} new, {dtype}, bound {max_len}")
    group = 12 if new > 80 else 2                            # 12: widened to 16 bits first, but under the wider bound
    b = Batch4(9, [240], [new], group * kv, kv, dim, 16, dtype)
    b.window = 101
    first = 240 - new
    spots = (239, first - 100, first + 1)
    for j in spots:
        pg, row = b.table[0, j // 16].item(), j % 16
        b.v_scale[pg, 0, row, 0] = 255                       # a block of NaN
        b.v[pg, row, 1] = 0
        b.v[pg, row, 1, 20] = 0x07                           # column 40 alone
        b.v_scale[pg, 1, row, 1] = 254 if dtype == BF else 142
    pg, row = b.table[0, 239 // 16].item(), 239 % 16
    b.k_scale[pg, 0, row, 0] = 255
    out, lse, _ = run_attention(b, max_len=max_len)
    o, z, _, ot, zt, _ = ref.attention(b)
    for t in range(new):
        sees = [j for j in spots if first + t - 101 < j <= first + t]
        for h in range(group * kv):
            if not sees or h >= 2 * group:
                assert bool(out[t, h].isfinite().all()) and bool(lse[t, h].isfinite())
                close(out[t, h], o[t, h], ot[t, h], f"row {t}")
                continue
            if h < group:
                assert bool(out[t, h, :32].isnan().all()), (t, h)
                if 239 not in sees:
                    assert bool(out[t, h, 32:].isfinite().all())
                    close(out[t, h, 32:], o[t, h, 32:], ot[t, h, 32:], f"row {t}")
            else:
                assert out[t, h, 40] == float("inf"), (t, h, out[t, h, 40])
                rest = [c for c in range(dim) if c != 40]
                close(out[t, h, rest], o[t, h, rest], ot[t, h, rest], f"row {t}")


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("new,group,weights", [(1, 1, False), (1, 4, True), (4, 4, False), (3, 5, True), (6, 4, False), (40, 4, True), (260, 4, False)])
@pytest.mark.parametrize("max_len", [None, 30000])
def test_infinite_values_that_every_row_sees(dim, dtype, new, group, weights, max_len):
    """Blocks of NaN and past the type's largest number in slots that every row sees, of a tile in the middle, of the last
    one and of the first new token: the columns with them are what the formula gives, the others are as close as ever."""
    say(f"infinite blocks, dim {dim}, {new} new, group {group}, {dtype}, weights {weights}, bound {max_len}")
    kv, n = (4 if dim < 256 else 2), 200 + new
    b = Batch4(19 + dim, [n], [new], kv * group, kv, dim, 16, dtype)
    b.q = (b.q / 4).to(dtype)                                # every weight is far above what 16 bits end at
    if weights:
        b.weights = torch.rand((b.P, kv, 16), generator=b.gen)
    top = 254 if dtype == BF else 142                        # 6 under it is infinite
    for i, j in enumerate((5, 100, 200)):                    # 200: the first new token's own
        pg, row = b.table[0, j // 16].item(), j % 16
        for h in range(1, kv):
            b.v_scale[pg, h, row, 1] = top
            b.v[pg, row, h, 16:32] = 0
            b.v[pg, row, h, 20] = (0x07, 0x70, 0xf7)[i]      # column 40: +, 0, +; column 41: 0, +, -
            b.v[pg, row, h, 24] = (0x7f, 0x00, 0x00)[i]      # column 48: -; 49: +
    pg, row = b.table[0, 33 // 16].item(), 33 % 16
    b.v_scale[pg, 0, row, 0] = 255
    out, lse, w = run_attention(b, max_len=max_len)
    o, z, ww, ot, zt, wt = ref.attention(b)
    close(lse, z, zt, "lse")
    if weights:
        close(w, ww, wt, "weights")
    inf = float("inf")
    for h in range(kv):
        got, want, tol = (x[:, h * group:(h + 1) * group] for x in (out, o, ot))
        odd = list(range(32)) if h == 0 else [40, 41, 48, 49]
        rest = [c for c in range(dim) if c not in odd]
        assert bool(got[..., rest].isfinite().all()), h
        close(got[..., rest], want[..., rest], tol[..., rest], f"head {h}")
        if h == 0:
            assert bool(got[..., odd].isnan().all())
        else:
            assert bool((got[..., 40] == inf).all()) and bool(got[..., 41].isnan().all()), (h, got[0, 0, odd])
            assert bool((got[..., 48] == -inf).all()) and bool((got[..., 49] == inf).all()), (h, got[0, 0, odd])


@pytest.mark.parametrize("new,heads", [(1, 2), (3, 8), (20, 2), (40, 2), (260, 8)])
def test_fp16_rows_over_what_bf16_rows_held(new, heads):
    """A value past fp16's largest number that bf16 rows left in a 4-bit cache is an infinity to fp16 rows."""
    say(f"fp16 rows over a cache of bf16 rows, {new} new, {heads} heads")
    n = 300 + new
    b, _ = append_batch([n], [n], heads, 2, 64, 16, BF, E2)
    k, v, ks, vs = pools(b)
    rows = torch.randn((n, 2, 64), generator=b.gen).to(BF)
    rows[:, 1, 32:] = 0                                      # under the power of 10^5, other values are 0 or infinite too
    rows[7, 1, 37], rows[150, 1, 50], rows[300, 1, 63] = 1e5, -1e5, 1e5
    args = (put(b.table), put(b.lens_t()))
    keys = torch.randn((n, 2, 64), generator=b.gen).to(BF)
    gm.keops_cache_append(put(keys), put(rows), k, v, *args, put(b.starts), k_scale=ks, v_scale=vs)
    q = (torch.randn((new, heads, 64), generator=b.gen) / 2).half()
    starts = torch.tensor([0, new], dtype=torch.int32).cuda()
    out = gm.keops_paged_attention(put(q), k, v, *args, starts, new, n, k_scale=ks, v_scale=vs)[0].cpu()
    inf, group = float("inf"), heads // 2
    want = torch.zeros(32)
    want[37 - 32], want[50 - 32], want[63 - 32] = inf, -inf, inf
    assert bool(out[:, :group].isfinite().all()) and bool(out[:, group:, :32].isfinite().all())
    assert torch.equal(out[:, group:, 32:].float(), want.expand(new, group, 32))


@pytest.mark.parametrize("dim,dtype", [(64, BF), (64, FP), (96, BF), (96, FP)])
@pytest.mark.parametrize("group", [1, 4, 6])
def test_hidden_infinities_of_heads_that_go_together(dim, dtype, group):
    """A work-group's four waves have a head each (their bounds fill the device): an infinity in the last slot of one head
    reaches that head's last row, all its lanes, and nothing else."""
    say(f"hidden infinities, four heads together, dim {dim}, group {group}, {dtype}")
    new, kv = 3, 8
    for first in (0, 2, 7):
        b = Batch4(29, [300], [new], group * kv, kv, dim, 16, dtype)
        pg, row = b.table[0, 299 // 16].item(), 299 % 16
        b.v_scale[pg, first, row] = 254 if dtype == BF else 142
        b.v[pg, row, first] = 0x77                           # 6 under that, in every column
        out, lse, _ = run_attention(b, max_len=30000)
        o, z, _, ot, zt, _ = ref.attention(b)
        close(lse, z, zt, "lse")
        there = torch.zeros((new, group * kv), dtype=torch.bool)
        there[-1, first * group:(first + 1) * group] = True
        assert bool((out[there] == float("inf")).all()) and bool(out[~there].isfinite().all())
        close(out[~there], o[~there], ot[~there], "rows without it")


@pytest.mark.parametrize("cache,dim,rows,least", [(E4, 64, 16, 4), (E4, 64, 32, 2), (E4, 96, 16, 3), (E4, 96, 32, 2), (E4, 128, 16, 3), (E4, 128, 32, 2),
                                                  (E4, 256, 16, 1), (E4, 256, 32, 1), (BF, 64, 16, 3), (BF, 64, 32, 2), (BF, 96, 16, 2),
                                                  (BF, 96, 32, 2), (BF, 128, 16, 2), (BF, 128, 32, 1), (BF, 256, 16, 1), (BF, 256, 32, 1)])
def test_work_groups_of_a_compute_unit(cache, dim, rows, least):
    """As many work-groups of few-rows attention share a compute unit as did before there were 4-bit caches: seen from the
    workspace, which has two parts of 16 or 32 rows, their sums and their maxima, for each of them."""
    import ctypes
    from geometric_map_reduce_amd import paged
    say(f"work-groups of a compute unit, {cache}, {dim}, {rows} rows")
    S, n = 64, 1 << 17
    k = torch.zeros((8, 16, 8, dim), dtype=torch.uint8 if cache == E4 else cache, device="cuda")
    k = k.view(E4) if cache == E4 else k
    scale = torch.ones(8, device="cuda") if cache == E4 else None
    table, lens = torch.zeros((S, n // 16), dtype=torch.int32, device="cuda"), torch.zeros(S, dtype=torch.int32, device="cuda")
    c = paged._cache(k, k, None, table, lens, scale, scale)[0]
    need = ctypes.c_int64(0)
    assert gm.lib().keops_paged_attention_workspace(c, 0, 8 * rows, S, 1, n, 0, ctypes.byref(need)) == 0
    groups = (need.value - 512) / (2 * rows * (dim * 4 + 8))
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert groups / cus > least - 0.01, (groups, cus)


@pytest.mark.parametrize("new,heads", [(2, 8), (30, 8), (40, 64)])
def test_absent_pages(new, heads):
    say(f"absent pages in 4 bits, {new} new, {heads} heads")
    b = Batch4(11, [100, 64], [new, new], heads, 2, 64, 16)
    b.weights = torch.rand((b.P, 2, 16), generator=b.gen)
    b.table[0, 1] = -1
    b.table[0, 3] = b.P
    b.table[1, :4] = 2 ** 31 - 1
    check_attention(b)
    out, lse, _ = run_attention(b)
    assert bool((out[new:] == 0).all()) and bool((lse[new:] == -float("inf")).all())
    b.table = b.table[:, :5].contiguous()
    check_attention(b)


@pytest.mark.parametrize("seed", range(24))
def test_attention_random(seed):
    rng = random.Random(seed)
    S, kv, dim = rng.choice([1, 2, 5, 70]), rng.choice([1, 2, 4]), rng.choice([64, 96, 128, 256])
    top = rng.choice([1, 1, 3, 6, 40, 150])
    lens, new = [], []
    for _ in range(S):
        n = rng.choice([0, 1, rng.randint(1, 50), rng.randint(1, 500 if S < 70 else 90)])
        lens.append(n)
        new.append(min(n, rng.randint(0, top)))
    if not sum(new):
        lens, new = lens + [9], new + [2]
    heads, page = kv * rng.choice([1, 2, 4, 5]), rng.choice([1, 5, 16, 20, 64, 128])
    dtype, window, weights = rng.choice([BF, FP]), rng.choice([0, 0, 1, 37, 200]), rng.random() < 0.5
    say(f"random attention in 4 bits {seed}: {S} sequences, {heads}/{kv} x {dim} page {page} {dtype} window {window} weights {weights} "
        f"lens {lens[:6]} new {new[:6]}")
    b = Batch4(seed, lens, new, heads, kv, dim, page, dtype)
    b.window = window
    if weights:
        b.weights = torch.rand((b.P, b.kv, b.page), generator=b.gen)
    check_attention(b, decay=0.25 if weights and seed % 2 else 0.0)


@pytest.mark.parametrize("new", [1, 33])
def test_strides(new):
    """Keys and values interleaved in one pool, heads outside slots."""
    say(f"strides of a 4-bit cache, {new} new")
    b = Batch4(13, [90, 41], [new, min(new, 41)], 8, 2, 128, 16, junk=0.0)
    want = run_attention(b)
    both = torch.stack([b.k, b.v], 1).cuda().view(E2)
    heads = torch.stack([b.k, b.v], 1).transpose(2, 3).contiguous().cuda().transpose(2, 3).view(E2)
    ks, vs = put(b.k_scale).view(E8), put(b.v_scale).view(E8)
    for pool in (both, heads):
        out, lse = gm.keops_paged_attention(put(b.q), pool[:, 0], pool[:, 1], put(b.table), put(b.lens_t()), put(b.starts), new, 90,
                                            k_scale=ks, v_scale=vs)
        assert torch.equal(out.cpu(), want[0]) and torch.equal(lse.cpu(), want[1])
        k, v = gm.keops_cache_read(pool[:, 0], pool[:, 1], put(b.table), put(b.lens_t()), put(b.starts), b.T, k_scale=ks, v_scale=vs)
        for got, p, s in ((k, b.k, b.k_scale), (v, b.v, b.v_scale)):
            for t, _, _, pg, row in sref.places(b):
                assert torch.equal(got[t].cpu().double(), sref.from_4bit(p[pg, row], s[pg, :, row]))


@pytest.mark.parametrize("dtype", [BF, FP])
def test_read_of_8_bits_is_rounded_once(dtype):
    """An e4m3 value times its scale has up to 28 bits: where these lie just beside a tie of the 16-bit type, 32 bits have
    only the tie.  Every value, under scales that put some of them there."""
    say(f"reading 8 bits, next to ties, {dtype}")
    import math
    from fractions import Fraction
    codes = [c for c in range(256) if c & 0x7f != 0x7f]
    value = torch.tensor(codes, dtype=torch.uint8).view(E4).double().tolist()
    place = torch.finfo(dtype).eps / 2                       # of a tie, beside 1
    near = []
    for m in (9, 11, 13, 15):                                # odd parts of e4m3 values
        for i in range(8):
            tie = Fraction(1) + Fraction(2 * i + 1) * Fraction(place)
            s = float(torch.tensor(float(tie * 8 / m), dtype=torch.float64).float())
            for _ in range(40):
                x = Fraction(s) * m / 8
                s2 = float(torch.tensor(float(x), dtype=torch.float64).float())
                if x != tie and Fraction(s2) == tie:
                    near.append(s)
                    break
                s = float(torch.nextafter(torch.tensor(s, dtype=torch.float32), torch.tensor(0.0)))
    assert len(near) >= 4, near
    H = len(near)
    k = torch.zeros((16, 16, H, 64), dtype=torch.uint8)
    k[:] = torch.tensor(codes + [0, 0], dtype=torch.uint8).repeat(16 * 16 * 64 // 256).view(16, 16, 1, 64)
    scale = torch.tensor(near, dtype=torch.float32)
    table = torch.arange(16, dtype=torch.int32)[None]
    n = torch.tensor([256], dtype=torch.int32)
    starts = torch.tensor([0, 256], dtype=torch.int32)
    got = gm.keops_cache_read(put(k).view(E4), put(k).view(E4), put(table), put(n), put(starts), 256, dtype=dtype, k_scale=put(scale),
                              v_scale=put(scale))
    bits = 1 - int(math.log2(torch.finfo(dtype).eps))        # of a number of the type
    low = -24 if dtype == FP else -133                       # the smallest one's power
    for h in range(H):
        for i, x in enumerate(value):
            want = Fraction(x) * Fraction(float(scale[h]))
            step = Fraction(2) ** max(math.frexp(float(want))[1] - bits, low)
            nearest = float(round(want / step) * step)       # a tie goes to the even one
            for t in got:
                assert t[i // 64, h, i % 64].item() == nearest, (h, x, float(scale[h]), float(want))


@pytest.mark.parametrize("lens,new,heads,kv,dim,dtype,window", [([400], [130], 8, 1, 128, BF, 0), ([500, 90, 0, 70], [270, 90, 0, 1], 8, 2, 64, FP, 0),
                                                               ([300, 290], [140, 140], 8, 1, 96, BF, 50), ([290], [260], 8, 2, 256, FP, 130)])
def test_attention_without_memory_to_widen(lens, new, heads, kv, dim, dtype, window):
    """Where there is no memory for the slots in 16 bits, prompts over a 4-bit cache are attended without."""
    say(f"no memory to widen, {lens} {new} {heads}/{kv} x {dim} {dtype} window {window}")
    b = Batch4(sum(lens) + dim, lens, new, heads, kv, dim, 24, dtype)
    b.window = window
    check_attention(b)
    gm.keops_set_option(gm.KEOPS_OPT_FAIL_ALLOC, 1)
    try:
        check_attention(b)
    finally:
        gm.keops_set_option(gm.KEOPS_OPT_FAIL_ALLOC, 0)
    # a call whose form without it needs workspace too has none: nothing is enqueued
    b = Batch4(7, [1300], [130], 8, 1, 64, 24, BF)
    k, v, ks, vs = pools(b)
    out, lse = torch.full((130, 8, 64), 3.0, dtype=BF, device="cuda"), torch.full((130, 8), 3.0, device="cuda")
    gm.keops_set_option(gm.KEOPS_OPT_FAIL_ALLOC, 1)
    try:
        with pytest.raises(gm.KeopsError) as e:
            gm.keops_paged_attention(put(b.q), k, v, put(b.table), put(b.lens_t()), put(b.starts), 130, 1300, k_scale=ks, v_scale=vs, out=out, lse=lse)
        assert e.value.status == -3
    finally:
        gm.keops_set_option(gm.KEOPS_OPT_FAIL_ALLOC, 0)
    torch.cuda.synchronize()
    assert bool((out == 3).all()) and bool((lse == 3).all())


def test_far_pages():
    """Byte offsets past 2^32 in the pool, and numbers of slots and heads past 2^31."""
    say("far pages of a 4-bit cache")
    b = Batch4(17, [70], [2], 8, 4, 64, 16, junk=0.0)
    P = (2 ** 31 + 2 ** 28) // (16 * 4)
    k, v = (torch.zeros((P, 16, 4, 32), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((P, 4, 16, 2), 127, dtype=torch.uint8, device="cuda") for _ in range(2))
    far = torch.arange(P - b.table.shape[1], P, dtype=torch.int32)
    for to, frm in ((k, b.k), (v, b.v), (ks, b.k_scale), (vs, b.v_scale)):
        to[far.long().cuda()] = put(frm)[put(b.table)[0].long()]
    cache = (k.view(E2), v.view(E2), far[None].cuda(), put(b.lens_t()), put(b.starts))
    scales = dict(k_scale=ks.view(E8), v_scale=vs.view(E8))
    o, z, _, ot, zt, _ = ref.attention(b)
    for max_q in (2, 40, 600):                                # each form
        out, lse = gm.keops_paged_attention(put(b.q), *cache, max_q, 70, **scales)
        close(out.cpu(), o, ot, "out")
        close(lse.cpu(), z, zt, "lse")
    nk, nv = torch.randn((2, 4, 64)).to(BF), torch.randn((2, 4, 64)).to(BF)
    gm.keops_cache_append(put(nk), put(nv), *cache, **scales)
    codes, power = sref.to_4bit(nk, BF)
    assert torch.equal(k[P - 1, 4:6].cpu(), codes) and torch.equal(ks[P - 1, :, 4:6].cpu(), power.permute(1, 0, 2))
    rk, rv = gm.keops_cache_read(*cache, 2, **scales)
    assert torch.equal(rk.cpu().double(), sref.from_4bit(codes, power))
    assert torch.equal(rv.cpu().double(), sref.from_4bit(*sref.to_4bit(nv, BF)))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("new,weights", [(1, False), (1, True), (4, False)])
def test_few_rows_lose_no_more_than_the_outputs_rounding(dim, dtype, new, weights):
    """Up to 16 rows: what is left of p's rounding is multiplied with V too.

    p as two parts is off by half * half of itself.  A score is off by (dim + 8) 2^-24 of the sum of its products' magnitudes
    (additions in 32 bits), which p is off by relatively, numerator and sum alike; exp2 and the sums of n terms add
    (n + 8) 2^-24 each.  That times sum p |v| / sum p, and the output's own rounding."""
    say(f"few rows over 4 bits, {dim} {dtype} {new} {weights}")
    b = Batch4(61, [5, 40, 300, 1900], [new] * 4, 8, 2, dim, 16, dtype, junk=0.0)
    if weights:
        b.weights = torch.zeros((b.P, 2, 16))
    out = run_attention(b)[0].double()
    k, v, ks, vs = pools(b)
    whole = torch.tensor([0] + b.lens, dtype=torch.int32).cumsum(0).int()
    K, V = (t.double().cpu() for t in gm.keops_cache_read(k, v, put(b.table), put(b.lens_t()), whole.cuda(), int(whole[-1]), dtype=dtype,
                                                          k_scale=ks, v_scale=vs))
    half, scale = torch.finfo(dtype).eps / 2, dim ** -0.5 if b.scale is None else b.scale
    for s, n in enumerate(b.lens):
        a, e, at = int(b.starts[s]), int(b.starts[s + 1]), int(whole[s])
        for h in range(8):
            q, kk, vv = b.q[a:e, h].double(), K[at:at + n, h // 4], V[at:at + n, h // 4]
            z = q @ kk.T * scale
            off = ((q.abs() @ kk.abs().T) * abs(scale)).amax(1) * (dim + 8) * 2.0 ** -24
            z.masked_fill_(torch.arange(n) > torch.arange(n - (e - a), n)[:, None], -float("inf"))
            p = torch.softmax(z, -1)
            o = p @ vv
            near = (half * half + 2 * off + 2 * (n + 8) * 2.0 ** -24)[:, None] * (p @ vv.abs())
            floor = 2.0 ** -25 if dtype is FP else 0.0
            close(out[a:e, h], o, o.abs() * half + near * (1 + half) + floor, "out")


@pytest.mark.parametrize("lens,new", [([700, 60, 31], [300, 1, 2]), ([700, 600, 31], [300, 256, 2]), ([300, 1, 0, 290], [300, 1, 0, 290])])
@pytest.mark.parametrize("weights", [False, True])
def test_prompts_beside_single_tokens(lens, new, weights):
    """Prompts whose caches are widened first, and ones that are not since most sequences have few rows."""
    say(f"prompts beside single tokens {lens} {new} {weights}")
    b = Batch4(57, lens, new, 8, 2, 64, 16)
    if weights:
        b.weights = torch.rand((b.P, 2, 16), generator=b.gen)
    check_attention(b, 0.5)


def test_widened_slots_do_not_see_what_was_left():
    """The workspace of a call that widens the cache first holds NaN of another one."""
    say("a workspace full of NaN")
    for window in (0, 100):
        b = Batch4(33, [500, 333], [140, 130], 8, 1, 64, 16)
        b.window = window
        k, v, ks, vs = pools(b)
        args = (put(b.q), k, v, put(b.table), put(b.lens_t()), put(b.starts), 140, 500)
        kw = dict(k_scale=ks, v_scale=vs, window=window)
        st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=st):
            fill = torch.empty(16 << 20, dtype=torch.uint8, device="cuda").fill_(255)
            del fill                                         # its memory is the workspace's next
            out, lse = gm.keops_paged_attention(*args, **kw)
        o, z, _, ot, zt, _ = ref.attention(b)
        for _ in range(3):
            graph.replay()
            torch.cuda.synchronize()
            close(out.cpu(), o, ot, "out")
            close(lse.cpu(), z, zt, "lse")


def test_results_repeat_on_every_stream():
    """The same bits on the current stream, on another, and under a graph that is replayed between eager calls."""
    for new in (1, 40, 300):
        say(f"4-bit attention repeated, {new} new")
        b = Batch4(29, [2000, 700], [new, new], 8, 2, 128, 16, junk=0.0)
        k, v, ks, vs = pools(b)
        args = (put(b.q), k, v, put(b.table), put(b.lens_t()), put(b.starts), new, 2000)
        kw = dict(k_scale=ks, v_scale=vs)
        want = gm.keops_paged_attention(*args, **kw)
        st = torch.cuda.Stream()
        torch.cuda.synchronize()
        here, there = gm.keops_paged_attention(*args, **kw), gm.keops_paged_attention(*args, stream=st, **kw)     # two at once
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            cap = gm.keops_paged_attention(*args, **kw)
        for got in (here, there):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for _ in range(3):
            cap[0].zero_()
            cap[1].zero_()
            graph.replay()
            eager = gm.keops_paged_attention(*args, **kw)
            torch.cuda.synchronize()
            for got in (cap, eager):
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ---- eviction and reading

@pytest.mark.parametrize("lens,heads,dim,page,budget,sink,recent", [
    ([1], 1, 64, 16, 1, 0, 0), ([20, 5, 17], 2, 64, 16, 16, 1, 4), ([100, 33], 2, 96, 24, 32, 4, 28), ([257], 1, 256, 20, 100, 0, 50),
    ([300, 10], 3, 128, 7, 11, 0, 0)])
def test_evict(lens, heads, dim, page, budget, sink, recent):
    say(f"evict from 4 bits {lens} {heads} x {dim} page {page} budget {budget} sink {sink} recent {recent}")
    more = sum(-(-min(n, budget) // page) for n in lens)
    b = Batch4(41, lens, [0] * len(lens), heads, heads, dim, page, BF, junk=0.0, spare=more + 1)
    b.weights = torch.rand((b.P, heads, page), generator=b.gen)
    width = max(-(-min(n, budget) // page) for n in lens)
    new = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(lens):
        c = -(-min(n, budget) // page)
        new[s, :c] = b.free[at:at + c]
        at += c
    rkept, rl, rk, rv, rw = ref.evict(b, new, budget, sink, recent)
    rks, rvs = b.k_scale.clone(), b.v_scale.clone()
    for s in range(len(lens)):
        for h in range(heads):
            for r, j in enumerate(rkept[s, h].tolist()):
                if j >= 0:
                    frm, to = b.table[s, j // page].item(), new[s, r // page].item()
                    rks[to, h, r % page], rvs[to, h, r % page] = b.k_scale[frm, h, j % page], b.v_scale[frm, h, j % page]
    k, v, ks, vs = pools(b)
    w = put(b.weights)
    kept, nl = gm.keops_cache_evict(k, v, w, put(b.table), put(b.lens_t()), put(new), budget, sink=sink, recent=recent, k_scale=ks,
                                    v_scale=vs)
    for name, got, want in (("lens", nl, rl), ("kept", kept, rkept), ("keys", k, rk), ("values", v, rv), ("weights", w, rw),
                            ("powers of keys", ks, rks), ("powers of values", vs, rvs)):
        assert torch.equal(raw(got), want.view(torch.uint8)), name


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FP, FP), (BF, E4), (FP, E4), (BF, E2), (FP, E2)])
@pytest.mark.parametrize("lens,new,heads,kv,dim,page,rot", APPEND)
def test_read(lens, new, heads, kv, dim, page, rot, dtype, cache):
    say(f"read {len(lens)} sequences, {kv} x {dim}, page {page}, {dtype} {cache}")
    b, _ = append_batch(lens, new, heads, kv, dim, page, dtype, cache)
    if len(lens) == 4:
        b.table[0, 0] = -1
        b.table[2, 3] = b.P
    k, v, ks, vs = pools(b)
    tokens = b.T + 2                                         # two rows of no sequence
    out = tuple(torch.full((tokens, kv, dim), 5.0, dtype=dtype, device="cuda") for _ in range(2))
    args = (k, v, put(b.table), put(b.lens_t()), put(b.starts))
    got = gm.keops_cache_read(*args, tokens, dtype=dtype, k_scale=ks, v_scale=vs, out=out)
    assert got[0] is out[0] and got[1] is out[1]
    plain = gm.keops_cache_read(*args, b.T, dtype=dtype, k_scale=ks, v_scale=vs)
    both = torch.zeros((b.T, 2, kv, dim), dtype=dtype, device="cuda")     # keys and values in alternate rows
    gm.keops_cache_read(*args, b.T, dtype=dtype, k_scale=ks, v_scale=vs, out=(both[:, 0], both[:, 1]))
    for name, x, y, z, pool, scale in (("k", out[0], plain[0], both[:, 0], b.k, b.k_scale), ("v", out[1], plain[1], both[:, 1], b.v, b.v_scale)):
        x = x.cpu()
        assert torch.equal(x[:b.T], y.cpu()) and torch.equal(y, z) and bool((x[b.T:] == 5).all()), name
        for t, s, j, pg, row in sref.places(b):
            if pg < 0:
                want = torch.zeros((kv, dim))
            elif cache == E2:
                want = sref.from_4bit(pool[pg, row], scale[pg, :, row])
            else:
                want = pool[pg, row].float() * (1.0 if scale is None else scale[:, None])
            assert torch.equal(x[t], want.to(dtype)), (name, t)


# ---- logits

def logit_case(seed, S, new, V, width, dtype, biases, mask=True, penalties=True):
    g = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)
    lens, rows = [], [0]
    for s in range(S):
        lens.append(rng.choice([width, rng.randint(0, width)]))
        rows.append(rows[-1] + rng.randint(0 if s else 1, new))
    T = rows[-1] + 1                                         # and one row of no sequence
    z = (torch.randn((T, V), generator=g) * 3).to(dtype)
    c = dict(starts=torch.tensor(rows, dtype=torch.int32))
    if penalties:
        text = (V * torch.rand((S, width), generator=g) ** 4).to(torch.int32)
        text[torch.rand((S, width), generator=g) < 0.05] = -1
        text[torch.rand((S, width), generator=g) < 0.02] = V + 3
        c.update(text=text, lens=torch.tensor(lens, dtype=torch.int32), prompt=torch.tensor([n // 3 for n in lens], dtype=torch.int32),
                 rep=0.5 + torch.rand(S, generator=g), pres=torch.rand(S, generator=g) - 0.3, freq=torch.rand(S, generator=g))
    if biases:
        ids = torch.randint(-2, V + 2, (S, biases), generator=g).to(torch.int32)
        if biases > 2:
            ids[:, biases // 2] = ids[:, 0]                  # twice the same: the last stands
        c.update(ids=ids, bias=torch.randn((S, biases), generator=g) * 4)
    if mask:
        m = torch.randint(-2 ** 31, 2 ** 31, (T, -(-V // 32)), generator=g).to(torch.int32)
        m[0] = 0                                             # nothing is left
        c.update(mask=m)
    return z, c


def run_logits(z, c, **kw):
    names = dict(text="tokens", prompt="prompt_lens", rep="repetition", pres="presence", freq="frequency", ids="bias_tokens")
    args = {names.get(k, k): put(v) for k, v in c.items() if k != "starts"}
    return gm.keops_adjust_logits(z, put(c["starts"]), **args, **kw)


def check_logits(got, z, c, fill):
    want = sref.logits(z, **c)
    none = want.isnan() & ~z.isnan()
    got = got.cpu()
    assert bool((got[none] == fill).all()), "rows of no sequence"
    half = torch.finfo(z.dtype).eps / 2
    floor = {FP: 2.0 ** -25, BF: 2.0 ** -134, F32: 2.0 ** -150}[z.dtype]
    want = torch.where(none, got.double(), want)
    # rounded once from 64 bits (by way of 32 where the type has 16)
    close(got, want, want.abs() * half * (1 + 2.0 ** -7) + floor, "logits")
    same = (want == z.double()) & ~none
    assert torch.equal(got[same], z[same])


@pytest.mark.parametrize("S,new,V,width,biases", [(1, 1, 1, 1, 1), (1, 1, 32, 5, 0), (1, 1, 33, 40, 3), (3, 4, 1000, 60, 7),
                                                  (5, 2, 4099, 300, 40), (2, 3, 9001, 2500, 300), (70, 1, 257, 20, 2),
                                                  (1, 2, 900, 30, 700), (2, 2, 3500, 9000, 600)])
@pytest.mark.parametrize("dtype", [BF, FP, F32])
def test_logits(S, new, V, width, biases, dtype):
    say(f"logits {S} x {new} x {V}, text {width}, {biases} biases, {dtype}")
    z, c = logit_case(S * 100 + V, S, new, V, width, dtype, biases)
    out = torch.full_like(z, 9.0).cuda()
    assert run_logits(put(z), c, out=out) is out
    check_logits(out, z, c, 9.0)
    # in place, in rows wider than the vocabulary, from a place that 16 bytes do not divide
    wide = torch.full((z.shape[0], V + 5), 3.0, dtype=dtype).cuda()
    view = wide[:, 1:V + 1]
    view.copy_(put(z))
    view[z.shape[0] - 1] = 9.0
    zz = z.clone()
    zz[-1] = 9.0
    assert run_logits(view, c, out=view) is view
    check_logits(view, zz, c, 9.0)
    assert bool((wide[:, 0] == 3).all()) and bool((wide[:, V + 1:] == 3).all())


@pytest.mark.parametrize("rules", ["text", "bias", "mask", "none", "repetition", "presence", "no prompt"])
def test_logits_rules_apart(rules):
    say(f"logits, {rules}")
    z, c = logit_case(5, 3, 3, 777, 90, F32, 11 if rules == "bias" else 0, rules == "mask", rules not in ("bias", "mask", "none"))
    for name in {"repetition": ("pres", "freq", "prompt"), "presence": ("rep", "freq"), "no prompt": ("prompt",)}.get(rules, ()):
        del c[name]
    out = torch.full_like(z, 9.0).cuda()
    run_logits(put(z), c, out=out)
    check_logits(out, z, c, 9.0)
    assert run_logits(put(z), c).shape == z.shape


def test_logits_non_finite():
    """Infinities and NaN pass through the rules; a masked one is -inf whatever it was."""
    say("logits, non-finite")
    V = 64
    z = torch.zeros((1, V))
    z[0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 1e38])
    z[0, 32:36] = z[0, :4]
    mask = torch.tensor([[-1, 0]], dtype=torch.int32)
    text = torch.tensor([[0, 1, 2, 3, 3, 5, -1]], dtype=torch.int32)
    c = dict(starts=torch.tensor([0, 1], dtype=torch.int32), text=text, lens=torch.tensor([7], dtype=torch.int32), rep=torch.tensor([0.001]),
             freq=torch.tensor([1.0]), mask=mask)
    got = run_logits(put(z), c).cpu()
    assert got[0, 0] == float("inf") and got[0, 1] == -float("inf") and bool(got[0, 2].isnan()) and got[0, 3] == float("inf")
    assert bool((got[0, 32:] == -float("inf")).all()) and got[0, 5] == -1.0 and bool((got[0, 6:32] == 0).all())
    c["rep"] = torch.tensor([0.0])
    got = run_logits(put(z), c).cpu()
    assert got[0, 0] == float("inf") and got[0, 3] == float("inf") and bool(got[0, 1].isnan()) and got[0, 5] == -1.0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_logits_infinite_repetition(dtype):
    """Divided by an infinity, a positive logit is 0, a negative one goes to -inf, and 0 times it is none."""
    say(f"logits, infinite repetition, {dtype}")
    z = torch.tensor([[2.0, -2.0, 0.0, 1e-38, 5.0]]).to(dtype)
    text = torch.tensor([[0, 1, 2, 3]], dtype=torch.int32)
    c = dict(starts=torch.tensor([0, 1], dtype=torch.int32), text=text, lens=torch.tensor([4], dtype=torch.int32),
             rep=torch.tensor([float("inf")]))
    got = run_logits(put(z), c).cpu()
    assert got[0, 0] == 0 and got[0, 1] == -float("inf") and bool(got[0, 2].isnan()) and got[0, 3] == 0 and got[0, 4] == 5


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("rule", ["frequency", "presence", "repetition", "bias"])
def test_logits_are_rounded_once(dtype, rule):
    """Results just beside a tie of the 16-bit type, nearer to it than 32 bits can tell: to the nearer neighbour."""
    say(f"logits next to ties, {dtype}, {rule}")
    V, base = 64, 256.0 if dtype == BF else 2048.0           # base: numbers are 2 apart from there on
    steps = torch.arange(32, dtype=torch.float64) * 2
    for side in (1, -1):
        add = torch.tensor(1.0 + side * 2.0 ** -20)
        z = torch.zeros((1, V), dtype=dtype)
        z[0, :32] = (base + steps).to(dtype)
        want = base + steps + (2 if side > 0 else 0)
        c = dict(starts=torch.tensor([0, 1], dtype=torch.int32))
        text = torch.arange(32, dtype=torch.int32)[None]
        if rule == "bias":
            c.update(ids=text, bias=add.expand(1, 32).contiguous())
        elif rule == "repetition":
            # 2 / r is above or below a tie of the type, 1 + half a step: r the next 32-bit number to 2 / that
            half = torch.finfo(dtype).eps / 2
            r = torch.tensor(2.0 / (1 + half), dtype=torch.float64).float()
            while (2.0 / r.double() > 1 + half) != (side > 0):
                r = torch.nextafter(r, torch.tensor(0.0 if side > 0 else 9.0))
            z[0, :32] = 2.0
            want = torch.full((32,), 1 + 2 * half if side > 0 else 1.0, dtype=torch.float64)
            c.update(text=text, lens=torch.tensor([32], dtype=torch.int32), rep=r[None])
        else:
            c.update(text=text, lens=torch.tensor([32], dtype=torch.int32), **{"pres" if rule == "presence" else "freq": -add[None]})
        step = 2 * half if rule == "repetition" else 2.0
        assert bool(((sref.logits(z, **c)[0, :32] - want).abs() < step / 2).all())         # the nearest number of the type
        for rows in (1, 300):                                # a work-group's piece is of either size
            if rows > 1:
                c["starts"] = torch.tensor([0, rows], dtype=torch.int32)
                if "lens" in c:
                    c["lens"] = torch.tensor([31 + rows], dtype=torch.int32)
            got = run_logits(put(z.expand(rows, V).contiguous()), c).cpu()
            assert torch.equal(got[0, :32].double(), want), (side, rows, got[0, :32], want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,biases", [(1, 256), (1, 257), (2, 5000), (300, 700), (1, 40000)])
def test_logits_long_lists(dtype, rows, biases):
    """Lists past what a work-group holds, tokens in them many times over: the last bias stands."""
    say(f"logits, {rows} rows, {biases} biases, {dtype}")
    V, g = 9001, torch.Generator().manual_seed(biases)
    z = torch.randn((rows, V), generator=g).to(dtype)
    ids = torch.randint(-5, V + 5, (1, biases), generator=g).to(torch.int32)
    ids[0, biases // 2:] = ids[0, biases // 2:] // 40 * 40   # a few tokens, many times
    c = dict(starts=torch.tensor([0, rows], dtype=torch.int32), ids=ids, bias=torch.randn((1, biases), generator=g) * 4,
             text=torch.arange(0, V, 7, dtype=torch.int32)[None], lens=torch.tensor([V], dtype=torch.int32), freq=torch.tensor([0.7]))
    got = run_logits(put(z), c)
    few = sorted({0, rows // 2, rows - 1})                   # rows differ in their logits alone: the text is past its width
    check_logits(got[few].cpu(), z[few], dict(c, starts=torch.tensor([0, len(few)], dtype=torch.int32)), 0.0)


def test_logits_long_lists_take_their_length():
    """40 times the list takes no more than 100 times as long (it took 1,000 times)."""
    say("logits, time of long lists")
    V, g, took = 32000, torch.Generator().manual_seed(1), []
    z, starts = torch.randn((1, V), generator=g).cuda(), torch.tensor([0, 1], dtype=torch.int32).cuda()
    for n in (250, 10000):
        ids, bias = torch.randperm(V, generator=g)[None, :n].to(torch.int32).cuda(), torch.randn((1, n), generator=g).cuda()
        out = gm.keops_adjust_logits(z, starts, bias_tokens=ids, bias=bias)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(5):
            gm.keops_adjust_logits(z, starts, bias_tokens=ids, bias=bias, out=out)
        b.record()
        torch.cuda.synchronize()
        took.append(a.elapsed_time(b))
        want = z.clone()
        want[0, ids[0].long()] = (z[0, ids[0].long()].double() + bias[0].double()).float()
        assert torch.equal(out, want)
    assert took[1] < 100 * took[0], took


def test_logits_follow_drafted_tokens():
    """Each of a sequence's rows has seen one token more; starts past the rows are cut, lens past the text too."""
    say("logits of drafted tokens")
    V, text = 40, torch.tensor([[3, 7, 7, 9, 11, 3]], dtype=torch.int32)
    z = torch.ones((4, V))
    for starts, lens in (([0, 4], [6]), ([0, 9], [6]), ([0, 4], [9]), ([0, 4], [2]), ([-3, 4], [6])):
        c = dict(starts=torch.tensor(starts, dtype=torch.int32), text=text, lens=torch.tensor(lens, dtype=torch.int32),
                 freq=torch.tensor([1.0]), rep=torch.tensor([2.0]))
        check_logits(run_logits(put(z), c), z, c, 0.0)


def test_logits_streams_and_graph():
    say("logits on streams and in a graph")
    z, c = logit_case(8, 6, 4, 5000, 700, BF, 30)
    c["starts"][-1] = z.shape[0]
    dev = put(z)
    want = run_logits(dev, c)
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    assert torch.equal(run_logits(dev, c, stream=st), want)
    held = {k: put(v) for k, v in c.items()}
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        got = run_logits(dev, held)
    for rep in range(3):
        dev.copy_(torch.randn(z.shape, generator=torch.Generator().manual_seed(rep)).to(BF))
        graph.replay()
        eager = run_logits(dev, held)
        torch.cuda.synchronize()
        assert torch.equal(got, eager)


def test_rows_far_apart():
    """Rows past 2^31 elements come out as the same rows by themselves."""
    say("rotary, 2.2e9 elements")
    T, H, D = 270000, 64, 128
    g = torch.Generator(device="cuda").manual_seed(9)
    freqs, at = gm.keops_rotary_frequencies(D, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda")
    x = torch.zeros((T, H, D), dtype=BF, device="cuda")
    for end in (slice(0, 70), slice(T // 2, T // 2 + 70), slice(T - 70, T)):
        x[end] = torch.randn((70, H, D), generator=g, device="cuda").to(BF)
    y = gm.keops_rotary(x, at, freqs)
    for end in (slice(0, 70), slice(T // 2, T // 2 + 70), slice(T - 70, T)):
        assert torch.equal(y[end], gm.keops_rotary(x[end].clone(), at[end].clone(), freqs))
    del x, y
    say("logits, 2.6e9 entries")
    T, V = 20000, 131072
    z = torch.zeros((T, V), dtype=BF, device="cuda")
    text = torch.tensor([[V - 1, 5, 5, 70000]], dtype=torch.int32, device="cuda").repeat(2, 1)
    rules = dict(tokens=text, lens=torch.tensor([4, 4], dtype=torch.int32, device="cuda"), frequency=torch.ones(2, device="cuda"))
    last = torch.randn((2, V), generator=g, device="cuda").to(BF)
    z[T - 2:] = last
    gm.keops_adjust_logits(z, torch.tensor([0, T - 2, T], dtype=torch.int32, device="cuda"), out=z, **rules)
    want = gm.keops_adjust_logits(last, torch.tensor([0, 0, 2], dtype=torch.int32, device="cuda"), **rules)
    assert torch.equal(z[T - 2:], want) and not torch.equal(want, last) and not bool(z[:T - 8].any())


# ---- together

@pytest.mark.parametrize("cache", [BF, E4, E2])
def test_a_step(cache):
    """The rotating append, attention, the adjustment of logits and verification as a serving step runs them, eager and as
    a graph that is replayed with other contents."""
    say(f"a serving step over {cache}")
    S, m, H, kv, D, V = 3, 3, 4, 2, 64, 300
    lens = [40, 9, 130]
    b, wide = append_batch(lens, [m] * S, H, kv, D, 16, BF, cache, seed=51)
    k, v, ks, vs = pools(b)
    table, n, starts = put(b.table), put(b.lens_t()), put(b.starts)
    freqs = gm.keops_rotary_frequencies(D).cuda()
    g = torch.Generator().manual_seed(4)
    head = torch.randn((H * D, V), generator=g).cuda() / 8
    text = torch.randint(0, V, (S, 130), generator=g).to(torch.int32).cuda()
    rules = dict(tokens=text, lens=n, repetition=torch.full((S,), 1.2).cuda(), presence=torch.full((S,), 0.3).cuda(),
                 mask=torch.randint(-2 ** 31, 2 ** 31, (S * m, -(-V // 32)), generator=g).to(torch.int32).cuda())
    drafts = torch.randint(0, V, (S, m - 1), generator=g).to(torch.int32).cuda()
    counts, ua, us = torch.full((S,), m - 1, dtype=torch.int32).cuda(), torch.rand((S, m - 1), generator=g).cuda(), torch.rand(S, generator=g).cuda()
    dev = put(wide)

    def step():
        q = gm.keops_cache_append_rotary(dev[:, :H], dev[:, H:H + kv], dev[:, H + kv:], k, v, table, n, starts, freqs, k_scale=ks, v_scale=vs)
        out, lse = gm.keops_paged_attention(q, k, v, table, n, starts, m, 130, k_scale=ks, v_scale=vs)
        z = gm.keops_adjust_logits(out.float().flatten(1) @ head, starts, **rules)
        p = torch.softmax(z, -1)
        return (q, out, lse, z, *gm.keops_verify_draft(p.view(S, m, V), None, drafts, counts, ua, us))
    eager = step()
    torch.cuda.synchronize()
    # the parts against their plain forms, each from the part before it
    at = torch.cat([torch.arange(x - m, x) for x in lens])
    wq = sref.rotate(wide[:, :H], at, freqs.cpu())
    close(eager[0].cpu(), wq, sref.rotate_bound(wide[:, :H], wq, freqs.cpu(), BF), "queries")
    b.q, b.k, b.v = eager[0].cpu(), raw(k) if cache == E2 else k.cpu(), raw(v) if cache == E2 else v.cpu()
    if cache == E2:
        b.k_scale, b.v_scale = raw(ks), raw(vs)
    o, lse, _, ot, zt, _ = ref.attention(b)
    close(eager[1].cpu(), o, ot, "out")
    close(eager[2].cpu(), lse, zt, "lse")
    z = (eager[1].float().flatten(1) @ head).cpu()
    wz = sref.logits(z, starts.cpu(), text.cpu(), lens, None, rules["repetition"].cpu(), rules["presence"].cpu(), None, None, None,
                     rules["mask"].cpu())
    close(eager[3].cpu(), wz, wz.abs() * ref.U32 * 1.01, "logits")
    p = torch.softmax(eager[3], -1).view(S, m, V)
    tokens, accepted = ref.verify(p.cpu(), None, drafts.cpu(), counts.cpu(), ua.cpu(), us.cpu())
    assert torch.equal(eager[4].cpu(), tokens) and torch.equal(eager[5].cpu(), accepted)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for rep in range(3):
        dev.copy_(torch.randn(wide.shape, generator=torch.Generator().manual_seed(rep)).to(BF))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        for x, y in zip(kept, step()):
            assert torch.equal(x, y)


def test_example_decodes_over_4_bits():
    """The example's other way runs, repeats itself, and its rules hold; what attention gave is the formula's over the values
    that the cache holds."""
    import importlib.util
    import os
    say("example, 4 bits and rules")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_decode.py")
    spec = importlib.util.spec_from_file_location("paged_decode", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    rounds = [0]

    def watch(st):
        rounds[0] += 1
        if rounds[0] % 5:
            return
        m, p, n = st["model"], st["pages"], st["lens"].tolist()
        whole = torch.tensor([0] + n, dtype=torch.int32).cumsum(0).int().cuda()
        k, v = (t.double().cpu() for t in gm.keops_cache_read(p.k, p.v, st["table"], st["lens"], whole, sum(n), **p.scales))
        for s in range(len(n)):
            a, e, at = int(st["starts"][s]), int(st["starts"][s + 1]), int(whole[s])
            q = st["q"][a:e].double().cpu()
            for h in range(m.heads):
                g = h // (m.heads // m.kv)
                z = q[:, h] @ k[at:at + n[s], g].T / m.dim ** 0.5
                z.masked_fill_(torch.arange(n[s]) > torch.arange(n[s] - (e - a), n[s])[:, None], -float("inf"))
                o = torch.softmax(z, -1) @ v[at:at + n[s], g]
                assert (st["out"][a:e, h].double().cpu() - o).abs().max() <= 2 ** -7 * v.abs().max()
    text = ex.decode(rounds=40, watch=watch, four_bit=True, rules=True)
    assert rounds[0] == 40 and all(40 <= len(t) <= 160 for t in text)
    # what was taken or drawn has mass under the rules
    assert all(x < 199 // 2 for t in text for x in t)
    assert ex.decode(rounds=10, four_bit=True, rules=True) == [t[:len(u)] for t, u in zip(text, ex.decode(rounds=10, four_bit=True, rules=True))]
