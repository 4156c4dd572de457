"""The bf16 paged cache on the GPU against the oracle: rotations and attention within
derived bounds, everything else bit for bit."""
import numpy as np
import pytest
import torch

from eviction_window_qk_amd import kvc, synth
from oracle import paged as og
import paged_utils as u
from q8_utils import dev_bf16, random_rows, rng_of

pytestmark = pytest.mark.gpu


def freq_of(r, base=10000.0):
    return base ** (-2.0 * np.arange(r // 2) / r)


# (n, heads, d, r, interleaved, backward, farthest position, mscale)
ROPE = [
    (1, 1, 64, 64, False, False, 1, 1.0),
    (5, 3, 128, 128, False, False, 131072, 1.0),
    (5, 3, 128, 128, True, False, 131072, 1.2),
    (7, 2, 64, 24, True, True, 4096, 1.0),
    (7, 2, 64, 24, False, True, 4096, 0.7),
    (3, 5, 128, 2, False, False, 100, 1.0),
    (3, 5, 128, 2, True, False, 100, 1.0),
    (4, 9, 64, 62, False, False, 2 ** 30, 1.0),
    (4, 9, 128, 126, True, False, 2 ** 31 - 1, 1.0),
    (33, 17, 128, 34, False, False, 70000, 1.0),
    (2, 40, 128, 96, False, False, 9, 0.0),
    (2, 300, 64, 64, False, False, 9, -1.0),
]


@pytest.mark.parametrize("case", ROPE, ids=[str(i) for i in range(len(ROPE))])
def test_rope(case):
    n, H, d, r, inter, back, far, m = case
    print(f"[case] rope {case}", flush=True)
    rng = rng_of(1, n, H, r)
    at = rng.integers(-far, far + 1, n).astype(np.int32)
    x = random_rows(2, n, H, d)
    plan = kvc.Rope(u.dev(freq_of(r)), interleaved=inter, mscale=m)
    ref, size = og.rope(og.widen(x), at, freq_of(r), m, inter, back)
    gx = dev_bf16(x)
    y = kvc.rope(plan, gx, u.dev(at), backward=back)
    u.check_rope(u.bits(y), ref, size, m)
    np.testing.assert_array_equal(u.bits(gx), x)
    # in place, out of a wider tensor, into a tensor of heads before tokens
    wide = dev_bf16(random_rows(3, n, H + 4, d + 8))
    view = wide[:, 2: 2 + H, :d]
    view.copy_(gx)
    rest = wide.clone()
    kvc.rope(plan, view, u.dev(at), y=view, backward=back)
    assert torch.equal(view.contiguous().view(torch.int16), y.view(torch.int16))
    wide[:, 2: 2 + H, :d] = rest[:, 2: 2 + H, :d]
    assert torch.equal(wide.view(torch.int16), rest.view(torch.int16))
    by_head = torch.zeros((H, n, d), dtype=torch.bfloat16, device="cuda")
    kvc.rope(plan, gx, u.dev(at), y=by_head.transpose(0, 1), backward=back)
    assert torch.equal(by_head.transpose(0, 1).contiguous().view(torch.int16), y.view(torch.int16))


def test_rope_is_its_own_gradient():
    """<rotate(x), g> = <x, backward(g)>, and differences of it: the map is linear, so they are exact
    up to the roundings of either side."""
    n, H, d, r = 6, 2, 64, 40
    plan = kvc.Rope(u.dev(freq_of(r)), mscale=1.3)
    at = torch.arange(n, dtype=torch.int32, device="cuda") * 1000
    x, g = dev_bf16(random_rows(4, n, H, d)), dev_bf16(random_rows(5, n, H, d))
    a = (kvc.rope(plan, x, at).double() * g.double()).sum()
    b = (x.double() * kvc.rope(plan, g, at, backward=True).double()).sum()
    # every value of either side is rounded to bf16 once
    room = 2.0 ** -8 * 1.3 * 2 * float((x.double().abs().sum() * g.double().abs().max()))
    assert abs(float(a - b)) <= room
    step = torch.zeros_like(x)
    step[2, 1, 3] = 1.0
    diff = (kvc.rope(plan, step, at).double() * g.double()).sum()
    assert abs(float(diff - kvc.rope(plan, g, at, backward=True)[2, 1, 3].double())) <= 2.0 ** -8 * 4 * float(g[2, 1].double().abs().max())


def test_rope_copies_what_it_does_not_rotate():
    """NaN and infinities behind the rotated part pass as they are."""
    x = random_rows(6, 3, 2, 64)
    x[:, :, 10:] = np.uint16(0x7F80)
    x[:, :, 11] = np.uint16(0x7FC1)
    for inter in (False, True):
        y = kvc.rope(kvc.Rope(u.dev(freq_of(10)), interleaved=inter), dev_bf16(x), torch.arange(3, dtype=torch.int32, device="cuda"))
        np.testing.assert_array_equal(u.bits(y)[:, :, 10:], x[:, :, 10:])


# (B, H, G, d, bs, lens, new, r, interleaved, holes, weights, pad)
APPEND = [
    (1, 1, 1, 64, 16, [1], [1], 64, False, 0.0, False, 0),
    (3, 2, 4, 128, 16, [5, 0, 33], [5, 0, 2], 128, False, 0.0, True, 3),
    (4, 3, 2, 64, 5, [7, 12, 3, 1], [1, 12, 0, 1], 22, True, 0.3, True, 0),
    (2, 2, 7, 128, 24, [100, 49], [70, 49], 32, False, 0.3, False, 1),
    (70, 1, 1, 64, 1, list(range(1, 71)), [1] * 70, 64, False, 0.0, True, 0),
    (2, 1, 64, 64, 4096, [5000, 4097], [2, 3], 64, True, 0.0, False, 0),
    (5, 2, 1, 128, 100, [3, 0, 9, 0, 0], [5, 2, 1, 0, 0], 100, False, 0.0, True, 0),     # more new than there are slots
]


@pytest.mark.parametrize("case", APPEND, ids=[str(i) for i in range(len(APPEND))])
@pytest.mark.parametrize("given", [False, True], ids=["slots", "positions"])
def test_append(case, given):
    B, H, G, d, bs, lens, new, r, inter, holes, weights, pad = case
    print(f"[case] append {case} {given}", flush=True)
    c = u.random_cache(10, B, H, d, bs, lens, holes=holes, weights=weights)
    starts = u.starts_of(new)
    n = int(starts[-1]) + pad
    at = rng_of(11, n).integers(0, 100000, n).astype(np.int32)
    qkv = random_rows(12, n, (G + 2) * H, d)
    dq = dev_bf16(qkv)
    q, k, v = dq[:, : G * H], dq[:, G * H: (G + 1) * H], dq[:, (G + 1) * H:]
    plan = kvc.Rope(u.dev(freq_of(r)), interleaved=inter, mscale=1.1)
    g = u.to_gpu(c)
    pos = u.dev(at) if given else None
    q_out = torch.full((n, G * H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    kvc.paged_append(g, k, v, u.dev(starts), positions=pos, rope=plan, q=q, q_out=q_out)
    np.testing.assert_array_equal(u.bits(dq), qkv)
    mine = {t: (b, slot) for t, b, slot in og.slots(c, starts, n)}
    where = np.array([at[t] if given else mine.get(t, (0, 0))[1] for t in range(n)])
    # q and k against fp64, then the pages bit for bit with what the kernel rotated
    ref, size = og.rope(og.widen(qkv), where, freq_of(r), 1.1, inter)
    got_q = u.bits(q_out)
    rows = sorted(mine)
    u.check_rope(got_q[rows], ref[rows, : G * H], size[rows, : G * H], 1.1)
    assert (got_q[[t for t in range(n) if t not in mine]] == 0x40E0).all()
    k_bits = np.zeros((n, H, d), np.uint16)
    gk = u.bits(g.k_pool)
    for t, (b, slot) in mine.items():
        place = c.at(b, slot) if slot >= 0 else None
        if place:
            k_bits[t] = gk[place[0], :, place[1]]
            u.check_rope(k_bits[t][None], ref[t: t + 1, G * H: (G + 1) * H], size[t: t + 1, G * H: (G + 1) * H], 1.1)
    og.append(c, k_bits, qkv[:, (G + 1) * H:], starts, at if given else None)
    u.same_cache(g, c)
    # without a rotation: rows as they are; q rotated in place, in the same tensor as k and v
    g2 = u.to_gpu(c)
    kvc.paged_append(g2, v, k, u.dev(starts), positions=pos)
    og.append(c, qkv[:, (G + 1) * H:], qkv[:, G * H: (G + 1) * H], starts, at if given else None)
    u.same_cache(g2, c)
    kvc.paged_append(g2, k, v, u.dev(starts), positions=pos, rope=plan, q=q, q_out=q)
    np.testing.assert_array_equal(u.bits(dq)[rows, : G * H], got_q[rows])
    np.testing.assert_array_equal(u.bits(dq)[:, G * H:], qkv[:, G * H:])
    u.same_cache(g2, _again(c, k_bits, qkv[:, (G + 1) * H:], starts, at if given else None))


def _again(c, k, v, starts, at):
    og.append(c, k, v, starts, at)
    return c


# (B, H, G, d, bs, lens, new, holes, pad)
ATTEND = [
    (1, 1, 1, 64, 16, [1], [1], 0.0, 0),
    (1, 1, 1, 128, 16, [700], [1], 0.0, 0),
    (3, 2, 4, 128, 16, [0, 1, 37], [0, 1, 1], 0.0, 2),
    (3, 2, 4, 64, 16, [0, 3, 37], [2, 5, 1], 0.0, 0),                 # an empty sequence with tokens, more tokens than slots
    (5, 1, 7, 128, 16, [1100, 512, 513, 127, 31], [1, 1, 1, 1, 1], 0.0, 0),
    (4, 2, 3, 64, 24, [200, 97, 1500, 24], [5, 1, 3, 24], 0.25, 3),
    (4, 1, 2, 128, 5, [200, 97, 700, 24], [16, 9, 8, 17], 0.25, 0),
    (2, 1, 16, 128, 1, [65, 130], [1, 2], 0.0, 0),
    (2, 1, 33, 64, 64, [65, 600], [1, 1], 0.0, 0),
    (1, 1, 64, 128, 100, [300], [2], 0.0, 0),
    (1, 2, 4, 128, 16, [300], [300], 0.0, 0),
    (1, 2, 4, 64, 16, [300], [300], 0.0, 1),
    (3, 1, 4, 128, 64, [1000, 129, 640], [100, 129, 1], 0.0, 5),
    (3, 1, 4, 64, 24, [1000, 129, 640], [100, 129, 1], 0.3, 5),
    (2, 1, 1, 128, 4096, [4100, 90], [70, 33], 0.0, 0),
    (3, 1, 2, 128, 7, [400, 65, 64], [65, 64, 63], 0.3, 0),
    (1, 1, 1, 64, 16, [2200], [129], 0.0, 0),
]


@pytest.mark.parametrize("weights", [False, True], ids=["plain", "weights"])
@pytest.mark.parametrize("case", ATTEND, ids=[str(i) for i in range(len(ATTEND))])
def test_attend(case, weights):
    B, H, G, d, bs, lens, new, holes, pad = case
    print(f"[case] attend {case} {weights}", flush=True)
    c = u.random_cache(20, B, H, d, bs, lens, holes=holes, weights=weights)
    starts = u.starts_of(new)
    n = int(starts[-1]) + pad
    q = random_rows(21, n, G * H, d)
    g = u.to_gpu(c)
    out = torch.full((n, G * H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, G * H), 3.0, device="cuda")
    kvc.paged_attend(g, dev_bf16(q), u.dev(starts), max_new=max(new), out=out, lse=lse)
    torch.cuda.synchronize()
    ref = og.attend(c, og.widen(q), starts)
    u.check_attention(ref, u.bits(out), lse, max(lens), untouched=0x40E0)
    assert (lse.cpu().numpy()[~ref["mine"]] == 3.0).all()
    if weights:
        u.check_weights(ref, c.weight, g.weight.cpu().numpy(), d, G * max(new))
        grown = g.weight.clone()
        c.weight[:] = grown.cpu().numpy()
    u.same_cache(g, c)
    # rows of a wider tensor, heads before tokens, without max_new and lse: the same bits
    if weights:
        g = u.to_gpu(c)
    wide = torch.zeros((n, G * H + 2, d + 8), dtype=torch.bfloat16, device="cuda")
    wide[:, 1: 1 + G * H, :d] = dev_bf16(q)
    by_head = torch.full((G * H, n, d), 7.0, dtype=torch.bfloat16, device="cuda")
    kvc.paged_attend(g, wide[:, 1: 1 + G * H, :d], u.dev(starts), out=by_head.transpose(0, 1))
    assert torch.equal(by_head.transpose(0, 1).contiguous().view(torch.int16), out.view(torch.int16))
    if weights:
        a, b = (g.weight - grown).cpu().numpy(), ref["add"]
        np.testing.assert_allclose(a, b, rtol=0, atol=2.0 ** -8 * max(1.0, float(b.max())))


@pytest.mark.parametrize("weights", [False, True], ids=["plain", "weights"])
@pytest.mark.parametrize("d", [64, 128])
def test_starts_outside_the_tokens_are_taken_as_clamped(d, weights):
    """Sequences of few and of many rows, in pieces, over starts below 0 and past n."""
    lens, n = [1300, 900, 700], 240
    c = u.random_cache(22, 3, 2, d, 16, lens, weights=weights)
    q = dev_bf16(random_rows(23, n, 4, d))
    for bad, good in (([-300, 100, 110, 10 ** 9], [0, 100, 110, n]), ([-2 ** 31, -5, 200, 2 ** 31 - 1], [0, 0, 200, n])):
        got = []
        for starts in (good, bad):
            g = u.to_gpu(c)
            out = torch.full((n, 4, d), 7.0, dtype=torch.bfloat16, device="cuda")
            _, lse = kvc.paged_attend(g, q, u.dev(np.int32(starts)), out=out, want_lse=True)
            kvc.paged_append(g, q[:, :2], q[:, 2:], u.dev(np.int32(starts)))
            kvc.prompt_attend(q, q[:, :2], q[:, 2:], u.dev(np.int32(starts)), out=(by := torch.zeros_like(out)))
            torch.cuda.synchronize()
            got.append([u.bits(out), lse.cpu().numpy(), u.bits(g.k_pool), u.bits(by)] +
                       ([g.weight.cpu().numpy()] if weights else []))
        for a, b in zip(*got):
            np.testing.assert_array_equal(a, b)


def test_a_scale_and_scores_that_climb():
    """Scores rise by hundreds from key to key, and the reverse."""
    d, T = 64, 700
    c = u.random_cache(30, 1, 1, d, 16, [T])
    ramp = np.linspace(-400, 400, T)
    for turn in (1, -1):
        k = np.zeros((c.n * c.bs, d), np.float32)
        for t in range(T):
            p, r = c.at(0, t)
            k[p * c.bs + r, 0] = ramp[::turn][t]
        c.k = synth.f32_to_bf16_bits(k).reshape(c.k.shape)
        for n in (1, 200):
            q = random_rows(31, n, 2, d)
            q[..., 0] = synth.f32_to_bf16_bits(np.float32([1.0]))[0]
            ref = og.attend(c, og.widen(q), [0, n], scale=0.7)
            out, lse = kvc.paged_attend(u.to_gpu(c), dev_bf16(q), u.dev(u.starts_of([n])), scale=0.7, want_lse=True)
            u.check_attention(ref, u.bits(out), lse, T)


# (H, G, d, lens, pad)
PROMPT = [
    (1, 1, 64, [1], 0),
    (1, 1, 128, [1, 1, 2], 1),
    (1, 2, 64, [128], 0),
    (2, 4, 128, [0, 33, 1, 0, 200, 64], 3),
    (2, 4, 64, [65, 0, 130], 0),
    (1, 7, 128, [127, 150], 0),
    (3, 1, 128, [257, 5], 2),
    (9, 3, 64, [40, 90], 0),
    (1, 64, 128, [9, 31], 0),
    (8, 1, 64, [300], 0),
    (1, 1, 64, [700], 0),
]


@pytest.mark.parametrize("case", PROMPT, ids=[str(i) for i in range(len(PROMPT))])
def test_prompt(case):
    H, G, d, lens, pad = case
    print(f"[case] prompt {case}", flush=True)
    starts = u.starts_of(lens)
    n = int(starts[-1]) + pad
    qkv = random_rows(40, n, (G + 2) * H, d)
    qkv[n - pad:] = u.NAN                               # nobody's rows are not looked at
    dq = dev_bf16(qkv)
    q, k, v = dq[:, : G * H], dq[:, G * H: (G + 1) * H], dq[:, (G + 1) * H:]
    out = torch.full((n, G * H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    _, lse = kvc.prompt_attend(q, k, v, u.dev(starts), out=out, want_lse=True)
    w = og.widen(qkv)
    ref = og.prompt(w[:, : G * H], w[:, G * H: (G + 1) * H], w[:, (G + 1) * H:], starts)
    u.check_attention(ref, u.bits(out), lse, max(lens), untouched=0x40E0)
    by_head = torch.full((G * H, n, d), 7.0, dtype=torch.bfloat16, device="cuda")
    kvc.prompt_attend(q.transpose(0, 1).contiguous().transpose(0, 1), k, v.contiguous(), u.dev(starts), out=by_head.transpose(0, 1))
    assert torch.equal(by_head.transpose(0, 1).contiguous().view(torch.int16), out.view(torch.int16))


def test_prompt_and_chunk_agree():
    """A prompt, and the same tokens as one chunk over pages that hold them."""
    H, G, d, n = 2, 4, 128, 333
    qkv = random_rows(41, n, (G + 2) * H, d)
    dq = dev_bf16(qkv)
    starts = u.dev(u.starts_of([n]))
    a = kvc.prompt_attend(dq[:, : G * H], dq[:, G * H: (G + 1) * H], dq[:, (G + 1) * H:], starts)
    g = u.to_gpu(u.random_cache(42, 1, H, d, 16, [n]))
    kvc.paged_append(g, dq[:, G * H: (G + 1) * H], dq[:, (G + 1) * H:], starts)
    b = kvc.paged_attend(g, dq[:, : G * H], starts)
    # each is within 2^-8 of its weights and 2^-8 of itself of the same number
    assert float((a.double() - b.double()).abs().max()) <= 4 * 2.0 ** -8 * float(dq[:, (G + 1) * H:].double().abs().max())


# (B, H, d, bs, lens, budget, sinks, recent, kind)
EVICT = [
    (1, 1, 64, 16, [2], 1, 0, 0, "random"),
    (2, 2, 128, 16, [65, 64], 64, 4, 8, "random"),
    (3, 2, 64, 24, [100, 10, 0], 50, 4, 16, "ties"),
    (2, 3, 128, 5, [200, 77], 10, 4, 16, "zero"),          # sinks and recent fill the budget
    (2, 1, 64, 16, [300, 299], 7, 3, 0, "odd"),            # NaN, -0, infinities, negative
    (1, 2, 128, 64, [1500], 1024, 0, 1, "shuffled"),
    (2, 2, 64, 100, [1030, 2100], 1029, 4, 64, "shuffled"),
    (1, 1, 64, 16, [1000], 3, 10, 10, "random"),           # more sinks than budget
    (2, 1, 64, 16, [90, 80], 50, 0, 100, "random"),        # all are recent
    (1, 3, 64, 256, [5000], 2500, 4, 64, "spread"),
    (2, 1, 64, 64, [16384, 16380], 5000, 4, 64, "random"),
    (2, 1, 64, 256, [40000, 16385], 20000, 4, 64, "spread"),
    (1, 2, 64, 256, [33000], 32996, 4, 64, "random"),
    (1, 1, 64, 256, [33000], 9000, 0, 0, "ties"),
    (1, 2, 64, 64, [2049], 2040, 4, 8, "odd"),
]


def _evict_case(case, seed=50):
    B, H, d, bs, lens, K, sinks, recent, kind = case
    rng = rng_of(seed, B, H, K)
    c = u.random_cache(seed, B, H, d, bs, lens, weights=True)
    shape = c.weight.shape
    if kind == "ties":
        c.weight = rng.integers(0, 3, shape).astype(np.float32)
    elif kind == "zero":
        c.weight[:] = 0
    elif kind == "odd":
        c.weight = rng.choice(np.float32([np.nan, 0.0, -0.0, np.inf, -np.inf, 1.0, -1.0, 1e-45, 3e38]), shape).astype(np.float32)
    elif kind == "spread":
        c.weight = np.exp(rng.normal(0, 20, shape)).astype(np.float32)
    seen = np.array(lens, np.int32)
    if kind == "shuffled":
        for n in range(shape[0]):
            L = max(1, int(lens[n // H]))
            c.pos[n, :L] = rng.permutation(3 * L)[:L]
        seen = 3 * seen
    return c, seen, K, sinks, recent


@pytest.mark.parametrize("case", EVICT, ids=[str(i) for i in range(len(EVICT))])
def test_evict(case):
    print(f"[case] evict {case}", flush=True)
    c, seen, K, sinks, recent = _evict_case(case)
    g = u.to_gpu(c)
    for _ in range(2):                                     # the second finds nothing to do
        kvc.paged_evict(g, u.dev(seen), K, sinks=sinks, recent=recent)
        og.evict(c, seen, K, sinks, recent)
        u.same_cache(g, c)


def test_evict_with_positions_that_repeat_stays_in_bounds():
    """Against the precondition: the counts still fit, ties stay in the order of the slots."""
    for lens, K, sinks in (([300, 150], 100, 0), ([300, 150], 148, 0), ([300, 103], 100, 9), ([20000, 3000], 2500, 0)):
        c, seen, K, sinks, recent = _evict_case((2, 2, 64, 16, lens, K, sinks, 0, "zero"))
        c.pos[:] = 5
        g = u.to_gpu(c)
        kvc.paged_evict(g, u.dev(seen), K, sinks=sinks, recent=recent)
        og.evict(c, seen, K, sinks, recent)
        u.same_cache(g, c)


@pytest.mark.parametrize("seed", range(4))
def test_trim(seed):
    from oracle import pages as op
    from q8_utils import pages_to_gpu, random_pages, same_pages
    t = random_pages(seed, 9, 7, 8, 60)
    rng = rng_of(seed, 60)
    t.lens = np.where(rng.random(9) < 0.7, rng.integers(-3, 60, 9), t.lens).astype(np.int32)
    t.table[3, 5] = 10 ** 6                                 # names no page: left as it is
    g = pages_to_gpu(t)
    kvc.pages_trim(g)
    op.trim(t)
    torch.cuda.synchronize()
    same_pages(g, t)
