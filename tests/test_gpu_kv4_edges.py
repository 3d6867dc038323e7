"""GPU tests of the 4-bit KV cache where it is easy to get wrong: values far past what
a block can hold, lengths past the page table, weights of one token, workspaces of
other calls, empty batches, and rows whose elements span fp16's range.  Each test
derives its own tolerance."""
import math

import pytest
import torch

from tests import kv4_reference as ref
from tests.test_gpu_kv4 import Setup, _aq

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("g", [2.0 ** -100, 2.0 ** -40, 2.0 ** -12, 1.0, 2.0 ** 20, 3e-30])
@pytest.mark.parametrize("dtype,rotate", [(F32, False), (BF16, False), (F32, True)])
def test_append_far_past_the_largest_value(g, dtype, rotate):
    """Values up to fp32's range saturate with their sign whatever the head's scale: bit for bit the
    documented steps, in which x / (g s) is an infinity of x's sign."""
    for amplitude in (g * 1e2, g * 1e6, 1e12, 1e30, 3e37):
        # (a rotation adds up to 64 values of up to nine times the amplitude: 576 x 5e35 is still in fp32's range)
        if not 1e-37 < amplitude < (5e35 if rotate else 1e38):
            continue
        st = Setup([40], 1, 64, dtype=dtype, rotate=rotate, seed=7, amplitude=amplitude, g=(g, g))
        # one block of every row far below the rest, so that both kinds of block are there
        st.K[..., 16:32] *= 1e-30
        st.V[..., 32:48] *= 1e-30
        _aq().attnq_kv4_append(st.cache, st.seqs, st.K.cuda(), st.V.cuda())
        K, V = st.read()
        k, v = st.held(0, 0)
        assert torch.equal(K[0, 0], k.float()) and torch.equal(V[0, 0], v.float())
        most = 6 * 448 * g
        if amplitude > 1e6 * most and not rotate:
            assert (V[0, 0, :, :32].abs() == most).any() and (V[0, 0] == -most).any()


@pytest.mark.parametrize("d,over,T", [(64, 1, 1), (64, 3, 8), (128, 20, 40), (64, 60, 40), (128, 2 ** 31 - 1 - 96, 5)])
def test_append_past_the_page_table(d, over, T):
    """A length past the table's capacity is reported; rows keep their places, those past the last place
    are dropped, and no other token loses its bits."""
    aq = _aq()
    cap = 96
    st = Setup([cap, 50], 2, d, 16, seed=over % 97)
    st.table = st.table[:, :6].contiguous()  # exactly 96 places
    gen = torch.Generator().manual_seed(T)
    K, V = (torch.randn((2, 2, T, d), generator=gen).to(BF16) for _ in range(2))
    lens = torch.tensor([cap + over, 50], dtype=torch.int32).cuda()
    aq.attnq_kv4_append(st.cache, aq.AttnqKv4Seqs(st.table, lens), K.cuda(), V.cuda())
    assert aq.attnq_device_status() == 6
    whole = torch.tensor([cap, 50], dtype=torch.int32).cuda()
    got = [torch.empty((2, 2, cap, d), device="cuda") for _ in range(2)]
    aq.attnq_kv4_read(st.cache, aq.AttnqKv4Seqs(st.table, whole, whole), *got)
    assert aq.attnq_device_status() == 0
    for new, old, out in ((K, st.K, got[0]), (V, st.V, got[1])):
        for b, L in ((0, cap + over), (1, 50)):
            want = old[b, :, :min(L, cap)].clone()
            for t in range(T):
                place = L - T + t
                if 0 <= place < cap:
                    want[:, place] = new[b, :, t]
            assert torch.equal(out[b, :, :min(L, cap)].cpu(), ref.held(want).float())
    # reading follows the same places and leaves the dropped rows as they were
    back = [torch.full((2, 2, T, d), -77.0, device="cuda") for _ in range(2)]
    aq.attnq_kv4_read(st.cache, aq.AttnqKv4Seqs(st.table, lens), *back)
    assert aq.attnq_device_status() == 6
    there = max(0, min(T, T - over))
    assert torch.equal(back[0][0, :, :there].cpu(), ref.held(K[0, :, :there]).float())
    assert (back[0][0, :, there:] == -77).all() and (back[1][0, :, there:] == -77).all()
    assert torch.equal(back[1][1].cpu(), ref.held(V[1]).float())


@pytest.mark.parametrize("T,G,pages", [(1, 4, 4), (1, 8, 4), (1, 4, 300), (9, 4, 4), (40, 8, 4)])
def test_weights_of_an_empty_batch(T, G, pages):
    """Sequences without tokens only: the call's last kernel has nothing to do, and still what follows in the
    stream sees all rows written (O = 0, lse = -infinity) and no weight changed."""
    aq = _aq()
    B, Hkv, d, page = 600, 2, 128, 256
    cache = aq.alloc_kv4_cache(1, page, Hkv, d)
    table = torch.zeros((B, pages), dtype=torch.int32, device="cuda")
    seqs = aq.AttnqKv4Seqs(table, torch.zeros(B, dtype=torch.int32, device="cuda"))
    Q = torch.randn((B, Hkv * G, T, d), generator=torch.Generator().manual_seed(T)).to(BF16).cuda()
    ws = torch.empty(aq.attnq_kv4_attn_workspace(cache, B, pages, Hkv * G, T), dtype=torch.uint8, device="cuda")
    O = torch.empty_like(Q)
    lse = torch.empty(Q.shape[:3], device="cuda")
    acc = torch.full((B, Hkv, pages * page), -77.0, device="cuda")
    seen = []
    for _ in range(8):
        O.fill_(-77.0)
        lse.fill_(-77.0)
        aq.attnq_kv4_attn(cache, seqs, Q, O, True, ws, lse=lse, acc_out=acc)
        seen.append(((O != 0).any(), (lse != -math.inf).any()))
    assert aq.attnq_device_status() == 0
    assert not any(bool(a) or bool(b) for a, b in seen)
    assert (acc == -77).all()


@pytest.mark.parametrize("T,G,dtype", [(1, 4, BF16), (1, 8, F32), (5, 4, BF16), (40, 4, BF16), (40, 4, F32)])
def test_workspaces_of_other_calls(T, G, dtype):
    """The workspace of a larger call leaves the result's bits as they are (its scores are past 64 MiB, this
    call's fit).  Without the scores' part O and lse keep their bits, and the weights come from K again: both
    ways take fp32 sums of d products (d 2^-23 of sum |q k| scale log2 e, below 48 here), round them and the
    row's sum a few times (2^-20 of them), so a weight moves by 2 (d 2^-23 + 2^-20) 48 < 2^-8 of itself."""
    aq = _aq()
    st = Setup([900, 0, 2000, 33], 2, 128, 64, dtype=dtype, seed=T + G)
    gen = torch.Generator().manual_seed(T)
    Q = torch.randn((4, 2 * G, T, 128), generator=gen).to(dtype).cuda()
    start = torch.rand((4, 2, st.max_pages * 64), generator=gen).cuda()
    rows = T * G
    tail = min(64 << 20, 4 * 2 * st.max_pages * 64 * (16 if rows <= 4 else 32 * -(-rows // 8)))
    own = aq.attnq_kv4_attn_workspace(st.cache, 4, st.max_pages, 2 * G, T)
    sizes = [own, aq.attnq_kv4_attn_workspace(st.cache, 64, 9000, 2 * G, 2 * T), own - -(-tail // 256) * 256]
    assert sizes[1] > sizes[0] > sizes[2]
    out = []
    for size in sizes:
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        O, lse = torch.zeros_like(Q), torch.zeros(Q.shape[:3], device="cuda")
        acc = torch.full_like(start, -77.0)
        aq.attnq_kv4_attn(st.cache, aq.AttnqKv4Seqs(st.table, st.lens_t), Q, O, True, ws, lse=lse, acc_in=start,
                          acc_out=acc)
        assert aq.attnq_device_status() == 0
        out.append((O, lse, acc))
    for x, y in zip(out[0], out[1]):
        assert torch.equal(x, y)
    assert torch.equal(out[0][0], out[2][0]) and torch.equal(out[0][1], out[2][1])
    for b, L in enumerate(st.lens):
        a, c = (out[i][2][b, :, :L] - start[b, :, :L] for i in (0, 2))
        tol = 2.0 ** -8 * a.abs() + 2.0 ** -23 * (start[b, :, :L] + rows) * 2
        assert ((a - c).abs() <= tol).all()
        assert (out[2][2][b, :, L:] == -77).all()
    with pytest.raises(aq.AttnqError):
        aq.attnq_kv4_attn(st.cache, aq.AttnqKv4Seqs(st.table, st.lens_t), Q, O, True,
                          torch.empty(sizes[2] - 1, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("T,pages", [(1, 1), (5, 1), (16, 1), (16, 9000), (40, 1)])
@pytest.mark.parametrize("size", [3.0, 40.0, 700.0])
def test_weight_of_an_only_token(T, pages, size):
    """A sequence of one token gives it the weight 1, however large the score.

    In log2 units let y = s c be the score, m its fp32 value and u its last place.  The exponent
    fma(s, c, 15 - m) is exact to 2^-21 (for m > 16 15 - m is a multiple of u that fp32 holds), so
    m + (log2 l - 15), rounded to fp32, is within u / 2 + 2^-18 of y (2^-18: an fp32 near 15, ex2, log2).  The
    weight's exponent is y or m less that: at most u + 2^-18, times ln 2 < 0.7.  Both come from the same raw
    sum s, but for T = 40, where tcgen05 adds the d products in another order: d 2^-23 of
    sum |q k| (= y here, q lies along k) on either side."""
    aq = _aq()
    B, d = 320, 64
    st = Setup([1] * B, 1, d, 16, dtype=F32, seed=T)
    gen = torch.Generator().manual_seed(int(size) + T)
    k = torch.stack([st.held(b, 0)[0][0] for b in range(B)])
    want = size * (1 + torch.rand((B, 1), generator=gen).double())
    Q = torch.zeros((B, 1, T, d))
    Q[:, 0, 0] = (want / math.log2(math.e) / 0.125 / (k * k).sum(-1, keepdim=True) * k).float()
    y = (Q[:, 0, 0].double() * k).sum(-1) * 0.125 * math.log2(math.e)
    table = torch.full((B, max(pages, st.max_pages)), -1, dtype=torch.int32, device="cuda")
    table[:, :st.max_pages] = st.table
    one = torch.ones(B, dtype=torch.int32, device="cuda")  # row 0 alone exists, whatever T
    acc = torch.zeros((B, 1, table.shape[1] * 16), device="cuda")
    ws = torch.empty(aq.attnq_kv4_attn_workspace(st.cache, B, table.shape[1], 1, T), dtype=torch.uint8, device="cuda")
    O = torch.empty((B, 1, T, d), device="cuda", dtype=BF16 if T == 40 else F32)
    aq.attnq_kv4_attn(st.cache, aq.AttnqKv4Seqs(table, st.lens_t, one), Q.cuda(), O, True, ws, acc_out=acc)
    assert aq.attnq_device_status() == 0
    u = torch.exp2(torch.floor(torch.log2(y)) - 23)
    tol = 0.7 * (u + 2.0 ** -18 + (2 * d * 2.0 ** -23 * y if T == 40 else 0.0))
    off = (acc[:, 0, 0].cpu().double() - 1).abs()
    assert (off <= tol).all(), (off / tol).max()


def test_binding_refuses_what_32_bits_do_not_hold():
    """Numbers past 32 bits would reach the library cut off: 2^32 + 1 rows as one, 2^32 sinks as none."""
    aq = _aq()
    st = Setup([40], 1, 64, 16, seed=3, spare=10)
    w = 1 << 32
    one = torch.zeros((1, 1, 1, 64), dtype=BF16, device="cuda")
    many = one.expand(1, 1, w + 1, 64)
    before = st.cache.pages.clone()
    with pytest.raises(aq.AttnqError):
        aq.attnq_kv4_append(st.cache, aq.AttnqKv4Seqs(st.table, st.lens_t), many, many)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    with pytest.raises(aq.AttnqError):
        aq.attnq_kv4_attn(st.cache, aq.AttnqKv4Seqs(st.table, st.lens_t), many, many, True, ws)
    big = aq.AttnqKv4Cache(st.cache.num_pages + w, 16, 1, 64, 0, None, None, None, st.cache.pages)
    with pytest.raises(aq.AttnqError):
        aq.attnq_kv4_append(big, aq.AttnqKv4Seqs(st.table, st.lens_t), one, one)
    used = set(st.table.flatten().tolist())
    dst = torch.tensor([[p for p in range(st.cache.num_pages) if p not in used][0]], dtype=torch.int32, device="cuda")
    acc = torch.rand((1, 1, st.max_pages * 16), device="cuda")
    new = torch.full((1,), -5, dtype=torch.int32, device="cuda")
    kept = torch.full((1, 1, 16), -5, dtype=torch.int32, device="cuda")
    for sink, recent in ((w, 4), (4, w), (w + 2, 4), (4, w + 2)):
        with pytest.raises(aq.AttnqError):
            aq.attnq_kv4_evict(st.cache, aq.AttnqKv4Seqs(st.table, st.lens_t), acc, 16, sink, recent, dst, new, kept, None,
                               ws)
    assert aq.attnq_device_status() == 0
    assert new.item() == -5 and (kept == -5).all() and torch.equal(before, st.cache.pages)


@pytest.mark.parametrize("span", [10, 24, 30])
@pytest.mark.parametrize("T,G,d,out", [(1, 4, 128, BF16), (1, 4, 64, F32), (1, 8, 64, BF16), (9, 2, 128, F32),
                                       (300, 1, 128, BF16), (300, 1, 64, BF16)])
def test_bf16_queries_that_span_fp16(T, G, d, out, span):
    """Unrotated bf16 queries with one element 2^span above the others, in a channel where the keys are 0: the
    others decide the scores and keep their bits.

    A row enters the products as fp16 with its largest element in [2^14, 2^15), so a bf16 element (8 bits)
    is exact from 2^-31 of the largest on and off by at most 2^-39 of it below: 2^-39 qmax sum |k| scale of
    a score, beside d 2^-23 of sum |q k| for the sum's roundings."""
    aq = _aq()
    st = Setup([T + 60, T], 2, d, 32, seed=T + span)
    st.K[..., 7] = 0.0
    aq.attnq_kv4_append(st.cache, st.seqs, st.K.cuda(), st.V.cuda())
    gen = torch.Generator().manual_seed(span)
    Q = torch.randn((2, 2 * G, T, d), generator=gen).to(BF16)
    Q[..., 7] = 2.0 ** span
    for weights in (False, True):
        O = torch.empty(Q.shape, dtype=out, device="cuda")
        lse = torch.empty(Q.shape[:3], device="cuda") if weights else None
        acc = torch.zeros((2, 2, st.max_pages * 32), device="cuda") if weights else None
        ws = torch.empty(aq.attnq_kv4_attn_workspace(st.cache, 2, st.max_pages, 2 * G, T), dtype=torch.uint8,
                         device="cuda")
        aq.attnq_kv4_attn(st.cache, aq.AttnqKv4Seqs(st.table, st.lens_t), Q.cuda(), O, True, ws, lse=lse, acc_out=acc)
        assert aq.attnq_device_status() == 0
        half, p_err, floor = (2.0 ** -8, 2.0 ** -11, 2.0 ** -32) if out == BF16 else (2.0 ** -24, 2.0 ** -21, 2.0 ** -40)
        for b, L in enumerate(st.lens):
            for h in range(2):
                k, v = st.held(b, h)
                total, w_tol = torch.zeros(L, dtype=torch.float64), torch.zeros(L, dtype=torch.float64)
                for hq in range(h * G, (h + 1) * G):
                    o, l, p, A, bound = ref.attention(Q[b, hq].double(), k, v, d ** -0.5, True)
                    e_s = bound * (d * 2.0 ** -23 + 2.0 ** -21) + 2.0 ** -21
                    e_s = e_s + 2.0 ** -39 * 2.0 ** span * k.abs().sum(-1).amax() * d ** -0.5
                    tol = half * o.abs() + A * (p_err + 2 * e_s + (L + 16) * 2.0 ** -23)[:, None] + floor * v.abs().sum(0)
                    got = O[b, hq].cpu().double()
                    assert ((got - o).abs() <= tol).all(), (b, hq, ((got - o).abs() / tol).max())
                    if weights:
                        e_l = e_s + (L + 16) * 2.0 ** -23 + 2.0 ** -22 * l.abs()
                        assert ((lse[b, hq].cpu().double() - l).abs() <= e_l).all()
                        total += p.sum(0)
                        w_tol += (p * (2 * e_s + e_l + 2.0 ** -20)[:, None]).sum(0)
                if weights:
                    tol = w_tol + total * 2.0 ** -23 * (2 + G * T)
                    assert ((acc[b, h, :L].cpu().double() - total).abs() <= tol).all()


@pytest.mark.parametrize("T,G,out", [(1, 4, BF16), (1, 4, F32), (300, 1, BF16), (300, 1, F32), (150, 4, BF16)])
def test_weights_near_the_smallest_held(T, G, out):
    """Most tokens 2^-20 to 2^-36 of a row's largest weight, with values 2^20 times the largest one's.

    P = 2^b p is held in fp16, whose last place is 2^-24: a weight is off by 2^-11 of itself or half of that
    step, 2^(-25 - b) of the row's largest; b = 15, or 7 in the kernel for many rows with bf16 outputs."""
    aq = _aq()
    d, L = 64, 3000
    st = Setup([L], 1, d, 64, seed=T + G)
    gen = torch.Generator().manual_seed(T)
    # constant rows are held as 6 s: one step of s, an eighth of it, is one level of scores
    level = torch.randint(3, 8, (L,), generator=gen).double()
    level[17] = 0.0
    st.K = (12.0 - level[None, None, :, None]).expand(1, 1, L, d).to(BF16).contiguous() * 1.5
    st.V = torch.randn((1, 1, L, d), generator=gen) * 1024
    st.V[0, 0, 17] /= 2.0 ** 20
    st.V = st.V.to(BF16)
    aq.attnq_kv4_append(st.cache, st.seqs, st.K.cuda(), st.V.cuda())
    k, v = st.held(0, 0)
    # one level is 5 to 7 in log2 units: 1.5 d beta scale log2 e
    beta = (5.0 + 2 * torch.rand((1, G, T, 1), generator=gen)) / (1.5 * d * 0.125 * math.log2(math.e))
    Q = beta.expand(1, G, T, d).to(BF16)
    O = torch.empty(Q.shape, dtype=out, device="cuda")
    ws = torch.empty(aq.attnq_kv4_attn_workspace(st.cache, 1, st.max_pages, G, T), dtype=torch.uint8, device="cuda")
    aq.attnq_kv4_attn(st.cache, aq.AttnqKv4Seqs(st.table, st.lens_t), Q.cuda(), O, False, ws)
    assert aq.attnq_device_status() == 0
    half, p_err, floor = (2.0 ** -8, 2.0 ** -11, 2.0 ** -40) if out == BF16 else (2.0 ** -24, 2.0 ** -21, 2.0 ** -40)
    if T * G > 32 and out == BF16:
        floor = 2.0 ** -32
    for hq in range(G):
        o, _, p, A, bound = ref.attention(Q[0, hq].double(), k, v, 0.125, False)
        e_s = bound * (d * 2.0 ** -23 + 2.0 ** -21) + 2.0 ** -21
        tol = half * o.abs() + A * (p_err + 2 * e_s + (L + 16) * 2.0 ** -23)[:, None]
        tol = tol + floor * p.amax(-1, keepdim=True) * v.abs().sum(0)
        assert p.amax() > 0.9 and p.median() < 2.0 ** -20
        assert ((O[0, hq].cpu().double() - o).abs() <= tol).all(), (hq, ((O[0, hq].cpu().double() - o).abs() / tol).max())


@pytest.mark.parametrize("T,G,out", [(4, 1, BF16), (6, 4, F32), (20, 2, BF16), (300, 1, BF16), (300, 1, F32)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_masked_value_that_is_not_finite(T, G, out, bad):
    """A NaN or an infinity in V or K of the last token is reported when it is written, and rows that do not see
    that token are as if it were not there (0 times a NaN would be one)."""
    aq = _aq()
    st = Setup([T + 70], 2, 64, 16, seed=T)
    L = T + 70
    gen = torch.Generator().manual_seed(G)
    Q = torch.randn((1, 2 * G, T, 64), generator=gen).to(BF16)
    one = aq.AttnqKv4Seqs(st.table, st.lens_t)
    for which in "VK":
        x = {"K": st.K[:, :, -1:].clone(), "V": st.V[:, :, -1:].clone()}
        x[which][..., 21] = bad
        aq.attnq_kv4_append(st.cache, one, x["K"].cuda(), x["V"].cuda())
        assert aq.attnq_device_status() == 4
        O = torch.empty(Q.shape, dtype=out, device="cuda")
        lse = torch.empty(Q.shape[:3], device="cuda")
        ws = torch.empty(aq.attnq_kv4_attn_workspace(st.cache, 1, st.max_pages, 2 * G, T), dtype=torch.uint8, device="cuda")
        aq.attnq_kv4_attn(st.cache, one, Q.cuda(), O, True, ws, lse=lse)
        aq.attnq_device_status()
        half, p_err, floor = (2.0 ** -8, 2.0 ** -11, 2.0 ** -32) if out == BF16 else (2.0 ** -24, 2.0 ** -21, 2.0 ** -40)
        for hq in range(2 * G):
            k, v = (t[:L - 1] for t in st.held(0, hq // G))
            o, l, _, A, bound = ref.attention(Q[0, hq, :T - 1].double(), k, v, 0.125, True)
            e_s = bound * (64 * 2.0 ** -23 + 2.0 ** -21) + 2.0 ** -21
            tol = half * o.abs() + A * (p_err + 2 * e_s + (L + 16) * 2.0 ** -23)[:, None] + floor * v.abs().sum(0)
            assert ((O[0, hq, :T - 1].cpu().double() - o).abs() <= tol).all(), (which, hq)
            e_l = e_s + (L + 16) * 2.0 ** -23 + 2.0 ** -22 * l.abs()
            assert ((lse[0, hq, :T - 1].cpu().double() - l).abs() <= e_l).all()
        aq.attnq_kv4_append(st.cache, one, st.K[:, :, -1:].cuda(), st.V[:, :, -1:].cuda())
