"""The distillation loss against a teacher's top logits, and its gradient,
against the plain 64-bit form.

Tolerances, to first order.  An fp16-rounded weight is off by at most 2^-11 of
itself and the tensor cores add in fp32, so a logit of the kernel is off by
dz_v <= (2^-11 + H 2^-23) sum_d |h_d w_vd|; an exact one by H 2^-23 of it.
lse: the mean of those errors under the softmax (over T), the teacher's tokens
with their exact error, plus a few fp32 steps.  loss: lse's and, under p, the
teacher logits'.  dh: each coefficient's error -- q_v (2 dz_v / T + the error
of lse) + half an fp16 step of the coefficient, below 2^-14 one of 2^-24 over
the scale 2^14 -- times |w_v|, plus 2^-11 + V 2^-23 of |coefficient w_v|, plus
the rounding to bf16."""
import pytest
import torch

from ops_ref import U, distill64, gen, make_table, table64
from verify_vocab_blocked_gb300 import build as qbuild
from verify_vocab_blocked_gb300 import qhead

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qbuild.build()
    qhead.lib()


def _case(M, V, H, bits, K, cap, seed, t_dtype=torch.float32, sb=torch.float16, near=True):
    head = qhead.Head(*make_table(V, H, bits, seed, sb), bits, softcap=cap)
    W = table64(head.wq, head.scales, head.biases, bits)
    g = gen(seed + 1)
    ids = torch.rand(M, V, device="cuda", generator=g).argsort(1)[:, :K] if V <= 4096 else \
        torch.randint(0, V, (M, K), device="cuda", generator=g)
    h = torch.randn(M, H, device="cuda", generator=g, dtype=torch.float64) * 0.5
    t = 3 * torch.randn(M, ids.shape[1], device="cuda", generator=g)
    if near:                                  # the student's mass near the teacher's
        rows = W[ids]
        h = 0.2 * h + torch.einsum("mk,mkh->mh", (8 + t.double()) / rows.square().sum(2), rows)
    return head, W, h.to(torch.bfloat16), ids.int(), t.to(t_dtype)


def _check(head, W, h, ids, t, T, mask=None, dloss=None):
    M, K = ids.shape
    V, cap, H = head.V, head.softcap, head.H
    if dloss is None:
        dloss = torch.rand(M, device="cuda", generator=gen(99)) * 2 - 1
    loss, lse, kept = qhead.distill_fwd(head, h, ids, t, T, mask)
    dh = qhead.distill_bwd(head, h, ids, t, kept, lse, dloss, T, mask)
    on = torch.ones(M, dtype=torch.bool, device="cuda") if mask is None else mask.bool()
    hd = h.double().requires_grad_(True)
    L, E, z, p = distill64(W, hd, ids, t, T, cap, mask)
    ref_dh, = torch.autograd.grad((L * dloss.double()).sum(), hd)
    L, E, z = L.detach(), E.detach(), z.detach()
    with torch.no_grad():
        mag = h.double().abs() @ W.abs().t()                         # sum |h w|
        ok = ids >= 0
        at = ids.clamp_min(0).long()
        q = (z / T - E[:, None]).exp()
        listed = torch.zeros_like(q).scatter_add_(1, at, ok.double()) > 0
        d_exact, d_mma = H * 2 * U * mag, (2.0 ** -11 + H * 2 * U) * mag
        step = 16 * U * (1 + z.abs().amax(1) / T)                    # fp32 steps on values this large
        e_lse = (q * torch.where(listed, d_exact, d_mma)).sum(1) / T + step
        e_zk = (d_exact.gather(1, at) + 8 * U * (1 + z.gather(1, at).abs())) * ok
        e_loss = e_lse + (p * e_zk).sum(1) / T + step * 4
        zr = z.gather(1, at) * ok
        assert (((kept[:, :K].double() - zr).abs() <= e_zk) | ~on[:, None]).all()
        assert (kept[~on][:, :K] == 0).all() and (lse[~on] == 0).all() and (loss[~on] == 0).all()
        assert (((lse.double() - E).abs() <= e_lse) | ~on).all()
        assert ((loss.double() - L).abs() <= e_loss).all(), \
            ((loss.double() - L).abs() / e_loss).max().item()
        ps = torch.zeros_like(q).scatter_add_(1, at, p)
        sech2 = 1 - (z / cap).square() if cap > 0 else torch.ones_like(z)
        coef = (q - ps) * sech2
        d = torch.where(listed, d_exact, d_mma)
        e_c = q * (2 * d / T + e_lse[:, None] + 16 * U * (1 + z.abs() / T)) + 8 * U * ps \
            + (2 * q * d / cap if cap > 0 else 0) + 2.0 ** -11 * coef.abs() + 2.0 ** -38
        e_dh = (e_c + (2.0 ** -11 + V * 2 * U) * coef.abs()) @ W.abs()
        g = (dloss.double().abs() / T)[:, None]
        some = (p.sum(1) > 0) & on
        ref_dh = torch.where(some[:, None], ref_dh, 0.0)
        tol = g * e_dh + 2.0 ** -8 * ref_dh.abs() + 1e-38
        assert dh.dtype == torch.bfloat16
        assert (((dh.double() - ref_dh).abs() <= 1.02 * tol) | ~some[:, None]).all(), \
            ((dh.double() - ref_dh).abs() / tol).max().item()
        assert (dh[~some] == 0).all()
        # no worse than a few parts in a thousand of the rows' norms, over all
        n = ref_dh.norm()
        if n > 0:
            assert ((dh.double() - ref_dh).norm() / n).item() <= 4e-3
    return loss, lse, kept, dh


@pytest.mark.parametrize("M,V,H,bits,K,cap,T,near", [
    (1, 300, 128, 4, 1, 0.0, 1.0, True),
    (1, 5, 256, 8, 5, 30.0, 1.0, True),
    (3, 1, 128, 4, 1, 0.0, 2.0, False),       # a vocabulary of one: loss and gradient 0
    (13, 2000, 256, 4, 20, 30.0, 1.0, True),
    (64, 1023, 384, 8, 7, 0.0, 3.5, True),
    (130, 2048, 640, 4, 64, 30.0, 2.0, True),
    (257, 1500, 1536, 8, 33, 0.0, 1.0, True),
    (300, 777, 512, 4, 128, 20.0, 0.5, True),
    (40, 3001, 2560, 4, 16, 30.0, 1.0, False),   # the student far from the teacher
    (20, 1500, 256, 4, 1024, 0.0, 1.0, True),
    (9, 1024, 128, 8, 1024, 0.0, 1.0, True),     # every vocabulary row listed
])
def test_against_64_bits(M, V, H, bits, K, cap, T, near):
    _check(*_case(M, V, H, bits, K, cap, M + V, near=near), T)


@pytest.mark.parametrize("t_dtype,sb", [(torch.bfloat16, torch.bfloat16),
                                        (torch.float16, torch.float16)])
def test_types(t_dtype, sb):
    _check(*_case(50, 900, 256, 4, 12, 30.0, 5, t_dtype, sb), 1.0)


def test_masks_padding_and_empty_rows():
    head, W, h, ids, t = _case(300, 1200, 256, 4, 10, 30.0, 17)
    mask = torch.rand(300, device="cuda", generator=gen(3)) < 0.6
    ids[::3, 4:] = -1                    # short lists
    ids[1::7] = -5                       # nothing listed
    t[2::11, ::2] = -float("inf")        # entries without mass
    t[5::13] = -float("inf")             # no mass at all
    t[ids < 0] = float("nan")            # what stands at a padding entry is not looked at
    tt = torch.where(ids < 0, -float("inf"), t)
    loss, _, _, dh = _check(head, W, h, ids, tt, 1.0, mask)
    loss2, lse2, zk2 = qhead.distill_fwd(head, h, ids, t, 1.0, mask.to(torch.uint8))
    assert torch.equal(loss, loss2)
    assert (loss[1::7] == 0).all() and (dh[1::7] == 0).all()
    _check(head, W, h, ids, tt, 1.0, torch.zeros(300, dtype=torch.bool, device="cuda"))


def test_lowest_values_and_far_apart_logits():
    head, W, h, ids, t = _case(20, 600, 256, 8, 8, 0.0, 23)
    t[:10, 1:] = torch.finfo(torch.float32).min      # a one-hot teacher
    t[10:] *= 1e4
    _check(head, W, h, ids, t, 1.0)


def test_duplicates_count_together():
    head, W, h, ids, t = _case(30, 500, 256, 4, 6, 30.0, 29)
    ids[:, 3] = ids[:, 0]
    ids[:, 5] = ids[:, 0]
    _check(head, W, h, ids, t, 1.0)


def test_bad_rows_are_nan_and_alone():
    head, W, h, ids, t = _case(8, 500, 256, 4, 6, 0.0, 31)
    good, glse, gzk = qhead.distill_fwd(head, h, ids, t)
    ids2, t2 = ids.clone(), t.clone()
    ids2[1, 2] = 500
    ids2[2, 0] = 2 ** 31 - 1
    t2[3, 1] = float("nan")
    t2[4, 5] = float("inf")
    loss, lse, kept = qhead.distill_fwd(head, h, ids2, t2)
    dl = torch.ones(8, device="cuda")
    dh = qhead.distill_bwd(head, h, ids2, t2, kept, lse, dl)
    bad = [1, 2, 3, 4]
    fine = [0, 5, 6, 7]
    assert torch.isnan(loss[bad]).all() and torch.isnan(dh[bad]).all()
    assert torch.equal(loss[fine], good[fine])
    assert torch.equal(dh[fine], qhead.distill_bwd(head, h, ids, t, gzk, glse, dl)[fine])


def test_reduces_to_the_target_loss():
    """A one-entry teacher is the target's negative log-probability: within the
    kernels' own error of the lse (a target's term exact here)."""
    head, W, h, ids, t = _case(200, 3000, 512, 4, 1, 30.0, 37)
    loss, lse, _ = qhead.distill_fwd(head, h, ids, t)
    logp, lse0, _ = qhead.fwd(head, h, ids[:, 0].contiguous())
    assert (loss + logp).abs().max() <= 2e-3
    assert (lse - lse0).abs().max() <= 2e-3


def test_gradient_against_differences():
    M, V, H, K = 6, 700, 256, 9
    head, W, h, ids, t = _case(M, V, H, 4, K, 30.0, 41)
    dl = torch.rand(M, device="cuda", generator=gen(4)) + 0.5
    loss, lse, kept = qhead.distill_fwd(head, h, ids, t, 1.5)
    dh = qhead.distill_bwd(head, h, ids, t, kept, lse, dl, 1.5).double()
    d = torch.randn(M, H, device="cuda", generator=gen(5), dtype=torch.float64)
    d /= d.norm()

    def f(e):
        return (distill64(W, h.double() + e * d, ids, t, 1.5, 30.0)[0] * dl.double()).sum().item()

    e = 1e-3
    quot = (f(e) - f(-e)) / (2 * e)
    got = (dh * d).sum().item()
    # dh is within 4e-3 of its norm (bf16 and fp16 operands), d has norm 1
    assert abs(quot - got) <= 4e-3 * dh.norm().item() + 1e-5


def test_deterministic_on_streams_and_in_a_graph():
    head, W, h, ids, t = _case(300, 2500, 256, 8, 24, 0.0, 43)
    dl = torch.rand(300, device="cuda", generator=gen(6))

    def both():
        loss, lse, kept = qhead.distill_fwd(head, h, ids, t, 2.0)
        return loss, lse, kept, qhead.distill_bwd(head, h, ids, t, kept, lse, dl, 2.0)

    first = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = both()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = both()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, third))


def test_several_vocab_chunks():
    """A coefficient block larger than its budget: the backward runs the
    vocabulary in chunks, each patched with its own listed tokens."""
    M, V, H, K = 33000, 70000, 128, 6
    head = qhead.Head(*make_table(V, H, 4, 47), 4)
    g = gen(48)
    h = torch.randn(M, H, device="cuda", generator=g).to(torch.bfloat16)
    ids = torch.randint(0, V, (M, K), device="cuda", generator=g).int()
    ids[:, 0] = torch.arange(M, device="cuda").int() % V
    t = torch.randn(M, K, device="cuda", generator=g)
    dl = torch.ones(M, device="cuda")
    rows = torch.tensor([0, 1, 127, 128, 255, 256, 16383, 16384, 20000, 32999], device="cuda")
    loss, lse, kept = qhead.distill_fwd(head, h, ids, t)
    dh = qhead.distill_bwd(head, h, ids, t, kept, lse, dl)
    W = table64(head.wq, head.scales, head.biases, 4)
    hd = h[rows].double().requires_grad_(True)
    L, E, _, _ = distill64(W, hd, ids[rows], t[rows], 1.0, 0.0)
    ref, = torch.autograd.grad(L.sum(), hd)
    assert (lse[rows].double() - E).abs().max() <= 2e-3
    assert (loss[rows].double() - L).abs().max() <= 2e-3
    assert ((dh[rows].double() - ref).norm(dim=1) <= 4e-3 * ref.norm(dim=1)).all()


def test_stalled_kernel_gives_nan():
    """The forward's time limit: a call whose loads never come ends by itself
    and its active rows are NaN; the backward's too."""
    head, W, h, ids, t = _case(20, 700, 256, 4, 4, 0.0, 53)
    loss, lse, kept = qhead.distill_fwd(head, h, ids, t)
    mask = torch.ones(20, dtype=torch.bool, device="cuda")
    mask[3] = False
    qhead.test_stall_next_call()
    bad, blse, _ = qhead.distill_fwd(head, h, ids, t, 1.0, mask)
    assert torch.isnan(bad[mask]).all() and torch.isnan(blse[mask]).all() and bad[3] == 0
    dl = torch.ones(20, device="cuda")
    qhead.test_stall_next_call()
    dh = qhead.distill_bwd(head, h, ids, t, kept, lse, dl, 1.0, mask)
    assert torch.isnan(dh[mask]).all() and (dh[3] == 0).all()
    assert torch.equal(loss, qhead.distill_fwd(head, h, ids, t)[0])


@pytest.mark.parametrize("M", [1, 8, 9, 16, 17, 127, 128, 129])
@pytest.mark.parametrize("bits,cap,T", [(4, 30.0, 1.0), (8, 0.0, 2.0)])
def test_row_counts_where_the_kernels_change(M, bits, cap, T):
    """Up to 16 rows the weight-streaming kernel, up to 128 the kept logits; a
    vocabulary that is no multiple of their blocks, some rows masked."""
    head, W, h, ids, t = _case(M, 1237, 384, bits, 11, cap, 60 + M)
    mask = torch.rand(M, device="cuda", generator=gen(M)) < 0.8
    _check(head, W, h, ids, t, T, mask)


@pytest.mark.parametrize("M", [6, 60, 200])
def test_student_far_from_its_teacher(M):
    """The student's mass on tokens that the teacher does not list, a few of
    them holding most of it: their logits are exact too, so the loss is within
    1e-5 of its value (the tail's 3e-4 logit errors, averaged)."""
    head, W, h, ids, t = _case(M, 4000, 256, 4, 8, 0.0, 71, near=False)
    g = gen(72)
    far = torch.randint(0, 4000, (M, 5), device="cuda", generator=g)
    rows = W[far]
    h = (0.1 * h.double() + torch.einsum("mk,mkh->mh", 14.0 / rows.square().sum(2), rows)).to(torch.bfloat16)
    loss, _, _, _ = _check(head, W, h, ids, t, 1.0)
    ref = distill64(W, h.double(), ids, t, 1.0, 0.0)[0]
    assert ((loss.double() - ref).norm() / ref.norm()).item() <= 1e-5


@pytest.mark.parametrize("M", [5, 40, 150])
def test_nan_rows_stay_alone(M):
    head, W, h, ids, t = _case(M, 900, 256, 8, 6, 30.0, 80)
    good, _, _ = qhead.distill_fwd(head, h, ids, t)
    h2 = h.clone()
    h2[2, 7] = float("nan")
    h2[4] = float("inf")
    loss, lse, kept = qhead.distill_fwd(head, h2, ids, t)
    dh = qhead.distill_bwd(head, h2, ids, t, kept, lse, torch.ones(M, device="cuda"))
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[2] = bad[4] = True
    assert torch.isnan(loss[2]) and not torch.isfinite(loss[4]) and torch.isnan(dh[2]).all()
    assert torch.equal(loss[~bad], good[~bad]) and torch.isfinite(dh[~bad]).all()


def test_many_rows_of_a_small_vocabulary():
    """More rows than a grid's second axis holds, logits kept."""
    M, V, H, K = 70001, 300, 128, 3
    head = qhead.Head(*make_table(V, H, 8, 90), 8, softcap=20.0)
    g = gen(91)
    h = torch.randn(M, H, device="cuda", generator=g).to(torch.bfloat16)
    ids = torch.randint(0, V, (M, K), device="cuda", generator=g).int()
    t = torch.randn(M, K, device="cuda", generator=g)
    loss, lse, kept = qhead.distill_fwd(head, h, ids, t)
    dh = qhead.distill_bwd(head, h, ids, t, kept, lse, torch.ones(M, device="cuda"))
    W = table64(head.wq, head.scales, head.biases, 8)
    hd = h.double().requires_grad_(True)
    L, E, _, _ = distill64(W, hd, ids, t, 1.0, 20.0)
    ref, = torch.autograd.grad(L.sum(), hd)
    assert (lse.double() - E).abs().max() <= 2e-3
    assert (loss.double() - L).abs().max() <= 2e-3
    assert ((dh.double() - ref).norm(dim=1) <= 4e-3 * ref.norm(dim=1) + 1e-7).all()


def test_logits_too_large_to_keep():
    """Past 4 GiB of logits the backward runs the logit kernel again: the same
    gradient as with the logits kept, within the coefficients' own rounding."""
    M, V, H, K = 4500, 262144, 128, 4
    head = qhead.Head(*make_table(V, H, 4, 92), 4)
    g = gen(93)
    h = torch.randn(M, H, device="cuda", generator=g).to(torch.bfloat16)
    ids = torch.randint(0, V, (M, K), device="cuda", generator=g).int()
    t = torch.randn(M, K, device="cuda", generator=g)
    dl = torch.ones(M, device="cuda")
    loss, lse, kept = qhead.distill_fwd(head, h, ids, t)
    assert kept.shape[1] < V
    dh = qhead.distill_bwd(head, h, ids, t, kept, lse, dl)
    n = 400
    loss2, lse2, kept2 = qhead.distill_fwd(head, h[:n], ids[:n], t[:n])
    assert kept2.shape[1] > V
    dh2 = qhead.distill_bwd(head, h[:n], ids[:n], t[:n], kept2, lse2, dl[:n])
    # an fp32 sum of V terms in two groupings; a coefficient's half step in fp16 twice,
    # half a step of bf16 twice
    assert (lse[:n] - lse2).abs().max() <= 1e-4 and (loss[:n] - loss2).abs().max() <= 1e-4
    assert ((dh[:n].double() - dh2.double()).norm() / dh2.double().norm()).item() <= 2 ** -7


@pytest.mark.parametrize("M,V,H,bits,on", [
    (9, 260, 2560, 4, 1.0), (16, 511, 2560, 8, 0.4), (12, 700, 3584, 4, 1.0), (13, 600, 4096, 8, 0.8),
    (16, 257, 8192, 4, 1.0), (11, 1, 128, 4, 1.0), (10, 100, 8192, 8, 0.5),
])
def test_two_groups_of_rows(M, V, H, bits, on):
    """9 to 16 rows: one pass over the table for both groups of 8 while their h fits
    shared memory, one for each where it does not."""
    head, W, h, ids, t = _case(M, V, H, bits, min(V, 9), 30.0, 90 + M)
    mask = torch.rand(M, device="cuda", generator=gen(91)) < on
    _check(head, W, h, ids, t, 1.0, mask if on < 1 else None)


def test_nan_row_of_the_second_group():
    head, W, h, ids, t = _case(12, 900, 256, 4, 6, 30.0, 80)
    good, lse0, _ = qhead.distill_fwd(head, h, ids, t)
    h[10, 3] = float("nan")
    loss, lse, kept = qhead.distill_fwd(head, h, ids, t)
    dh = qhead.distill_bwd(head, h, ids, t, kept, lse, torch.ones(12, device="cuda"))
    rest = torch.arange(12, device="cuda") != 10
    assert torch.isnan(loss[10]) and torch.isnan(dh[10]).all()
    assert torch.equal(loss[rest], good[rest]) and torch.equal(lse[rest], lse0[rest])
    assert torch.isfinite(dh[rest]).all()
