"""The output head's losses (head_loss, head_distill) and the embedding's gradient
(embed_grad).

On the CPU: the refusals. On the GPU: every result against a plain implementation
in 64 bits, at sizes around the kernels' tiles, for each type, with masks, views,
strides, groups of rows, streams and graphs, and in one run with the update over a
list of tensors.

Tolerances. Elementwise, from the roundings that a result goes through. With
u(t) = finfo(t).eps / 2, a half step of type t relative to the value, and f = 2^-24:
  a logit z = sum h w of `dim` products: dim + 2 roundings of float32 of the sum's
    magnitude S = sum |h| |w|; with float32 inputs each product is good to 3 * 2^-22
    (two halves of 11 bits each, the product of the low halves left out)
  log-sum-exp: the error of the largest such logit, twice that of the exponential's
    argument (in units of log 2, of magnitude up to Z: 4 Z f) and of the hardware's
    exponential and logarithm (8 f), and the sum's roundings (32 in a lane, 2 across
    lanes, then one per 64 columns at most: (V / 64 + 40) f)
  a gradient's softmax value p: the two errors above, relative; and its roundings to
    the type, ROUNDINGS of them at most: once as an exponential, once normalized or
    moved by its row's factor, and the hidden row times that factor. Float32 values
    are held in 22 bits each time: 2^-22
  a gradient: that of its terms, one rounding of float32 for each term and for each
    of up to 64 splits, and the result's own rounding
Rounding halves of the smallest subnormal of float16 come on top."""
import ctypes
import math

import numpy as np
import pytest
import torch

import resumable_checkpoint_state_amd as rcs
from resumable_checkpoint_state_amd import vocabulary

gpu = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]
F = 2.0 ** -24
ROUNDINGS = 3
IGNORE = -100


# ----------------------------------------------------------- the plain forms

def unit(dtype):
    return 2.0 ** -22 if dtype == F32 else torch.finfo(dtype).eps / 2


def least(dtype):
    """Half of the smallest step there is."""
    return 2.0 ** -25 if dtype == F16 else 2.0 ** -134


def one_hot(targets, vocab):
    """The targets' distribution: (rows, vocab), and which rows have a loss."""
    ok = targets != IGNORE
    q = torch.zeros(targets.numel(), vocab, dtype=torch.float64, device=targets.device)
    q.scatter_(1, targets.clamp(min=0).view(-1, 1).long(), 1.0)
    return q * ok.view(-1, 1), ok


def teacher(index, logits, vocab, tau):
    there = (index >= 0) & (logits != -math.inf)
    ok = there.any(1)
    y = (logits.double() / tau).masked_fill(~there, -math.inf)
    p = torch.softmax(torch.where(ok.view(-1, 1), y, torch.zeros_like(y)), 1) * there
    q = torch.zeros(index.shape[0], vocab, dtype=torch.float64, device=index.device)
    q.scatter_add_(1, index.clamp(min=0).long(), p)
    logp = torch.where(p > 0, torch.log(p), torch.zeros_like(p))
    return q * ok.view(-1, 1), ok, (p * logp).sum(1)


def plain(h, w, q, ok, scale, mean, tau=1.0, entropy=None):
    """Loss, losses and gradients in 64 bits, and how far each may be off."""
    dtype, (t, d), v = h.dtype, h.shape, w.shape[0]
    h, w = h.double(), w.double()
    h = torch.where(ok.view(-1, 1), h, torch.zeros_like(h))
    z = h @ w.t() / tau
    size = (h.abs() @ w.abs().t() / tau).amax(1)  # S
    lse = torch.logsumexp(z, 1)
    losses = lse - (q * z).sum(1)
    if entropy is not None:
        losses = (losses + entropy) * tau * tau
    losses = losses * ok
    n = max(int(ok.sum()), 1) if mean else 1
    p = torch.exp(z - lse.view(-1, 1)) * ok.view(-1, 1)
    g = (p - q) * (scale * tau / n)
    # the errors
    product = 3 * 2.0 ** -22 if dtype == F32 else 0.0
    top = z.abs().amax(1) / math.log(2)
    e_z = size * ((d + 2) * F + product)
    e_lse = e_z + (8 * top + 16 + v / 64 + 40) * F
    e_loss = (e_z + e_lse + 8 * F * top) * (tau * tau) + 4 * F * losses.abs()
    if entropy is not None:
        e_loss = e_loss + tau * tau * 64 * F * (1 + top + entropy.abs())
    loss, e_total = losses.sum() / n, e_loss.sum() / n + 4 * F * losses.sum().abs() / n
    k = scale * tau / n
    e_g = (p * (e_z + e_lse + 16 * F).view(-1, 1) + p * 16 * F + q * 64 * F) * abs(k) + \
        g.abs() * (1 + unit(dtype)) ** ROUNDINGS * ROUNDINGS * unit(dtype)
    if dtype != BF16:  # held as 2^14 times as much, in steps of 2^-25 at least, twice
        e_g = e_g + 2 * 2.0 ** -39 * abs(k)
    else:  # exponentials, whose factor is at most 1, below the normal numbers may be zero
        e_g = e_g + 2.0 ** -126 * abs(k)
    gh, gw = g @ w, g.t() @ h
    terms = lambda n_terms: (n_terms + 64) * F  # noqa: E731
    e_gh = e_g @ w.abs() + terms(v) * (g.abs() @ w.abs())
    e_gw = e_g.t() @ h.abs() + terms(t) * (g.abs().t() @ h.abs())
    if dtype == F32:  # the other side's 22 bits
        e_gh = e_gh + 3 * 2.0 ** -22 * (g.abs() @ w.abs())
        e_gw = e_gw + 3 * 2.0 ** -22 * (g.abs().t() @ h.abs())
    return (loss, losses, gh, gw), (e_total, e_loss, e_gh, e_gw)


def near(got, want, err, what):
    got = got.double().view(want.shape)
    assert torch.isfinite(got).all(), what
    off = (got - want).abs()
    out = dict(what=what, worst=float((off - err).max()), off=float(off.max()))
    assert bool((off <= err).all()), out


def check(h, w, q, ok, results, scale, mean, tau=1.0, entropy=None, before=None):
    """results: loss, losses, gh, gw (None: not asked for); before: what gw held."""
    want, err = plain(h, w, q, ok, scale, mean, tau, entropy)
    for name, got, x, e in zip(("loss", "losses", "grad_hidden", "grad_weight"), results, want,
                               err):
        if got is None:
            continue
        if name == "grad_weight" and before is not None:
            x = x + before.double()
            e = e + 2 * F * x.abs()
        half = torch.finfo(got.dtype).eps / 2
        near(got, x, e * (1 + half) + x.abs() * half + least(got.dtype) + 1e-300, name)


def data(t, v, d, dtype, seed=0, spread=1.5, masked=0.0, view=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    h, w = rand(t, d).to(dtype), (rand(v, d) * (spread / math.sqrt(d))).to(dtype)
    targets = torch.randint(0, v, (t,), generator=g, device="cuda")
    targets[torch.rand(t, generator=g, device="cuda") < masked] = IGNORE
    if view:  # at odd offsets, and with rows further apart than they are long
        flat = torch.zeros(t * (d + 3) + 5, dtype=dtype, device="cuda")
        hv = flat[5:].view(t, d + 3)[:, :d]
        hv.copy_(h)
        flat = torch.zeros(v * d + 7, dtype=dtype, device="cuda")
        wv = flat[7:].view(v, d)
        wv.copy_(w)
        h, w = hv, wv
    return h, w, targets


def scale_of(dtype):
    return 1024.0 if dtype == F16 else 1.0


def run_loss(h, w, targets, grads=True, gw_type=None, **more):
    losses = torch.full(targets.shape, 7.0, device="cuda")
    gh = gw = None
    if grads:
        gh = torch.full(h.shape, 7.0, dtype=h.dtype, device="cuda")
        gw = torch.full(w.shape, 7.0, dtype=gw_type or w.dtype, device="cuda")
        more = dict(grad_hidden=gh, grad_weight=gw, accumulate=False) | more
    loss = rcs.head_loss(h, w, targets, losses=losses, **more)
    return loss, losses, gh, gw


# ------------------------------------------------------------------ refusals

def _args(**more):
    a = vocabulary._Head(hidden=256, weight=512, rows=4, vocab=8, dim=16, hidden_stride=16,
                         weight_stride=16, type=1, mean=1, scale=1.0, loss=64, limit=1 << 20,
                         workspace=4096, workspace_bytes=1 << 30)
    for k, x in more.items():
        setattr(a, k, x)
    return a


@pytest.mark.parametrize("bad", [
    {"rows": -1}, {"rows": (1 << 23) + 1}, {"vocab": 0}, {"vocab": -3},
    {"vocab": (1 << 22) + 1}, {"dim": 0}, {"dim": (1 << 16) + 1}, {"type": 3}, {"type": -1},
    {"grad_weight": 1024, "grad_weight_type": 9, "grad_weight_stride": 16}])
def test_workspace_refuses_bad_sizes(bad):
    assert rcs.lib().rcs_head_workspace(ctypes.byref(_args(**bad)), 0) == rcs.EINVAL


def test_workspace_sizes():
    size = lambda entries=0, **m: rcs.lib().rcs_head_workspace(  # noqa: E731
        ctypes.byref(_args(**m)), entries)
    assert size() > 0
    assert size(entries=-1) == rcs.EINVAL and size(entries=1025) == rcs.EINVAL
    assert size(entries=1024) > size(entries=1)
    # it holds the rows' exponentials, and of no more of them than the limit allows
    big = dict(rows=65536, vocab=131072, dim=64, grad_hidden=1024, grad_hidden_stride=64,
               hidden_stride=64, weight_stride=64)
    assert size(limit=1 << 40, **big) > 65536 * 131072 * 2
    assert size(limit=1 << 30, **big) < 2 << 30
    assert rcs.lib().rcs_head_workspace(None, 0) == rcs.EINVAL
    assert rcs.lib().rcs_embed_workspace(10, 100, 64) > 0
    for bad in ((-1, 10, 4), (1, 0, 4), (1, 10, 0), (1, 10, (1 << 16) + 1),
                ((1 << 23) + 1, 10, 4), (1, (1 << 30) + 1, 4)):
        assert rcs.lib().rcs_embed_workspace(*bad) == rcs.EINVAL


@pytest.mark.parametrize("bad", [
    {"scale": math.inf}, {"scale": math.nan}, {"hidden_stride": 15}, {"weight_stride": 15},
    {"hidden": None}, {"weight": None}, {"hidden": 257}, {"weight": 513}, {"loss": None}])
def test_calls_refuse_on_the_host(bad):
    L = rcs.lib()
    assert L.head_loss(ctypes.byref(_args(**bad)), 128, 1, -100, None) == rcs.EINVAL
    assert L.head_distill(ctypes.byref(_args(**bad)), 128, 1, 128, 0, 2, 1.0, None) == rcs.EINVAL


def test_calls_refuse_targets_on_the_host():
    L, a = rcs.lib(), ctypes.byref(_args())
    assert L.head_loss(None, 128, 1, -100, None) == rcs.EINVAL
    assert L.head_loss(a, 128, 2, -100, None) == rcs.EINVAL
    assert L.head_loss(a, None, 1, -100, None) == rcs.EINVAL
    assert L.head_distill(a, 128, 1, 128, 0, 0, 1.0, None) == rcs.EINVAL
    assert L.head_distill(a, 128, 1, 128, 0, 1025, 1.0, None) == rcs.EINVAL
    for tau in (0.0, -1.0, math.inf, math.nan):
        assert L.head_distill(a, 128, 1, 128, 0, 2, tau, None) == rcs.EINVAL
    assert L.head_distill(a, 128, 1, 128, 5, 2, 1.0, None) == rcs.EINVAL
    for tau in (1e-39, 1e20):  # 1 / tau, or its square, is out of float32's range
        assert L.head_distill(a, 128, 1, 128, 0, 2, tau, None) == rcs.EINVAL
    big = ctypes.byref(_args(scale=1e38))  # its product with the temperature is
    assert L.head_distill(big, 128, 1, 128, 0, 2, 10.0, None) == rcs.EINVAL
    e = lambda **m: L.embed_grad(*(dict(  # noqa: E731
        rows=256, rs=16, rt=0, count=4, tokens=128, it=1, grad=512, gs=16, gt=0, vocab=8, dim=16,
        scale=1.0, ws=4096, bytes=1 << 20, stream=None) | m).values())
    for bad in ({"rt": 4}, {"gt": -1}, {"it": 7}, {"scale": math.nan}, {"rs": 15}, {"gs": 8},
                {"count": -1}, {"vocab": 0}, {"rows": 258}, {"rows": None}, {"tokens": 129},
                {"grad": 514}, {"grad": None}):
        assert e(**bad) == rcs.EINVAL, bad


def test_binding_refuses_host_tensors():
    h, w, t = torch.zeros(4, 8), torch.zeros(16, 8), torch.zeros(4, dtype=torch.long)
    with pytest.raises(TypeError, match="CUDA"):
        rcs.head_loss(h, w, t)
    with pytest.raises(TypeError, match="CUDA"):
        rcs.head_distill(h, w, t.view(4, 1), torch.zeros(4, 1))
    with pytest.raises(TypeError, match="CUDA"):
        rcs.embed_grad(h, t, w)


@gpu
def test_binding_refuses():
    h, w, t = data(6, 40, 16, BF16)
    ok = dict(grad_hidden=torch.empty_like(h), grad_weight=torch.empty_like(w))
    for bad, kind in [
            (dict(hidden=h.float()), TypeError), (dict(hidden=h.double()), TypeError),
            (dict(weight=w.half()), TypeError), (dict(weight=w[:, :8]), ValueError),
            (dict(weight=w[:0]), ValueError), (dict(weight=w.t()), ValueError),
            (dict(weight=w.t().contiguous().t()), TypeError),
            (dict(hidden=h.t().contiguous().t()), TypeError),
            (dict(hidden=h[:1].expand(6, 16)), TypeError), (dict(hidden=h[:, :0]), ValueError),
            (dict(targets=t[:5]), ValueError), (dict(targets=t.float()), TypeError),
            (dict(targets=t.view(6, 1)), ValueError), (dict(targets=t.cpu()), TypeError),
            (dict(grad_hidden=h[:5]), ValueError), (dict(grad_hidden=h.float()), TypeError),
            (dict(grad_weight=w.double()), TypeError), (dict(grad_weight=w[:39]), ValueError),
            (dict(losses=torch.empty(6, 1, device="cuda")), ValueError),
            (dict(losses=torch.empty(6, device="cuda", dtype=BF16)), TypeError),
            (dict(losses=torch.empty(12, device="cuda")[::2]), TypeError),
            (dict(out=torch.empty(2, device="cuda")), ValueError),
            (dict(out=torch.empty(1, device="cuda", dtype=torch.float64)), TypeError),
            (dict(reduction="none"), ValueError), (dict(scale=math.inf), rcs.RcsError),
            # what is written overlaps what is read or written
            (dict(grad_hidden=h), rcs.RcsError), (dict(grad_weight=w), rcs.RcsError),
            (dict(grad_hidden=ok["grad_weight"][:6]), rcs.RcsError)]:
        args = dict(hidden=h, weight=w, targets=t) | ok | bad
        with pytest.raises(kind):
            rcs.head_loss(args.pop("hidden"), args.pop("weight"), args.pop("targets"), **args)
    index, logits = torch.zeros(6, 3, dtype=torch.long, device="cuda"), torch.zeros(6, 3).cuda()
    for bad, kind in [
            (dict(indices=index[:, :2].contiguous()), ValueError), (dict(indices=index.float()), TypeError),
            (dict(indices=index[:5], logits=logits[:5]), ValueError),
            (dict(indices=index.t().contiguous().t()), TypeError),
            (dict(logits=logits.double()), TypeError), (dict(temperature=0.0), rcs.RcsError),
            (dict(indices=index[:, :0], logits=logits[:, :0]), rcs.RcsError),
            (dict(indices=index.repeat(1, 400), logits=logits.repeat(1, 400)), rcs.RcsError)]:
        args = dict(indices=index, logits=logits) | bad
        with pytest.raises(kind):
            rcs.head_distill(h, w, args.pop("indices"), args.pop("logits"), **args)
    for bad, kind in [(dict(rows=h[:, :8]), ValueError), (dict(tokens=t[:5]), ValueError),
                      (dict(tokens=t.float()), TypeError), (dict(grad=w[:0]), ValueError),
                      (dict(grad=w.t()), ValueError), (dict(scale=math.nan), rcs.RcsError),
                      (dict(rows=w[:6]), rcs.RcsError), (dict(grad=w.double()), TypeError)]:
        args = dict(rows=h, tokens=t, grad=w) | bad
        with pytest.raises(kind):
            rcs.embed_grad(args.pop("rows"), args.pop("tokens"), args.pop("grad"), **args)


@gpu
def test_calls_refuse_short_workspaces():
    h, w, t = data(6, 40, 16, BF16)
    out = torch.empty(1, device="cuda")
    work = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    a = _args(hidden=h.data_ptr(), weight=w.data_ptr(), rows=6, vocab=40, loss=out.data_ptr(),
              workspace=work.data_ptr())
    need = rcs.lib().rcs_head_workspace(ctypes.byref(a), 0)
    call = lambda: rcs.lib().head_loss(ctypes.byref(a), t.data_ptr(), 1, -100, None)  # noqa: E731
    a.workspace_bytes = need - 1
    assert call() == rcs.ESIZE
    a.workspace_bytes, a.workspace = need, work.data_ptr() + 16
    assert call() == rcs.EINVAL
    a.workspace = h.data_ptr() // 256 * 256
    assert call() in (rcs.EINVAL, rcs.ESIZE)
    a.workspace = work.data_ptr()
    assert call() == rcs.OK
    torch.cuda.synchronize()


# -------------------------------------------------------------- cross entropy

# around one column, a product's fragment, a wave's and a block's tile, and a step of
# the sums; one size each of rows, vocabulary and width is not a multiple of anything
SIZES = [(1, 1, 1), (1, 2, 3), (2, 63, 8), (3, 64, 64), (5, 65, 7), (31, 127, 63), (63, 128, 65),
         (64, 129, 128), (65, 255, 16), (127, 256, 129), (128, 257, 192), (129, 1000, 100),
         (257, 515, 320), (300, 5003, 64), (1023, 700, 33)]


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,v,d", SIZES)
def test_loss(t, v, d, dtype):
    h, w, targets = data(t, v, d, dtype, seed=t)
    s = scale_of(dtype)
    r = run_loss(h, w, targets, scale=s)
    q, ok = one_hot(targets, v)
    check(h, w, q, ok, r, s, True)
    # without gradients
    r2 = run_loss(h, w, targets, grads=False, reduction="sum")
    check(h, w, q, ok, r2, 1.0, False)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [512, 500])
def test_loss_large_tiles(dtype, d):
    """Sizes at which each of the products is done in large tiles: whole rounds of
    them, a rest in splits, and splits of the sum over the vocabulary."""
    t, v = 2049, 66001
    h, w, targets = data(t, v, d, dtype, masked=0.01)
    s = scale_of(dtype) * 16
    r = run_loss(h, w, targets, scale=s)
    q, ok = one_hot(targets, v)
    check(h, w, q, ok, r, s, True)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,v,d", [(300, 20000, 64), (520, 33000, 64), (1100, 9000, 260)])
def test_loss_items_of_several_steps(t, v, d, dtype):
    h, w, targets = data(t, v, d, dtype)
    s = scale_of(dtype)
    r = run_loss(h, w, targets, scale=s)
    q, ok = one_hot(targets, v)
    check(h, w, q, ok, r, s, True)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("masked", [0.5, 0.99, 1.1])
def test_loss_masked_rows_take_no_part(masked, dtype):
    t, v, d = 200, 300, 72
    h, w, targets = data(t, v, d, dtype, masked=masked)
    h[targets == IGNORE] = math.nan
    h[targets == IGNORE, ::3] = math.inf
    s = scale_of(dtype)
    r = run_loss(h, w, targets, scale=s)
    q, ok = one_hot(targets, v)
    check(h, w, q, ok, r, s, True)
    assert (r[1][~ok] == 0).all() and (r[2][~ok] == 0).all()
    if masked > 1:  # no row at all: nothing is added, either
        assert r[0].item() == 0 and (r[3] == 0).all()
        gw = torch.full_like(w, 3.0)
        rcs.head_loss(h, w, targets, grad_weight=gw)
        assert (gw == 3.0).all()


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_loss_of_no_rows(dtype):
    h, w = torch.empty(0, 24, dtype=dtype, device="cuda"), torch.ones(50, 24, dtype=dtype).cuda()
    t = torch.empty(0, dtype=torch.long, device="cuda")
    r = run_loss(h, w, t)
    assert r[0].item() == 0 and (r[3] == 0).all()
    gw = torch.full_like(w, 3.0)
    assert rcs.head_loss(h, w, t, grad_weight=gw, reduction="sum").item() == 0
    assert (gw == 3.0).all()


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 61])
def test_loss_views_strides_and_index_types(d, dtype):
    t, v = 77, 333
    h, w, targets = data(t, v, d, dtype, view=True, masked=0.2)
    s = scale_of(dtype)
    q, ok = one_hot(targets, v)
    # gradients in the middle of larger arrays, whose other elements stay
    gh_all = torch.full((t, d + 5), 5.0, dtype=dtype, device="cuda")
    gw_all = torch.full((v + 2, d + 9), 5.0, dtype=dtype, device="cuda")
    gh, gw = gh_all[:, 2:2 + d], gw_all[1:-1, 3:3 + d]
    losses = torch.empty(t, device="cuda")
    loss = rcs.head_loss(h, w, targets.int(), grad_hidden=gh, grad_weight=gw, accumulate=False,
                         scale=s, losses=losses)
    check(h, w, q, ok, (loss, losses, gh, gw), s, True)
    gh.fill_(5.0), gw.fill_(5.0)
    assert (gh_all == 5).all() and (gw_all == 5).all()
    # leading dimensions
    h3 = h.contiguous().view(7, 11, d)
    l3 = torch.empty(7, 11, device="cuda")
    loss3 = rcs.head_loss(h3, w, targets.view(7, 11), grad_hidden=torch.empty_like(h3), losses=l3)
    assert torch.equal(l3.view(-1), losses) and torch.equal(loss3, loss)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gw_type", TYPES)
def test_loss_accumulates_in_any_type(dtype, gw_type):
    """As two micro-batches; the last one in groups of rows."""
    t, v, d = 300, 700, 100
    s = scale_of(dtype) / 2
    h, w, t1 = data(2 * t, v, d, dtype, seed=3)
    gw = torch.full(w.shape, 7.0, dtype=gw_type, device="cuda")
    rcs.head_loss(h[:t], w, t1[:t], grad_weight=gw, accumulate=False, scale=s)
    q, ok = one_hot(t1[:t], v)
    check(h[:t], w, q, ok, (None, None, None, gw), s, True)
    before = gw.clone()
    gh = torch.empty_like(h[t:])
    loss = rcs.head_loss(h[t:], w, t1[t:], grad_weight=gw, grad_hidden=gh, scale=s, max_bytes=1)
    q, ok = one_hot(t1[t:], v)
    check(h[t:], w, q, ok, (loss, None, gh, gw), s, True, before=before)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_loss_in_groups_of_rows(dtype):
    """More rows than max_bytes holds: the same results, to their roundings; and the
    rows with a loss end before the last group begins."""
    t, v, d = 700, 900, 40
    for masked in (0.0, 0.3, 0.9):
        h, w, targets = data(t, v, d, dtype, masked=masked)
        s = scale_of(dtype)
        q, ok = one_hot(targets, v)
        check(h, w, q, ok, run_loss(h, w, targets, scale=s, max_bytes=1), s, True)
        check(h, w, q, ok, run_loss(h, w, targets, scale=s, max_bytes=300 * 2 * 1024), s, True)
        r = run_loss(h, w, targets, grads=False, max_bytes=1)
        check(h, w, q, ok, r, 1.0, True)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_loss_large_logits(dtype):
    """Logits far above their targets' (in bfloat16, beyond what the exponentials
    relative to the target's logit can hold), and far below them."""
    t, v, d = 130, 1500, 64
    for spread in (20.0, 60.0):
        h, w, targets = data(t, v, d, dtype, spread=spread)
        z = h.double() @ w.double().t()
        targets[::3] = z[::3].argmax(1)
        targets[1::3] = z[1::3].argmin(1)
        s = scale_of(dtype)
        q, ok = one_hot(targets, v)
        r = run_loss(h, w, targets, scale=s)
        check(h, w, q, ok, r, s, True)
        assert r[1].max() > 64 * math.log(2)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_loss_bad_targets_and_values_give_nan(dtype):
    t, v, d = 40, 90, 32
    h, w, targets = data(t, v, d, dtype)
    good = run_loss(h, w, targets)
    for bad in (-1, v, 2 ** 40, -2 ** 40):
        x = targets.clone()
        x[7] = bad
        r = run_loss(h, w, x)
        rest = torch.arange(t, device="cuda") != 7
        assert torch.isnan(r[0]).all() and torch.isnan(r[1][7]) and torch.isnan(r[2][7]).all()
        assert torch.equal(r[1][rest], good[1][rest]) and torch.equal(r[2][rest], good[2][rest])
        assert torch.isnan(r[3]).any(0).all()
    x = h.clone()
    x[3, 5] = math.inf
    r = run_loss(x, w, targets)
    rest = torch.arange(t, device="cuda") != 3
    assert torch.isnan(r[1][3]) and torch.isfinite(r[1][rest]).all()
    x = w.clone()
    x[11, 2] = math.nan
    r = run_loss(h, x, targets)
    assert torch.isnan(r[1]).all() and torch.isnan(r[0]).all()


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_a_bad_target_in_large_tiles_leaves_other_rows(dtype):
    # a vocabulary of whole tiles: a row's place -1 is the last one of the row before
    t, v, d = 1030, 13312, 64
    h, w, targets = data(t, v, d, dtype)
    good = run_loss(h, w, targets, reduction="sum", scale=scale_of(dtype))
    for at in (0, 7, t - 1):
        x = targets.clone()
        x[at] = -1
        r = run_loss(h, w, x, reduction="sum", scale=scale_of(dtype))
        rest = torch.arange(t, device="cuda") != at
        assert torch.isnan(r[1][at]) and torch.isnan(r[2][at]).all()
        assert torch.equal(r[1][rest], good[1][rest]) and torch.equal(r[2][rest], good[2][rest])
        assert torch.isnan(r[3]).any(0).all()


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_loss_repeats_bit_for_bit(dtype):
    for t, v, d in ((700, 5003, 96), (2049, 33003, 256)):
        h, w, targets = data(t, v, d, dtype, masked=0.1)
        a, b = run_loss(h, w, targets), run_loss(h, w, targets)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@gpu
def test_gradients_against_differences():
    """The loss's change along a direction against the gradients. With steps of e the
    quotient is off by the losses' errors over e and by e^2 / 6 times the third
    derivative, at most 2 c^3 for logits that change by c; a product's size on each
    side is that of the tests above."""
    t, v, d, e = 60, 400, 48, 2.0 ** -7
    h, w, targets = data(t, v, d, F32, masked=0.2)
    index = torch.randint(0, v, (t, 6), device="cuda")
    logits = torch.randn(t, 6, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    dh, dw = (torch.randn(x.shape, generator=g, device="cuda") * 2.0 ** -3 for x in (h, w))

    def of(h, w, **more):
        return [rcs.head_loss(h, w, targets, **more),
                rcs.head_distill(h, w, index, logits, temperature=2.0, **more)]

    for k, tau in ((0, 1.0), (1, 2.0)):
        for a, b in ((dh, 0 * dw), (0 * dh, dw)):
            gh, gw = torch.empty_like(h), torch.zeros_like(w)
            more = dict(grad_hidden=gh, grad_weight=gw, accumulate=False)
            if k == 0:
                rcs.head_loss(h, w, targets, **more)
            else:
                rcs.head_distill(h, w, index, logits, temperature=2.0, **more)
            want = float((gh.double() * a).sum() + (gw.double() * b).sum())
            up, down = of(h + e * a, w + e * b)[k], of(h - e * a, w - e * b)[k]
            got = float((up.double() - down.double()) / (2 * e))
            c = float((a.double() @ w.double().t() + h.double() @ b.double().t()).abs().max())
            off = 2 * 2.0 ** -19 * tau * tau / e + e * e * c ** 3 / 3
            assert abs(got - want) <= off, (k, got, want, off)
            assert off < 0.05 * max(abs(want), 0.1)


# --------------------------------------------------------------- distillation

def teacher_data(t, v, k, seed=1, logits_type=F32, masked=0.0, index_type=torch.long):
    g = torch.Generator(device="cuda").manual_seed(seed)
    index = torch.rand(t, v, generator=g, device="cuda").topk(k, 1)[1]
    logits = (torch.randn(t, k, generator=g, device="cuda") * 2).to(logits_type)
    index[torch.rand(t, generator=g, device="cuda") < masked] = -1
    return index.to(index_type), logits


def run_distill(h, w, index, logits, tau, grads=True, **more):
    losses = torch.full((h.shape[0],), 7.0, device="cuda")
    gh = gw = None
    if grads:
        gh, gw = torch.full_like(h, 7.0), torch.full_like(w, 7.0)
        more = dict(grad_hidden=gh, grad_weight=gw, accumulate=False) | more
    loss = rcs.head_distill(h, w, index, logits, temperature=tau, losses=losses, **more)
    return loss, losses, gh, gw


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,v,d,k,tau", [
    (1, 5, 3, 1, 1.0), (3, 64, 64, 64, 2.0), (65, 300, 33, 5, 0.7), (130, 1111, 100, 17, 1.0),
    (70, 2000, 64, 1024, 3.0), (520, 33000, 64, 8, 2.0)])
def test_distill(t, v, d, k, tau, dtype):
    h, w, _ = data(t, v, d, dtype)
    index, logits = teacher_data(t, v, k)
    s = scale_of(dtype)
    q, ok, entropy = teacher(index, logits, v, tau)
    check(h, w, q, ok, run_distill(h, w, index, logits, tau, scale=s), s, True, tau, entropy)
    r = run_distill(h, w, index, logits, tau, grads=False, reduction="sum")
    check(h, w, q, ok, r, 1.0, False, tau, entropy)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("logits_type", TYPES)
def test_distill_entries_that_are_not_there(dtype, logits_type):
    """Negative indices, logits of -inf and of the type's lowest value, the same index
    several times, rows with nothing left, and what these rows hold."""
    t, v, d, k, tau = 90, 500, 40, 7, 2.0
    h, w, _ = data(t, v, d, dtype)
    index, logits = teacher_data(t, v, k, logits_type=logits_type, index_type=torch.int32)
    index[5:20, 2] = -1
    index[10:30, 0] = -7
    logits[15:40, 3] = -math.inf
    logits[20:25, 1] = torch.finfo(logits_type).min
    index[30:50, 4] = index[30:50, 1]
    index[35:45, 6] = index[35:45, 1]
    index[60:64] = -1
    logits[64:66] = -math.inf
    logits[60] = math.nan  # where no entry is
    h[60:66] = math.nan
    s = scale_of(dtype)
    q, ok, entropy = teacher(index, torch.where(index >= 0, logits.double(), torch.tensor(
        -math.inf, dtype=torch.float64, device="cuda")), v, tau)
    assert (~ok).sum() == 6
    for more in ({}, {"max_bytes": 1}):
        r = run_distill(h, w, index, logits, tau, scale=s, **more)
        check(h, w, q, ok, r, s, True, tau, entropy)
        assert (r[1][~ok] == 0).all() and (r[2][~ok] == 0).all()
    x = index.clone()
    x[2, 2] = v
    r = run_distill(h, w, x, logits, tau)
    assert torch.isnan(r[1][2]) and torch.isnan(r[2][2]).all() and torch.isnan(r[0]).all()
    assert torch.isfinite(r[1][3:60]).all() and torch.isfinite(r[2][3:60]).all()


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_distill_of_one_entry_is_cross_entropy(dtype):
    t, v, d = 100, 777, 64
    h, w, targets = data(t, v, d, dtype)
    s = scale_of(dtype)
    q, ok = one_hot(targets, v)
    r = run_distill(h, w, targets.view(-1, 1), torch.full((t, 1), 3.0, device="cuda"), 1.0,
                    scale=s)
    check(h, w, q, ok, r, s, True, entropy=torch.zeros(t, device="cuda"))


# ------------------------------------------------------------------ embedding

def check_embed(rows, tokens, grad, before, scale, touched_only=True):
    ok = (tokens >= 0) & (tokens < grad.shape[0])
    at, x = tokens[ok].long(), rows[ok].double() * scale
    want = before.double().index_add_(0, at, x)
    size = torch.zeros_like(want).index_add_(0, at, x.abs())
    n = torch.zeros(grad.shape[0], dtype=torch.float64, device="cuda").index_add_(
        0, at, torch.ones_like(at, dtype=torch.float64)).view(-1, 1)
    # one rounding of float32 a row of the token, the product with scale and the sum
    # with what was there; then the gradient's type
    err = size * (n + 3) * F + want.abs() * (2 * F + torch.finfo(grad.dtype).eps / 2) + \
        least(grad.dtype)
    near(grad, want, err, "grad")
    free = (n == 0).view(-1)
    assert torch.equal(grad[free], before[free])


@gpu
@pytest.mark.parametrize("rt", TYPES)
@pytest.mark.parametrize("gt", TYPES)
@pytest.mark.parametrize("t,v,d", [
    (1, 1, 1), (2, 3, 2), (7, 5, 3), (8, 70, 4), (9, 70, 5), (31, 64, 255), (33, 600, 256),
    (1023, 513, 321), (1025, 40, 260), (3078, 2 ** 18, 17), (8193, 300000, 64),
    (17001, 2 ** 20, 9)])
def test_embed(t, v, d, rt, gt):
    g = torch.Generator(device="cuda").manual_seed(t)
    rows = torch.randn(t, d, generator=g, device="cuda").to(rt)
    before = torch.randn(v, d, generator=g, device="cuda").to(gt)
    for kind in ("any", "one", "hot", "masked", "sorted"):
        tokens = torch.randint(0, v, (t,), generator=g, device="cuda")
        if kind == "one":
            tokens[:] = v - 1
        elif kind == "hot":
            tokens[torch.rand(t, generator=g, device="cuda") < 0.5] = v // 2
        elif kind == "masked":
            tokens[torch.rand(t, generator=g, device="cuda") < 0.5] = -100
            tokens[0] = v
            tokens[-1] = 2 ** 40
        elif kind == "sorted":
            tokens = tokens.sort(descending=True)[0]
        grad = before.clone()
        rcs.embed_grad(rows, tokens, grad, scale=0.5)
        check_embed(rows, tokens, grad, before, 0.5)
        again = before.clone()
        rcs.embed_grad(rows, tokens, again, scale=0.5)
        assert torch.equal(grad, again)


@gpu
def test_embed_views_strides_and_index_types():
    t, v, d = 500, 90, 50
    rows_all = torch.randn(t, d + 3, device="cuda").to(BF16)
    grad_all = torch.randn(v + 2, d + 1, device="cuda").to(F16)
    rows, grad = rows_all[:, 1:1 + d], grad_all[1:-1, 1:]
    before, whole = grad.clone(), grad_all.clone()
    tokens = torch.randint(-3, v + 3, (t,), device="cuda", dtype=torch.int32)
    rcs.embed_grad(rows, tokens, grad)
    check_embed(rows, tokens, grad, before, 1.0)
    grad.copy_(before)
    assert torch.equal(grad_all, whole)
    rows3 = rows.contiguous().view(5, 100, d)
    rcs.embed_grad(rows3, tokens.view(5, 100), grad, scale=-2.0)
    check_embed(rows, tokens, grad, before, -2.0)
    # no rows, and none that is met: nothing changes
    grad.copy_(before)
    rcs.embed_grad(rows[:0], tokens[:0], grad)
    rcs.embed_grad(rows, torch.full_like(tokens, -1), grad)
    assert torch.equal(grad, before)


# --------------------------------------------------------- streams and graphs

@gpu
def test_calls_on_another_stream():
    h, w, targets = data(300, 2000, 64, BF16)
    want = run_loss(h, w, targets)
    rows, tokens = torch.randn(500, 64, device="cuda"), torch.randint(0, 2000, (500,)).cuda()
    g_want = torch.zeros(2000, 64, device="cuda")
    rcs.embed_grad(rows, tokens, g_want)
    torch.cuda.synchronize()
    for raw in (False, True):
        s = torch.cuda.Stream()
        arg = s.cuda_stream if raw else s
        gh, gw, grad = torch.empty_like(h), torch.empty_like(w), torch.zeros_like(g_want)
        s.wait_stream(torch.cuda.current_stream())
        loss = rcs.head_loss(h, w, targets, grad_hidden=gh, grad_weight=gw, accumulate=False,
                             stream=arg)
        rcs.embed_grad(rows, tokens, grad, stream=arg)
        # work on the current stream, whose allocations must not touch the other's
        for _ in range(4):
            torch.empty(1 << 22, device="cuda").fill_(1e30)
        s.synchronize()
        assert torch.equal(loss, want[0]) and torch.equal(gh, want[2])
        assert torch.equal(gw, want[3]) and torch.equal(grad, g_want)


@gpu
def test_captured_calls_replay():
    """Two graphs, each of a loss, a distillation and an embedding's gradient, replayed
    in turn, together on two streams, and between eager calls."""
    t, v, d = 260, 3000, 96
    graphs = []
    for seed, dtype in ((1, BF16), (2, F32)):
        h, w, targets = data(t, v, d, dtype, seed=seed, masked=0.1)
        index, logits = teacher_data(t, v, 4, seed)
        bufs = [torch.zeros_like(h), torch.zeros_like(h), torch.zeros(v, d, device="cuda"),
                torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")]

        def step(h=h, w=w, targets=targets, index=index, logits=logits, b=bufs):
            rcs.head_loss(h, w, targets, grad_hidden=b[0], grad_weight=b[2], accumulate=False,
                          out=b[3])
            rcs.head_distill(h, w, index, logits, grad_hidden=b[1], grad_weight=b[2], out=b[4])
            rcs.embed_grad(b[0], targets, b[2])

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        graphs.append((graph, step, h, targets, bufs))
    streams = [torch.cuda.Stream() for _ in graphs]
    for turn in range(4):
        wants = []
        for graph, step, h, targets, bufs in graphs:  # new inputs in the same places
            h.copy_(torch.randn(h.shape, device="cuda"))
            targets.copy_(torch.randint(0, v, targets.shape, device="cuda"))
            step()
            wants.append([b.clone() for b in bufs])
            for b in bufs:
                b.fill_(9.0)
        torch.cuda.synchronize()
        for s, (graph, *_) in zip(streams, graphs):
            with torch.cuda.stream(s if turn % 2 else streams[0]):
                graph.replay()
        torch.cuda.synchronize()
        for want, (*_, bufs) in zip(wants, graphs):
            assert all(torch.equal(a, b) for a, b in zip(want, bufs)), turn


# --------------------------------------------- together, as a training run has them

def tied_steps(steps, state, dtype, resume=None):
    """A model of an embedding, a gain and the tied head: two micro-batches an update,
    both ends' gradients into one matrix, then the update over the list. Returns the
    list and the losses; `resume`: a step file's arrays after the first two updates."""
    v, d, t = 600, 80, 96
    g = torch.Generator(device="cuda").manual_seed(11)
    emb = (torch.randn(v, d, generator=g, device="cuda") * 0.1).to(dtype)
    gain = torch.ones(d, device="cuda", dtype=dtype)
    grads = [torch.zeros_like(emb), torch.zeros_like(gain)]
    opt = rcs.AdamWList([emb, gain], grads, state_bits=state, wd=[0.01, 0.0])
    losses = []
    if resume is not None:
        opt.import_state(*resume)
    for step in range(1, steps + 1):
        for micro in range(2):
            g.manual_seed(100 * step + micro)
            tokens = torch.randint(0, v, (t + 1,), generator=g, device="cuda")
            if resume is not None and step <= 2:
                continue
            x = emb[tokens[:-1]]
            gh = torch.empty_like(x)
            losses.append(rcs.head_loss(x * gain, emb, tokens[1:], grad_hidden=gh,
                                        grad_weight=grads[0], scale=0.5).clone())
            grads[1] += (gh * x).sum(0)
            rcs.embed_grad(gh * gain, tokens[:-1], grads[0])
        if resume is not None and step <= 2:
            continue
        if step == 1:
            first = [x.clone() for x in grads]
        opt.step(step, lr=1e-2, clip=1.0)
        torch._foreach_zero_(grads)
        if step == 2:
            mid = [x.clone() for x in opt.payload()]
    return opt, losses, (None if resume is not None else (first, mid))


@gpu
@pytest.mark.parametrize("state,dtype", [(32, F32), (8, BF16)])
def test_a_tied_model_trains_and_resumes(state, dtype):
    opt, losses, (first, mid) = tied_steps(4, state, dtype)
    # the first update's gradients: those of the whole model, in 64 bits
    v, d, t = 600, 80, 96
    g = torch.Generator(device="cuda").manual_seed(11)
    emb = (torch.randn(v, d, generator=g, device="cuda") * 0.1).to(dtype).double()
    emb.requires_grad_()
    gain = torch.ones(d, device="cuda", dtype=torch.float64, requires_grad=True)
    for micro in range(2):
        g.manual_seed(100 + micro)
        tokens = torch.randint(0, v, (t + 1,), generator=g, device="cuda")
        z = (emb[tokens[:-1]] * gain) @ emb.t().contiguous()
        loss = torch.nn.functional.cross_entropy(z, tokens[1:])
        (0.5 * loss).backward()
        assert abs(losses[micro].item() - loss.item()) < 1e-5
    # about six roundings of the type on the way to each gradient, in the norm
    for got, want in zip(first, (emb.grad, gain.grad)):
        off = float((got.double() - want).norm() / want.norm())
        assert off < 6 * (2.0 ** -20 if dtype == F32 else torch.finfo(dtype).eps / 2), off
    # a run that is resumed after two updates repeats the other two bit for bit
    again, more, _ = tied_steps(4, state, dtype, resume=mid)
    assert all(torch.equal(a, b) for a, b in zip(losses[4:], more))
    assert all(torch.equal(a, b) for a, b in zip(opt.payload(), again.payload()))


@gpu
def test_a_tied_model_beside_autograd():
    """The calls around a body that torch differentiates: both ends' gradients in one
    matrix, and the body's."""
    b, n, v, d = 3, 50, 700, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    emb = torch.randn(v, d, generator=g, device="cuda") * 0.3
    mix = torch.randn(d, d, generator=g, device="cuda") * d ** -0.5
    tokens = torch.randint(0, v, (b, n), generator=g, device="cuda")
    targets = torch.randint(0, v, (b, n), generator=g, device="cuda")
    targets[1, 30:] = IGNORE

    def body(x, mix):
        return torch.tanh(x.view(-1, d) @ mix).view(x.shape)

    m = mix.clone().requires_grad_()
    emb_grad = torch.zeros_like(emb)
    x = torch.nn.functional.embedding(tokens, emb).requires_grad_()
    hidden = body(x, m)
    gh = torch.empty_like(hidden)
    loss = rcs.head_loss(hidden, emb, targets, grad_hidden=gh, grad_weight=emb_grad)
    hidden.backward(gh)
    rcs.embed_grad(x.grad, tokens, emb_grad)

    e, m64 = emb.double().requires_grad_(), mix.double().requires_grad_()
    z = body(torch.nn.functional.embedding(tokens, e), m64).view(-1, d) @ e.t()
    want = torch.nn.functional.cross_entropy(z, targets.view(-1))
    want.backward()
    assert abs(loss.item() - want.item()) < 1e-5
    # sums of at most 700 terms, a few roundings of float32 each, in the norm
    for got, ref in ((emb_grad, e.grad), (m.grad, m64.grad)):
        assert float((got.double() - ref).norm() / ref.norm()) < 800 * F


@gpu
def test_a_bad_target_leaves_the_weights():
    h, w, targets = data(64, 100, 32, F32)
    grad = torch.zeros_like(w)
    opt = rcs.AdamWList([w], [grad])
    before = w.clone()
    targets[3] = 100
    rcs.head_loss(h, w, targets, grad_weight=grad)
    opt.step(1, lr=1e-2, clip=1.0)
    assert torch.equal(w, before) and torch.isnan(torch.tensor(float(rcs.last_grad_norm())))


def test_tolerances_count_half_steps():
    assert unit(BF16) == 2.0 ** -8 and unit(F16) == 2.0 ** -11
    assert np.isclose(least(F16), np.float64(np.nextafter(np.float16(0), np.float16(1))) / 2)
