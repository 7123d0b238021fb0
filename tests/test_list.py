"""The update over a list of tensors (AdamWList and the rcs_list calls).

On the CPU: the refusals, and the 8-bit form's own properties on the reference
(tests/list_reference.py). On the GPU: every result against that reference, at
sizes around the vectors, blocks and chunks of the kernels, for each type of
weights and gradients, on views at odd offsets.

Tolerances. 32-bit moments and the weights beside them follow one float32
operation sequence, which numpy repeats: they are compared bit for bit, weights
of 16 bits after one rounding. 8-bit moments are compared code for code. Weights
beside 8-bit moments are evaluated more freely; WEIGHT_ULPS below counts their
roundings."""
import ctypes
import os

import numpy as np
import pytest
import torch
from torch.multiprocessing.reductions import StorageWeakRef

import list_reference as ref
import resumable_checkpoint_state_amd as rcs
from resumable_checkpoint_state_amd import tensor_list

gpu = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
# 0: no chunk at all; around one lane's 8 elements, a block of 128, two chunks of
# 512, several of them (CHUNK_SIZES: around one)
SIZES = [0, 1, 7, 8, 9, 127, 128, 129, 130, 1023, 1024, 1025, 2048, 5003]

# Steps of 2^-24 (half a unit in float32's last place, relative to the larger of
# the two terms) by which w * decay - m / (da * sqrt(v) + db), as
# adamw_clip_step_list gives the weight beside 8-bit moments, may be off
# weights64: w * decay 1; the denominator's da 1, the hardware's root 2 (a whole
# unit), their sum with db 1; the hardware's reciprocal 2; the difference 2 (it
# may be twice the larger term); and weights64 takes bc1 and bc2 rounded to
# float32, 1 and (under the root) 1/2. 10.5 in all.
WEIGHT_ULPS = 10.5


# --------------------------------------------------------------- the reference

@pytest.mark.parametrize("which", ["m", "v"])
def test_reference_roundtrip_is_exact(which):
    """decode(encode(decode(x))) == decode(x), and every value is a bfloat16."""
    rng = np.random.default_rng(1)
    for scale in (1e-30, 1e-12, 1.0, 3e38 / 8):
        x = rng.standard_normal(4000) * scale * np.exp(rng.normal(0, 4, 4000))
        x = np.clip(x, -3e38, 3e38).astype(np.float32)
        x[::17] = 0.0
        x = np.abs(x) if which == "v" else x
        for add in (None, rng.integers(0, 1 << 20, x.size)):
            y = ref.decode(*ref.encode(x, which, add), which, x.size)
            z = ref.decode(*ref.encode(y, which), which, x.size)
            assert (y.view(np.uint32) == z.view(np.uint32)).all()
            assert (y.view(np.uint32) & 0xFFFF == 0).all()


@pytest.mark.parametrize("which", ["m", "v"])
def test_reference_error_bounds(which):
    """The nearest value is within 2^-4 of x (3 mantissa bits), a randomly
    rounded one within 2^-3, its mean within what 2,000 draws allow; below the
    range m is within half of its smallest value."""
    rng = np.random.default_rng(2)
    x = np.exp(rng.normal(0, 2, 512)).astype(np.float32)
    e = np.repeat(ref.exponents(x, which), 128)
    least = 1.25 * 2.0 ** (e - 127.0 - (16 if which == "m" else 32))
    y = ref.decode(*ref.encode(x, which), which, x.size)
    inside = x >= least
    assert inside.mean() > 0.9
    assert (np.abs(y - x)[inside] <= x[inside] * 2.0 ** -4).all()
    if which == "m":
        assert (np.abs(y - x)[~inside] <= least[~inside] / 2).all()
    draws = np.stack([ref.decode(*ref.encode(x, which, ref.random_bits(3, t, 0, 512) >> 12), which,
                                 512) for t in range(1, 2001)]).astype(np.float64)
    assert (np.abs(draws - x)[:, inside] <= x[inside] * 2.0 ** -3).all()
    # standard error of a value between two grid points d apart: at most d/2 / sqrt(2000)
    bound = 6 * (x * 2.0 ** -3) / 2 / np.sqrt(2000)
    assert (np.abs(draws.mean(0) - x)[inside] <= bound[inside]).all()


def test_reference_v_is_zero_only_where_it_is_zero():
    x = np.array([0.0, 1e-44, 1e-38, 1e-30, 1e-20, 1.0] + [0.0] * 122, np.float32)
    y = ref.decode(*ref.encode(x, "v"), "v", x.size)
    assert ((y > 0) == (x > 0)).all()


# ----------------------------------------------------------------- the refusals

@pytest.fixture(scope="module")
def L():
    if not os.path.exists(rcs.LIB_PATH):
        rcs.build()
    return rcs.lib()


FAKE = 0x1000  # never followed: refused before any device check


def _row(**kw):
    d = dict(w=FAKE, g=FAKE + 0x10000, m=FAKE + 0x20000, v=FAKE + 0x30000, exps=FAKE + 0x40000,
             copy=None, n=16, wd=0.0, w_type=0, g_type=0, copy_type=0)
    return tensor_list._Tensor(*[{**d, **kw}[f] for f, _ in tensor_list._Tensor._fields_])


@pytest.mark.parametrize("change", [
    dict(n=-1), dict(n=(1 << 40) + 1), dict(w_type=3), dict(w_type=-1), dict(g_type=7),
    dict(wd=float("nan")), dict(wd=float("inf")), dict(n=0), dict(w=None), dict(w=FAKE + 2),
    dict(copy=FAKE + 0x50000, w_type=1, copy_type=1), dict(copy=FAKE + 0x50000, copy_type=0),
])
def test_create_refuses_bad_rows(L, change):
    h = ctypes.c_void_p()
    rows = (tensor_list._Tensor * 1)(_row(**change))
    assert L.rcs_list_create(rows, 1, 32, ctypes.byref(h)) == rcs.EINVAL
    assert not h


def test_create_refuses_bad_arguments(L):
    h = ctypes.c_void_p()
    rows = (tensor_list._Tensor * 1)(_row())
    assert L.rcs_list_create(rows, 1, 32, None) == rcs.EINVAL
    for args in ((None, 1, 32), (rows, 0, 32), (rows, -1, 32), (rows, 1, 16), (rows, 1, 0)):
        assert L.rcs_list_create(*args, ctypes.byref(h)) == rcs.EINVAL
    # more chunks than a launch's work-items can number
    many = (tensor_list._Tensor * 1)(_row(n=1 << 40))
    assert L.rcs_list_create(many, 1, 32, ctypes.byref(h)) == rcs.EINVAL


def test_null_lists_are_refused(L):
    assert L.rcs_list_destroy(None) == rcs.OK
    assert L.rcs_list_elements(None) == -1
    assert L.rcs_list_bind_grads(None, None, 0, None) == rcs.EINVAL
    assert L.grad_global_norm_list(None, 1.0, FAKE, None) == rcs.EINVAL
    assert L.adamw_clip_step_list(None, 1, 1e-3, 1.0, 1.0, 0.9, 0.999, 1e-8, 0, None,
                                  None) == rcs.EINVAL
    assert L.rcs_list_export(None, FAKE, 0, None, 0, None, 0, None) == rcs.EINVAL
    assert L.rcs_list_import(None, FAKE, 0, None, 0, None, 0, None) == rcs.EINVAL


def test_binding_refuses_before_the_device():
    a = torch.zeros(8)
    with pytest.raises(ValueError):
        rcs.AdamWList([], [])
    with pytest.raises(ValueError):
        rcs.AdamWList([a], [a], state_bits=16)
    with pytest.raises(ValueError):
        rcs.AdamWList([a], [a, a])
    with pytest.raises(ValueError):
        rcs.AdamWList([a], [a], wd=[0.1, 0.2])
    with pytest.raises(TypeError):
        rcs.AdamWList([a], [a])  # host memory


class _Binds:
    """A library whose rcs_list_bind_grads succeeds, on a stream that is being
    captured or not."""

    capturing = False

    def rcs_stream_capturing(self, stream):
        return int(self.capturing)

    def rcs_list_bind_grads(self, handle, ptrs, count, stream):
        return rcs.OK


def test_what_a_binding_keeps_alive(monkeypatch):
    """Until the replay of a captured binding the device has the gradients from
    before it, and at each replay again those of the call: both stay. An eager
    binding lets go of the ones it replaces, but not of a graph's."""
    stub = _Binds()
    monkeypatch.setattr(tensor_list, "lib", lambda: stub)
    monkeypatch.setattr(tensor_list, "_checked", lambda t, *args: t.detach())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    lst = rcs.AdamWList.__new__(rcs.AdamWList)
    lst._h, lst._captured = ctypes.c_void_p(1), []
    lst._params, lst._gtypes = [torch.zeros(8)], [F32]
    first, captured, later, last = (torch.zeros(8) for _ in range(4))
    held = {k: StorageWeakRef(x.untyped_storage()) for k, x in
            dict(first=first, captured=captured, later=later, last=last).items()}
    lst._grads = [first.detach()]
    stub.capturing = True
    lst.bind_grads([captured], stream=0)
    del first, captured
    assert not held["first"].expired() and not held["captured"].expired()
    stub.capturing = False
    lst.bind_grads([later], stream=0)
    del later
    assert held["first"].expired()
    assert not held["captured"].expired() and not held["later"].expired()
    lst.bind_grads([last], stream=0)
    assert held["later"].expired() and not held["captured"].expired()
    lst._h = None  # nothing to destroy


# --------------------------------------------------------------------- the GPU

@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    rcs.lib()
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def host(t):
    return t.detach().float().cpu().numpy()


def raw(t):
    """The bits of a tensor, as integers on the host."""
    return t.detach().view({4: torch.int32, 2: torch.int16, 1: torch.uint8, 8: torch.int64}[
        t.element_size()]).cpu().numpy()


class Case:
    """A list on views into flat buffers with gaps between them, and copies of
    everything on the host."""

    def __init__(self, dev, sizes, w=F32, g=F32, bits=32, copy=None, gap=1, seed=1, sigma=0.1,
                 wd=None, state=True):
        self.dev, self.sizes, self.bits, self.seed = dev, list(sizes), bits, seed
        gen = torch.Generator(device=dev).manual_seed(seed)
        total = sum(sizes) + gap * (len(sizes) + 1)

        def flat(dtype, s, shift=0.0):
            return (torch.randn(total, generator=gen, device=dev) * s + shift).to(dtype)

        self.fw, self.fg = flat(w, 0.5, 0.25), flat(g, sigma)
        self.fc = self.fw.to(copy) if copy else None
        self.at = []
        p = gap
        for n in sizes:
            self.at.append(p)
            p += n + gap
        self.w, self.g = self.cut(self.fw), self.cut(self.fg)
        self.c = self.cut(self.fc) if copy else None
        self.wd = [0.01 * (k % 3) for k in range(len(sizes))] if wd is None else wd
        self.list = rcs.AdamWList(self.w, self.g, state_bits=bits, wd=self.wd, copies=self.c,
                                  seed=77)
        self.n = sum(sizes)
        if state:
            v = (torch.randn(self.n, generator=gen, device=dev) * 2).exp() * sigma * sigma
            m = torch.randn(self.n, generator=gen, device=dev) * v.sqrt()
            m[::5] = 0
            self.list.import_state(m=m, v=v)
        torch.cuda.synchronize()

    def cut(self, flat):
        return [flat[a:a + n] for a, n in zip(self.at, self.sizes)]

    def moments(self):
        m, v = (torch.full((self.n,), -7.0, device=self.dev) for _ in range(2))
        self.list.export_state(m=m, v=v)
        torch.cuda.synchronize()
        return host(m), host(v)

    def parts(self, flat):
        return np.split(flat, np.cumsum(self.sizes)[:-1])

    def gaps(self, flat):
        """The elements of a flat buffer that belong to no tensor."""
        mask = np.ones(flat.numel(), bool)
        for a, n in zip(self.at, self.sizes):
            mask[a:a + n] = False
        return raw(flat)[mask]


def norm_of(case, scale=1.0, without=()):
    f = np.float32(scale)
    return np.sqrt(sum(((host(g) * f).astype(np.float64) ** 2).sum()
                       for k, g in enumerate(case.g) if k not in without))


@gpu
@pytest.mark.parametrize("g", [F32, BF16, F16])
@pytest.mark.parametrize("sizes", [SIZES, [1], [3], [1 << 20, 5, 300_001], [4096] * 300])
def test_norm(dev, g, sizes):
    """Against a 64-bit sum: n roundings of 2^-53 at most, doubled for the
    reference's own."""
    case = Case(dev, sizes, g=g, gap=3, state=False)
    for scale in (1.0, 1.0 / 3):
        got = float(case.list.grad_norm(grad_scale=scale).cpu())
        want = norm_of(case, scale)
        assert abs(got - want) <= 2 * case.n * 2.0 ** -53 * want
    assert float(rcs.last_grad_norm().cpu()) == got
    pinned = torch.zeros(1, dtype=torch.float64, pin_memory=True)
    case.list.grad_norm(out=pinned, grad_scale=1.0 / 3)
    torch.cuda.synchronize()
    assert float(pinned) == got


def check_step(case, t, lr, clip, scale=1.0, b1=0.9, b2=0.999, eps=1e-8, without=()):
    """One update of case's list against the reference."""
    w0 = [host(x) for x in case.w]
    m0, v0 = (case.parts(x) for x in case.moments())
    gaps = [case.gaps(x) for x in (case.fw, case.fc) if x is not None]
    out = torch.full((1,), -1.0, dtype=torch.float64, device=case.dev)
    case.list.step(t, lr, clip, grad_scale=scale, beta1=b1, beta2=b2, eps=eps, norm_out=out)
    torch.cuda.synchronize()
    norm = float(out.cpu())
    want = norm_of(case, scale, without)
    assert abs(norm - want) <= 2 * max(case.n, 16) * 2.0 ** -53 * want
    m1, v1 = (case.parts(x) for x in case.moments())
    codes = None
    if case.bits == 8:
        blocks = np.cumsum([-(-n // 128) for n in case.sizes])[:-1]
        codes = [np.split(raw(x), blocks * 128) for x in (case.list.m, case.list.v)]
        exps = np.split(raw(case.list.exps), blocks)
    first = 0
    for k, n in enumerate(case.sizes):
        dtype = case.w[k].dtype
        if k in without:
            assert (host(case.w[k]) == w0[k]).all()
            assert (m1[k] == m0[k]).all() and (v1[k] == v0[k]).all()
            first += n
            continue
        args = (w0[k], host(case.g[k]), m0[k], v0[k], norm, t, lr, case.wd[k], clip, scale, b1,
                b2, eps)
        rw, rm, rv = ref.update32(*args)
        if case.bits == 32:
            assert (rm.view(np.uint32) == m1[k].view(np.uint32)).all(), ("m", k, n)
            assert (rv.view(np.uint32) == v1[k].view(np.uint32)).all(), ("v", k, n)
            assert (raw(torch.from_numpy(rw).to(dtype)) == raw(case.w[k])).all(), ("w", k, n)
        else:
            bits = ref.random_bits(77, t, first, n)
            for which, x, add in (("m", rm, bits & np.uint64(0xFFFFF)),
                                  ("v", rv, bits >> np.uint64(12))):
                c, e = ref.encode(x, which, add)
                assert (exps[k][:, "mv".index(which)] == e).all(), (which, k, n)
                assert (codes["mv".index(which)][k] == c).all(), (which, k, n)
            w64, size = ref.weights64(w0[k], rm, rv, t, lr, case.wd[k], b1, b2, eps)
            # and half a step of the weights' own type
            tol = WEIGHT_ULPS * 2.0 ** -24 * size
            half = torch.finfo(dtype).eps / 2
            tiny = float(torch.finfo(dtype).smallest_normal) * half
            if dtype != F32:
                tol = tol + np.abs(w64) * half + tiny
            got = host(case.w[k])
            assert (np.abs(got - w64) <= tol).all(), (
                "w", k, n, np.max(np.abs(got - w64) / tol))
        if case.c is not None:
            assert (raw(case.w[k].to(case.c[k].dtype)) == raw(case.c[k])).all()
        first += n
    for before, x in zip(gaps, [x for x in (case.fw, case.fc) if x is not None]):
        assert (before == case.gaps(x)).all()  # nothing beside the tensors
    return norm


TYPES = [(w, g) for w in (F32, BF16, F16) for g in (F32, BF16, F16)]


@gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("w,g", TYPES)
@pytest.mark.parametrize("gap", [0, 1, 8])
def test_step(dev, bits, w, g, gap):
    """Every type, sizes around the kernels' vectors, blocks and chunks, views
    at odd and even offsets; clipped and not, betas and eps of one's own."""
    case = Case(dev, SIZES, w=w, g=g, bits=bits, gap=gap)
    assert check_step(case, 1, 3e-3, 1.0) > 1.0
    check_step(case, 2, 3e-3, float("inf"), scale=0.25)
    check_step(case, 1000, 1e-2, 0.5, b1=0.8, b2=0.95, eps=1e-6)


# Around the kernels' chunk, 512 elements, and around one and a fraction: with
# 32-bit moments the chunks of a tensor of more than 512 begin where its m lies on
# a 256-byte boundary, so what matters there is where the tensor begins in the
# list, too. The single elements move what follows them.
CHUNK_SIZES = [511, 512, 513, 1, 512, 513, 575, 1, 576, 577, 62, 639, 640, 641, 3, 1023, 1,
               1087, 1088, 1089, 1536, 1537]


@gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("w,g", [(F32, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("gap", [0, 1])
def test_step_around_a_chunk(dev, bits, w, g, gap):
    case = Case(dev, CHUNK_SIZES, w=w, g=g, bits=bits, gap=gap)
    check_step(case, 3, 3e-3, 1.0)
    check_step(case, 4, 3e-3, float("inf"))
    n = case.n
    got = [torch.full((n + 1,), 3.0, device=dev) for _ in range(3)]
    case.list.export_state(*(x[:n] for x in got))
    m, v = case.moments()
    assert (host(got[0])[:n] == host(torch.cat(case.w))).all()
    assert (host(got[1])[:n] == m).all() and (host(got[2])[:n] == v).all()
    assert all(float(x[n].cpu()) == 3.0 for x in got)
    other = Case(dev, CHUNK_SIZES, w=w, g=g, bits=bits, gap=gap, seed=2)
    gaps = other.gaps(other.fw)
    other.list.import_state(*(x[:n] for x in got))
    torch.cuda.synchronize()
    assert (raw(torch.cat(other.w)) == raw(torch.cat(case.w))).all()
    # the values, that is: where an update rounded a block's largest down to the
    # next power of two, and for a zero, the codes of the same values differ
    om, ov = other.moments()
    assert (om.view(np.uint32) == m.view(np.uint32)).all()
    assert (ov.view(np.uint32) == v.view(np.uint32)).all()
    assert (other.gaps(other.fw) == gaps).all()


@gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("copy", [BF16, F16])
def test_step_writes_the_copies(dev, bits, copy):
    case = Case(dev, SIZES, bits=bits, copy=copy, g=BF16)
    case.list.import_state(w=torch.cat(case.w))
    check_step(case, 3, 1e-3, 1.0)


@gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("n", [3 * (1 << 20) + 5, 9_000_001])
def test_step_of_many_chunks(dev, bits, n):
    """Both launch forms: the final reduction in the update (up to 8,388,608
    elements) and before it."""
    case = Case(dev, [n - 1000, 1, 999], bits=bits, g=BF16, sigma=1e-3)
    check_step(case, 5, 1e-3, 1.0)


@gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_many_small_tensors_of_mixed_types(dev, bits):
    """700 tensors (three batches of gradient pointers), each of its own type."""
    types = TYPES * 78
    gen = torch.Generator(device=dev).manual_seed(3)
    sizes = [1 + (37 * k) % 300 for k in range(len(types))]
    ws = [torch.randn(n, generator=gen, device=dev).to(t[0]) for n, t in zip(sizes, types)]
    gs = [torch.randn(n, generator=gen, device=dev).to(t[1]) for n, t in zip(sizes, types)]
    lst = rcs.AdamWList(ws, gs, state_bits=bits, wd=0.1, seed=1)
    other = [(g.float() * 2).to(g.dtype) for g in gs]
    lst.bind_grads(other)
    w0 = [host(w) for w in ws]
    norm = float(lst.grad_norm().cpu())
    want = np.sqrt(sum((host(g).astype(np.float64) ** 2).sum() for g in other))
    assert abs(norm - want) <= 1e-11 * want
    lst.step(1, 1e-2, 1.0)
    torch.cuda.synchronize()
    for k, w in enumerate(ws):
        z = np.zeros(sizes[k], np.float32)
        rw, rm, rv = ref.update32(w0[k], host(other[k]), z, z, norm, 1, 1e-2, 0.1, 1.0)
        w64, size = ref.weights64(w0[k], rm, rv, 1, 1e-2, 0.1)
        half = torch.finfo(w.dtype).eps / 2
        tiny = float(torch.finfo(w.dtype).smallest_normal) * half
        tol = WEIGHT_ULPS * 2.0 ** -24 * size + (np.abs(w64) * half + tiny) * (w.dtype != F32)
        assert (np.abs(host(w) - w64) <= tol).all(), k


@gpu
@pytest.mark.parametrize("n", [262_144, 9_000_001])
def test_step_is_the_flat_update(dev, n):
    """float32 throughout: the list's update and adamw_clip_step give the same
    bits when neither clips (the sums' orders differ, so a clip factor could)."""
    case = Case(dev, [n // 2, n - n // 2], gap=0, wd=[0.02, 0.02])
    w, g = case.fw.clone(), case.fg.clone()
    m, v = (x.clone() for x in (case.list.m, case.list.v))
    for t in (4, 5):
        case.list.step(t, 1e-3, float("inf"), grad_scale=0.5)
        rcs.adamw_clip_step_accum(w, g, m, v, t, 1e-3, 0.02, float("inf"), 0.5)
    torch.cuda.synchronize()
    for a, b in ((case.fw, w), (case.list.m, m), (case.list.v, v)):
        assert (raw(a) == raw(b)).all()


@gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("n", [5000, 8_400_000])
def test_a_norm_that_is_not_finite_changes_nothing(dev, bits, bad, n):
    case = Case(dev, [n, 77], bits=bits, copy=BF16)
    case.g[1][5] = bad
    before = [raw(x).copy() for x in (case.fw, case.fc, case.list.m, case.list.v)]
    out = torch.zeros(1, dtype=torch.float64, device=dev)
    case.list.step(1, 1e-3, 1.0, norm_out=out)
    torch.cuda.synchronize()
    assert not np.isfinite(float(out.cpu()))
    for x, b in zip((case.fw, case.fc, case.list.m, case.list.v), before):
        assert (raw(x) == b).all()


@gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_tensors_without_a_gradient_are_left_alone(dev, bits):
    """None adds nothing to the norm and leaves weights, moments and copy as
    they are, whichever tensor it is, until a gradient is bound."""
    case = Case(dev, [2000, 300, 1500], bits=bits)
    grads = case.g
    for without in ((0,), (1, 2), (0, 2)):
        case.list.bind_grads([None if k in without else g for k, g in enumerate(grads)])
        check_step(case, 2, 1e-3, 1.0, without=without)
    case.list.bind_grads([None] * 3)
    assert float(case.list.grad_norm().cpu()) == 0.0
    case.list.step(3, 1e-3, 1.0)
    case.list.bind_grads(grads)
    check_step(case, 4, 1e-3, 1.0)


@gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_zero_gradients(dev, bits):
    """A zero norm does not clip; zero moments stay zero and the weights decay."""
    case = Case(dev, [1030], bits=bits, state=False, wd=[0.1])
    case.g[0].zero_()
    check_step(case, 1, 1e-2, 1.0)
    m, v = case.moments()
    assert not m.any() and not v.any()


@gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("lr", [0.0, 1e-44, 1e-12, -1e-3, 1e6, 1e20])
def test_extreme_learning_rates(dev, bits, lr):
    case = Case(dev, [2000, 515], bits=bits)
    case.g[0][::7] = 0
    check_step(case, 1, lr, 1.0)
    check_step(case, 50, lr, float("inf"), eps=1e-16)
    if bits == 8:  # nothing would be left of eps
        with pytest.raises(rcs.RcsError):
            case.list.step(1, 1e30, 1.0)


@gpu
@pytest.mark.parametrize("t", [1, 50])
@pytest.mark.parametrize("eps", [1e-12, 1e-15, 1e-20, 1e-30])
@pytest.mark.parametrize("w,g", [(F32, F32), (BF16, BF16)])
def test_second_moments_below_the_normal_floats(dev, w, g, eps, t):
    """Gradients whose squares are subnormal floats or nothing, beside an eps
    that the square root of such a float (up to 1e-19) stands out from: with
    weights of zero the step is all there is to see."""
    case = Case(dev, [4096, 515], w=w, g=g, bits=8, state=False, wd=[0.0, 0.0])
    for x, y in zip(case.g, case.w):
        tiny = torch.logspace(-22.5, -12, x.numel(), device=dev, dtype=torch.float64)
        tiny[::3] *= -1
        x.copy_(tiny)
        y[::2] = 0
    check_step(case, t, 1e-3, 1.0, eps=eps)


# One rounding more than WEIGHT_ULPS: where the denominator does not fit the
# floats whose reciprocal is a normal one, the quotient is rounded before it is
# scaled (by a power of two).
SCALED_ULPS = WEIGHT_ULPS + 1


@gpu
@pytest.mark.parametrize("w,g", [(F32, F32), (BF16, BF16)])
@pytest.mark.parametrize("lr,eps", [(1e-18, 1e-8), (1e-20, 1e-8), (-1e-30, 1e-8), (1e-38, 1e-8),
                                    (1e-42, 1e-8), (1e-30, 1e-30), (1e-3, 1e37), (1e-8, 1e33)])
def test_denominators_beyond_the_normal_reciprocals(dev, w, g, lr, eps):
    """lr so small, or eps so large, that (sqrt(v / bc2) + eps) bc1 / lr passes
    2^126, whose reciprocal is no normal float. Weights of zero show the step
    alone; where it is subnormal, one unit of 2^-149 for its two roundings."""
    case = Case(dev, [4096, 515], w=w, g=g, bits=8, state=False, wd=[0.0, 0.0])
    for x, y in zip(case.g, case.w):
        wide = torch.logspace(-10, 18.5, x.numel(), device=dev, dtype=torch.float64)
        wide[::3] *= -1
        x.copy_(wide)
        y.zero_()
    norm = torch.zeros(1, dtype=torch.float64, device=dev)
    case.list.step(1, lr, float("inf"), eps=eps, norm_out=norm)
    torch.cuda.synchronize()
    for x, y in zip(case.g, case.w):
        z = np.zeros(x.numel(), np.float32)
        _, rm, rv = ref.update32(z, host(x), z, z, float(norm.cpu()), 1, lr, 0.0, float("inf"),
                                 eps=eps)
        w64, size = ref.weights64(z, rm, rv, 1, lr, 0.0, eps=eps)
        assert (np.abs(w64) > 0).all()
        tol = SCALED_ULPS * 2.0 ** -24 * size + 2.0 ** -149
        if w != F32:
            tol = tol + np.abs(w64) * 2.0 ** -8 + 2.0 ** -134
        got = host(y).astype(np.float64)
        assert (np.abs(got - w64) <= tol).all(), np.max(np.abs(got - w64) / tol)


@gpu
@pytest.mark.parametrize("w,g", TYPES)
def test_step_with_a_small_eps_or_lr(dev, w, g):
    """The kernels of the weight's other form, for each pair of types and both
    launch forms, on views at odd offsets, copies included."""
    for sizes in (SIZES, [8_400_001, 515]):
        case = Case(dev, sizes, w=w, g=g, bits=8, gap=1, copy=F16 if w == F32 else None)
        if case.c is not None:
            case.list.import_state(w=torch.cat(case.w))
        check_step(case, 1, 3e-3, 1.0, eps=1e-20)
        check_step(case, 2, 1e-19, 1.0)


@gpu
def test_infinite_moments(dev):
    """An infinite 8-bit moment stays infinite, alone in its block; a beta of
    zero forgets it."""
    case = Case(dev, [256], bits=8, state=False)
    v = torch.ones(256, device=dev)
    m = torch.ones(256, device=dev)
    v[5], m[7], m[8] = float("inf"), float("inf"), float("-inf")
    case.list.import_state(m=m, v=v)
    case.list.step(1, 1e-3, 1.0)
    gm, gv = case.moments()
    assert gv[5] == np.inf and gm[7] == np.inf and gm[8] == -np.inf
    assert np.isfinite(np.delete(gm, [7, 8])).all() and np.isfinite(np.delete(gv, 5)).all()
    case.list.step(2, 1e-3, 1.0, beta1=0.0, beta2=0.0)
    gm, gv = case.moments()
    assert np.isfinite(gm).all() and np.isfinite(gv).all()


@gpu
def test_extreme_moments(dev):
    """Gradients from float32's smallest to its largest whose squares under- or
    overflow: the codes still follow the float32 sequence."""
    case = Case(dev, [4096], bits=8, state=False)
    g = torch.logspace(-44, 18, 4096, device=dev, dtype=torch.float64).float()
    g[::3] *= -1
    g[100:140] = 0
    case.g[0].copy_(g)
    check_step(case, 1, 1e-3, float("inf"))
    check_step(case, 2, 1e-3, 1.0)
    case.g[0].copy_(g * 1e19)  # squares beyond the largest float: held as infinity
    check_step(case, 3, 1e-3, float("inf"), scale=1.0)
    m, v = case.moments()
    assert np.isinf(v).any()


@gpu
@pytest.mark.parametrize("sizes", [SIZES, [300_001, 128]])
@pytest.mark.parametrize("w", [F32, BF16, F16])
@pytest.mark.parametrize("flat", [F32, BF16])
def test_import_and_export(dev, sizes, w, flat):
    """8-bit moments are the nearest values they can hold, export gives them
    exactly in either type and leaves what lies beside its arrays alone, and
    importing them again changes nothing."""
    case = Case(dev, sizes, w=w, bits=8, copy=BF16 if w == F32 else None)
    n = case.n
    gen = torch.Generator(device=dev).manual_seed(9)
    wi = torch.randn(n, generator=gen, device=dev).to(flat)
    mi = (torch.randn(n, generator=gen, device=dev) *
          (torch.randn(n, generator=gen, device=dev) * 4).exp()).to(flat)
    vi = mi.square()
    vi[::50] = -1.0
    case.list.import_state(w=wi, m=mi, v=vi)
    buf = torch.full((3 * n + 4,), 3.0, device=dev, dtype=flat)
    out = [buf[1 + k * (n + 1):1 + k * (n + 1) + n] for k in range(3)]
    case.list.export_state(*out)
    torch.cuda.synchronize()
    assert (host(buf)[0::n + 1] == 3.0).all()
    assert (raw(out[0]) == raw(wi.to(w).to(flat))).all()
    if case.c is not None:
        assert (raw(torch.cat(case.c)) == raw(wi.to(w).to(BF16))).all()
    v_in = np.maximum(host(vi), 0)
    for which, x, y in (("m", host(mi), out[1]), ("v", v_in, out[2])):
        for a, b in zip(case.parts(x), case.parts(host(y))):
            if a.size:
                want = ref.decode(*ref.encode(a, which), which, a.size)
                assert (want.view(np.uint32) == b.view(np.uint32)).all()
    case.list.import_state(m=out[1], v=out[2])
    again = [torch.empty(n, device=dev, dtype=flat) for _ in range(2)]
    case.list.export_state(m=again[0], v=again[1])
    torch.cuda.synchronize()
    assert (raw(again[0]) == raw(out[1])).all() and (raw(again[1]) == raw(out[2])).all()


@gpu
def test_import_of_what_is_not_finite(dev):
    """Infinities and NaN are held as infinities of their sign, and only the
    block they are in loses its small values."""
    case = Case(dev, [300], bits=8, state=False)
    m = torch.ones(300, device=dev)
    v = torch.ones(300, device=dev)
    m[3], m[4], v[5], v[6], v[7] = float("-inf"), float("nan"), float("inf"), float("nan"), -3.0
    case.list.import_state(m=m, v=v)
    gm, gv = case.moments()
    assert gm[3] == -np.inf and gm[4] == np.inf and (gv[5:7] == np.inf).all() and gv[7] == 0
    assert np.isfinite(np.delete(gm, [3, 4])).all() and (gm[128:] == 1).all()
    assert (gv[128:] == 1).all()


@gpu
def test_import_of_the_largest_floats(dev):
    """What rounds beyond the largest float becomes an infinity, as the
    reference has it; half a step below does not."""
    m = torch.full((128,), 3.0e38, device=dev)
    m[1], m[2], m[3] = 3.4e38, -3.4e38, 3.25e38
    v = m.abs()
    case = Case(dev, [128], bits=8, state=False)
    case.list.import_state(m=m, v=v)
    for got, x, which in zip(case.moments(), (host(m), host(v)), "mv"):
        want = ref.decode(*ref.encode(x, which), which, 128)
        assert (got.view(np.uint32) == want.view(np.uint32)).all()
        assert np.isinf(got[1]) and np.isfinite(got[0])


@gpu
def test_many_chunks_of_unaligned_tensors(dev):
    """Whole windows of chunks, both with loads kept in the cache and without,
    on tensors off every line boundary; export and import of the same."""
    for n, w in ((1_500_007, BF16), (1_500_007, F32)):
        case = Case(dev, [n, 3, n], bits=8, w=w, g=BF16, gap=3, copy=BF16 if w == F32 else None,
                    sigma=1e-3)
        if case.c is not None:
            case.list.import_state(w=torch.cat([x.float() for x in case.w]))
        check_step(case, 7, 1e-3, 1.0)
    case = Case(dev, [n, 3, n], bits=32, w=BF16, g=BF16, gap=5, sigma=1e-3)
    check_step(case, 7, 1e-3, 1.0)


@gpu
def test_import_and_export_of_32_bits(dev):
    case = Case(dev, SIZES, w=BF16, bits=32, state=False)
    m, v, w = (torch.randn(case.n + 1, device=dev)[1:] for _ in range(3))
    case.list.import_state(m=m)
    case.list.import_state(w=w, v=v)
    out = [torch.empty(case.n, device=dev) for _ in range(3)]
    case.list.export_state(*out)
    torch.cuda.synchronize()
    assert (raw(out[0]) == raw(w.to(BF16).float())).all()
    assert (raw(out[1]) == raw(m)).all() and (raw(out[2]) == raw(v)).all()
    assert (raw(case.list.m) == raw(m)).all()


@gpu
@pytest.mark.parametrize("async_write", [False, True])
@pytest.mark.parametrize("bits,w", [(8, BF16), (8, F32), (32, BF16)])
def test_a_run_continues_bit_identically_from_its_step_file(dev, tmp_path, bits, w, async_write):
    """The operators together, as a training loop uses them: gradients that
    follow the weights, steps, a step file through the checkpointer, and a
    fresh list that resumes from it, against the run that never stopped."""
    sizes = [1000, 37, 4096, 129]

    def grads_of(case, t):
        gen = torch.Generator(device=dev).manual_seed(100 + t)
        for p, g in zip(case.w, case.g):
            noise = torch.randn(p.numel(), generator=gen, device=dev)
            g.copy_((p.float() * 0.3 + 0.1 * noise).to(g.dtype))

    def train(case, a, b, ck):
        for t in range(a, b + 1):
            grads_of(case, t)
            case.list.step(t, 1e-2, 1.0)
            if ck is not None:
                assert not ck.after_step(t, case.list)

    def make(seed):
        return Case(dev, sizes, w=w, g=BF16, bits=bits, copy=F16 if w == F32 else None, seed=seed,
                    state=False)

    straight = make(5)
    ck = rcs.StepFileCheckpointer(tmp_path, straight.n, every=7, keep=1, install_signals=False,
                                  async_write=async_write)
    train(straight, 1, 7, ck)
    ck.flush()
    assert os.path.getsize(tmp_path / "step_000007.bin") == 8 + 12 * straight.n
    resumed = make(6)  # other weights: all of them have to come from the file
    assert ck.resume(resumed.list) == 7
    train(straight, 8, 12, None)
    train(resumed, 8, 12, None)
    torch.cuda.synchronize()
    for a, b in zip(straight.w + (straight.c or []), resumed.w + (resumed.c or [])):
        assert (raw(a) == raw(b)).all()
    for a, b in zip(straight.moments(), resumed.moments()):
        assert (a.view(np.uint32) == b.view(np.uint32)).all()
    ck.close()


@gpu
def test_a_model_trains_on_the_gradients_it_accumulates(dev):
    """README's loop on a model's own parameters: every step sees the gradients
    of its own backward pass alone."""
    gen = torch.Generator(device=dev).manual_seed(4)
    x = torch.randn(9, 131, generator=gen, device=dev).to(BF16)

    class Model(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.gain = torch.nn.Parameter(torch.full((9, 131), 0.5, device=dev, dtype=BF16))
            self.bias = torch.nn.Parameter(torch.zeros(131, device=dev, dtype=BF16))

        def forward(self):
            return (x * self.gain + self.bias).square().sum()

    model, plain = Model(), Model()
    params = list(model.parameters())
    for p in params:
        p.grad = torch.zeros_like(p)
    grads = [p.grad for p in params]
    opt = rcs.AdamWList(params, grads, state_bits=8,
                        wd=[0.01 if p.dim() > 1 else 0.0 for p in params])
    other = list(plain.parameters())
    ref_opt = rcs.AdamWList(other, [None] * 2, state_bits=8, wd=[0.01, 0.0])
    for t in range(1, 5):
        model().backward()
        fresh = list(torch.autograd.grad(plain(), other))
        ref_opt.bind_grads(fresh)
        assert all(bool((a == b).all()) for a, b in zip(grads, fresh))
        opt.step(t, lr=3e-3, clip=1.0)
        ref_opt.step(t, lr=3e-3, clip=1.0)
        torch._foreach_zero_(grads)
        torch.cuda.synchronize()
        assert all(p.grad is g and not bool(g.any()) for p, g in zip(params, grads))
    for a, b in zip(params, other):
        assert (raw(a) == raw(b)).all() and not bool((a == 0.5).all())


@gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("n", [5000, 8_400_000])
def test_captured_and_replayed(dev, bits, n):
    """A graph of norm and step, replayed four times with eager work and
    synchronizations between, against eager calls."""
    a, b = (Case(dev, [n, 333], bits=bits, g=BF16, w=BF16) for _ in range(2))
    norms = [torch.zeros(1, dtype=torch.float64, device=dev) for _ in range(4)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        a.list.grad_norm(out=norms[0])
        a.list.step(3, 1e-3, 1.0, norm_out=norms[1])
    for k in range(4):
        for case in (a, b):
            case.fg.normal_(generator=torch.Generator(device=dev).manual_seed(k))
        torch.cuda.synchronize()
        graph.replay()
        b.list.grad_norm(out=norms[2])
        b.list.step(3, 1e-3, 1.0, norm_out=norms[3])
        float(torch.randn(100, device=dev).sum())
        torch.cuda.synchronize()
        assert len({float(x.cpu()) for x in norms}) == 1
        for x, y in ((a.fw, b.fw), (a.list.m, b.list.m), (a.list.v, b.list.v)):
            assert (raw(x) == raw(y)).all(), k


@gpu
def test_streams(dev):
    """Steps on a side stream; norms of one list on several streams at once,
    while a graph that holds another is replayed."""
    case = Case(dev, [200_001, 50], bits=8)
    want = float(case.list.grad_norm().cpu())
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = [torch.zeros(1, dtype=torch.float64, device=dev) for _ in range(5)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        case.list.grad_norm(out=outs[4])
    torch.cuda.synchronize()
    for _ in range(20):
        for s, o in zip(streams, outs):
            case.list.grad_norm(out=o, stream=s)
        graph.replay()
    torch.cuda.synchronize()
    assert all(float(o.cpu()) == want for o in outs)
    other = Case(dev, [200_001, 50], bits=8)
    with torch.cuda.stream(streams[0]):
        other.list.step(1, 1e-3, 1.0)
    case.list.step(1, 1e-3, 1.0, stream=streams[1])
    torch.cuda.synchronize()
    assert (raw(case.fw) == raw(other.fw)).all() and (raw(case.list.v) == raw(other.list.v)).all()


@gpu
def test_a_captured_binding_binds_at_each_replay(dev):
    """And a captured step without one uses what is bound when it is replayed."""
    case = Case(dev, [3001, 700], bits=8)
    mine = case.g
    twice, four = ([g * k for g in mine] for k in (2.0, 4.0))
    norms = [torch.zeros(1, dtype=torch.float64, device=dev) for _ in range(2)]
    binds, plain = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(binds):
        case.list.bind_grads(twice)
        case.list.step(1, 1e-3, 1.0, norm_out=norms[0])
    with torch.cuda.graph(plain):
        case.list.step(2, 1e-3, 1.0, norm_out=norms[1])
    one = norm_of(case)
    for _ in range(3):
        for grads, factor in ((mine, 1), (four, 4)):
            case.list.bind_grads(grads)
            plain.replay()
            torch.cuda.synchronize()
            assert abs(float(norms[1].cpu()) - factor * one) <= 1e-11 * factor * one
        binds.replay()
        plain.replay()
        torch.cuda.synchronize()
        for x in norms:
            assert abs(float(x.cpu()) - 2 * one) <= 1e-11 * 2 * one


@gpu
def test_gradients_from_before_a_captured_binding_stay(dev):
    """The caller drops the gradients bound before the capture, then those that
    the graph binds: eager calls before the first replay still have the former
    ones, the replays the latter."""
    case = Case(dev, [300_001, 700], bits=8)
    one = norm_of(case)
    twice = [g * 2 for g in case.g]
    norms = [torch.zeros(1, dtype=torch.float64, device=dev) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        case.list.bind_grads(twice)
        case.list.grad_norm(out=norms[0])
    del case.g, case.fg, twice
    torch.cuda.empty_cache()
    junk = [torch.full((300_701,), 9.0, device=dev) for _ in range(8)]
    case.list.grad_norm(out=norms[1])
    torch.cuda.synchronize()
    assert abs(float(norms[1].cpu()) - one) <= 1e-11 * one
    for _ in range(3):
        graph.replay()
        float(junk[0].sum())
        torch.cuda.synchronize()
        assert abs(float(norms[0].cpu()) - 2 * one) <= 1e-11 * 2 * one


@gpu
def test_an_export_spares_the_gradients_of_a_captured_binding(dev):
    """Both sets may be what the device has bound: neither is exported over."""
    case = Case(dev, [600, 400], gap=0)
    other, third = torch.randn(1000, device=dev), torch.randn(1000, device=dev)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        case.list.bind_grads(case.cut(other))
    kept = [raw(x).copy() for x in (case.fg, other)]
    for _ in range(2):
        for x in (case.fg, other):
            with pytest.raises(rcs.RcsError):
                case.list.export_state(w=x)
        case.list.export_state(w=third)
        graph.replay()
        torch.cuda.synchronize()
    assert all((raw(x) == k).all() for x, k in zip((case.fg, other), kept))
    assert (raw(third) == raw(case.fw)).all()
    case.list.bind_grads(case.cut(third))
    case.list.export_state(w=other)
    with pytest.raises(rcs.RcsError):
        case.list.export_state(w=third)
    torch.cuda.synchronize()


@gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("n", [5000, 8_400_000])
def test_last_grad_norm_reports_a_step(dev, bits, n):
    """Whatever ran on the stream before, wherever else the norm goes, and for a
    step that is skipped too; each stream has its own, and a captured step
    leaves it."""
    case = Case(dev, [n, 77], bits=bits)
    flat = torch.ones(1000, device=dev)
    want = float(case.list.grad_norm().cpu())
    outs = (None, torch.zeros(1, dtype=torch.float64, device=dev),
            torch.zeros(1, dtype=torch.float64, pin_memory=True))

    def last(**kw):
        x = rcs.last_grad_norm(**kw)
        torch.cuda.synchronize()
        return float(x.cpu())

    rcs.grad_global_norm(flat)
    ones = last()
    for out in outs:
        rcs.grad_global_norm(flat)
        assert last() == ones != want
        case.list.step(1, 0.0, 1.0, norm_out=out)
        assert last() == want
        assert out is None or float(out.cpu()) == want
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    case.list.step(2, 0.0, 1.0, grad_scale=0.5, stream=side)
    assert last(stream=side) == want / 2 and last() == want
    rcs.grad_global_norm(flat)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        case.list.step(3, 0.0, 1.0, norm_out=outs[1])
    graph.replay()
    assert last() == ones and float(outs[1].cpu()) == want
    case.g[1][3] = float("inf")
    case.list.step(4, 0.0, 1.0)
    assert last() == float("inf")


@gpu
def test_a_step_on_a_fresh_stream_while_another_is_captured(dev):
    """The stream's workspace is made on the way; the capture goes on."""
    case, other = Case(dev, [3000]), Case(dev, [3000], bits=8)
    want, mine = norm_of(case), float(other.list.grad_norm().cpu())
    side, norm_side = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.zeros(1, dtype=torch.float64, device=dev) for _ in range(3)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        case.list.grad_norm(out=outs[0])
        other.list.step(1, 0.0, 1.0, norm_out=outs[1], stream=side)
        other.list.grad_norm(out=outs[2], stream=norm_side)
    torch.cuda.synchronize()
    assert float(outs[1].cpu()) == float(outs[2].cpu()) == mine
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert abs(float(outs[0].cpu()) - want) <= 1e-11 * want


@gpu
def test_norms_of_several_lists_in_turn_on_one_stream(dev):
    """Norms of 1, 37 and 256 blocks and the flat norm take turns in one
    workspace, steps and a graph between them."""
    cases = [Case(dev, sizes, g=BF16, w=BF16) for sizes in ([7], [300_001, 9], [9_000_001])]
    flat = torch.randn(100_003, device=dev)
    want = [norm_of(c) for c in cases]
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    held = torch.zeros(1, dtype=torch.float64, device=dev)
    with torch.cuda.graph(graph):
        cases[1].list.grad_norm(out=held)
    outs = [torch.zeros(1, dtype=torch.float64, device=dev) for _ in range(4)]
    first = None
    with torch.cuda.stream(stream):
        for k in range(25):
            for c, o in zip(cases, outs):
                o.zero_()
                c.list.grad_norm(out=o)
            rcs.grad_global_norm(flat, out=outs[3])
            graph.replay()
            cases[2].list.step(k + 1, 0.0, 1.0)  # its own count, on the same list
            stream.synchronize()
            now = [float(x.cpu()) for x in (*outs, held)]
            first = first or now
            assert now == first
    for c, x, y in zip(cases, first, want):
        assert abs(x - y) <= 2 * max(c.n, 16) * 2.0 ** -53 * y
    assert first[4] == first[1]


@gpu
def test_determinism(dev):
    """The same list and inputs give the same bits, wherever the gradients lie."""
    a, b = Case(dev, [1_000_003, 17], bits=8), Case(dev, [1_000_003, 17], bits=8, gap=1)
    moved = [torch.empty(g.numel() + 5, device=dev)[k + 1:k + 1 + g.numel()].copy_(g)
             for k, g in enumerate(b.g)]
    b.list.bind_grads(moved)
    for t in (1, 2, 3):
        a.list.step(t, 1e-3, 1.0)
        b.list.step(t, 1e-3, 1.0)
    torch.cuda.synchronize()
    for x, y in ((a.fw, b.fw), (a.list.m, b.list.m), (a.list.v, b.list.v)):
        assert (raw(x) == raw(y)).all()


@gpu
def test_rounding_keeps_the_mean(dev):
    """A gradient that keeps v a tenth of a grid step above a held value: the
    mean over 200,000 elements of what is held follows (with nearest rounding
    it would not move). Standard error: half a step / sqrt(n)."""
    n = 200_000
    case = Case(dev, [n], bits=8, state=False, wd=[0.0])
    v0 = torch.full((n,), 1.125, device=dev)
    v0[::128] = 2.0  # the block's largest
    case.list.import_state(m=torch.zeros(n, device=dev), v=v0)
    # v1 = 0.999 v + 0.001 g^2 = 1.1375, a tenth of the step of 0.125 up
    case.g[0].fill_(float(np.sqrt((1.1375 - 0.999 * 1.125) / 0.001)))
    case.list.step(1, 1e-3, float("inf"))
    _, v = case.moments()
    v = v[np.arange(n) % 128 != 0]
    assert set(np.unique(v)) == {np.float32(1.125), np.float32(1.25)}
    assert abs(v.mean(dtype=np.float64) - 1.1375) <= 6 * 0.125 / 2 / np.sqrt(v.size)


@gpu
def test_more_than_2_to_the_32_elements(dev):
    """Positions past 32 bits: 2^32 - 3 elements before the second tensor, whose
    random bits run over the carry inside one lane's vector."""
    big = (1 << 32) - 3
    w = torch.zeros(big, dtype=BF16, device=dev)
    g = torch.zeros(big, dtype=BF16, device=dev)
    g[-5:] = 2.0
    w2, g2 = torch.randn(1500, device=dev), torch.randn(1500, device=dev)
    lst = rcs.AdamWList([w, w2], [g, g2], state_bits=8, seed=77, wd=0.0)
    w0 = host(w2)
    norm = float(lst.grad_norm().cpu())
    want = np.sqrt((host(g2).astype(np.float64) ** 2).sum() + 20.0)
    assert abs(norm - want) <= 1e-11 * want
    lst.step(1, 1e-3, 1.0)
    torch.cuda.synchronize()
    z = np.zeros(1500, np.float32)
    rw, rm, rv = ref.update32(w0, host(g2), z, z, norm, 1, 1e-3, 0.0, 1.0)
    bits = ref.random_bits(77, 1, big, 1500)
    for which, x, add, codes in (("m", rm, bits & np.uint64(0xFFFFF), lst.m),
                                 ("v", rv, bits >> np.uint64(12), lst.v)):
        c, _ = ref.encode(x, which, add)
        assert (raw(codes[-1536:]) == c).all()
    w64, size = ref.weights64(w0, rm, rv, 1, 1e-3, 0.0)
    assert (np.abs(host(w2) - w64) <= WEIGHT_ULPS * 2.0 ** -24 * size).all()
    # lr * m_hat / sqrt(v_hat) = lr where g > 0, rounded to bf16
    assert bool((w[-5:].float() + 1e-3).abs().max() <= 2.0 ** -8 * 1e-3)
    assert not bool(w[:-5].any())
    out = torch.empty(lst.n, dtype=BF16, device=dev)
    lst.export_state(w=out)
    torch.cuda.synchronize()
    assert (raw(out[-1500:]) == raw(w2.to(BF16))).all() and (raw(out[big - 5:big]) == raw(w[-5:])).all()


@gpu
def test_refusals_on_the_device(dev):
    """What the host refuses leaves the arrays as they are."""
    L = rcs.lib()
    case = Case(dev, [500, 100], bits=8)
    lst = case.list
    before = [raw(x).copy() for x in (case.fw, lst.m, lst.v)]
    for kw in (dict(t=0), dict(lr=float("nan")), dict(clip=0.0), dict(clip=float("nan")),
               dict(grad_scale=0.0), dict(grad_scale=float("inf")), dict(beta1=1.0),
               dict(beta2=-0.1), dict(beta1=float("nan")), dict(eps=0.0), dict(eps=1e-40)):
        with pytest.raises(rcs.RcsError):
            lst.step(**{**dict(t=1, lr=1e-3, clip=1.0), **kw})
    with pytest.raises(rcs.RcsError):
        lst.grad_norm(grad_scale=-1.0)
    with pytest.raises(TypeError):
        lst.grad_norm(out=torch.zeros(1, dtype=torch.float64))  # pageable
    flat = [torch.zeros(600, device=dev) for _ in range(3)]
    with pytest.raises(rcs.RcsError):
        lst.import_state(m=flat[0])  # 8-bit moments come together
    with pytest.raises(rcs.RcsError):
        lst.export_state()
    with pytest.raises(rcs.RcsError):
        lst.export_state(w=flat[0], m=flat[0])
    with pytest.raises(ValueError):
        lst.export_state(w=torch.zeros(599, device=dev))
    with pytest.raises(TypeError):
        lst.export_state(w=torch.zeros(600, device=dev, dtype=F16))
    with pytest.raises(TypeError):
        lst.export_state(w=torch.zeros(1200, device=dev)[::2])
    with pytest.raises(rcs.RcsError):  # into the list's own weights
        lst.export_state(w=case.fw[1:601])
    # the same tensor twice, a gradient that is written, an overlapping copy
    w, g = torch.zeros(64, device=dev), torch.zeros(64, device=dev)
    for ws, gs in (([w, w], [g, g]), ([w, w[32:]], [g, g[32:]]), ([w], [w])):
        with pytest.raises(rcs.RcsError):
            rcs.AdamWList(ws, gs)
    with pytest.raises(rcs.RcsError):
        rcs.AdamWList([w], [g], copies=[w.view(BF16)[:64]])
    with pytest.raises(TypeError):
        rcs.AdamWList([w.to(BF16)], [g], copies=[g.to(BF16)])
    with pytest.raises(ValueError):
        rcs.AdamWList([w], [g[:32]])
    with pytest.raises(TypeError):
        rcs.AdamWList([w.double()], [g])
    with pytest.raises(TypeError):
        rcs.AdamWList([torch.zeros(8, 8, device=dev).t()], [torch.zeros(8, 8, device=dev)])
    with pytest.raises(ValueError):
        lst.bind_grads([case.g[0]])
    with pytest.raises(TypeError):
        lst.bind_grads([case.g[0].to(BF16), case.g[1]])
    with pytest.raises(rcs.RcsError):
        lst.bind_grads([case.g[0], case.w[1]])
    # a short array: it ends outside its allocation
    rows = (tensor_list._Tensor * 1)(_row(w=w.data_ptr(), g=g.data_ptr(), m=lst.m.data_ptr(),
                                          v=lst.v.data_ptr(), exps=lst.exps.data_ptr(),
                                          n=1 << 36))
    h = ctypes.c_void_p()
    assert L.rcs_list_create(rows, 1, 8, ctypes.byref(h)) in (rcs.ESIZE, rcs.EINVAL)
    torch.cuda.synchronize()
    for x, b in zip((case.fw, lst.m, lst.v), before):
        assert (raw(x) == b).all()
    lst.close()
    with pytest.raises(ValueError):
        lst.step(1, 1e-3, 1.0)
    lst.close()


@gpu
def test_a_list_may_go_while_another_graph_is_captured(dev):
    """close() (as a collector may call it) during a capture on another stream
    neither fails nor breaks the capture."""
    case, gone = Case(dev, [1000]), Case(dev, [1000])
    out = torch.zeros(1, dtype=torch.float64, device=dev)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        case.list.grad_norm(out=out)
        gone.list.close()
    graph.replay()
    torch.cuda.synchronize()
    assert float(out.cpu()) == float(case.list.grad_norm().cpu())


@gpu
def test_the_list_keeps_its_memory(dev):
    """Tensors that are dropped or given other storage do not take the list's
    memory with them."""
    w, g = torch.ones(1000, device=dev), torch.ones(1000, device=dev)
    alias = w.detach()
    lst = rcs.AdamWList([w], [g])
    w.data = torch.zeros(1000, device=dev)
    del g
    lst.step(1, 1e-3, float("inf"))
    torch.cuda.synchronize()
    assert not w.any() and bool((alias < 1).all())
