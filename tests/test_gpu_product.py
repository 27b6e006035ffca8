"""GPU tests of the products on FP4 weights: fp4q_linear, fp4q_linear_group,
fp4q_matmul, fp4q_matmul_group, against the same formula in 64 bits.

Two kinds of comparison:

* exact: small integers and power-of-two scales, so that every product and
  every partial sum is a multiple of one power of two below 2^24 units of it.
  Then binary32 sums are exact in any order and the outputs must be equal;
* bounded: real distributions, |y - ref| within a bound counted from the
  roundings (see _bound)."""
import itertools

import numpy as np
import pytest
import torch

import fp4_post_weight_grid_b200 as fq
import synth

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
GRID = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
BLOCK = {fq.NVFP4: 16, fq.MXFP4: 32}
NAMES = {fq.NVFP4: "nvfp4", fq.MXFP4: "mxfp4"}
FORMS = [(p, f) for p in ("linear", "matmul") for f in (fq.NVFP4, fq.MXFP4)]
form_ids = [f"{p}-{NAMES[f]}" for p, f in FORMS]


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _scale_values(fmt, b):
    """Block scale bytes as values, float64."""
    if fmt == fq.NVFP4:
        return b.view(torch.float8_e4m3fn).double()
    return torch.where(b == 255, torch.nan, torch.exp2(b.double() - 127))


def _decode(fmt, codes, scales):
    """Values of codes [..., r, c/2] and row-major scales, float64, without the global scale."""
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    return GRID.to(codes.device)[nib] * _scale_values(fmt, scales).repeat_interleave(BLOCK[fmt], -1)


def _fp4(fmt, rows, cols, g, exact):
    """Random codes and scale bytes on the GPU.  exact: scales 1, 2 or 4."""
    codes = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, generator=g)
    shape = (rows, cols // BLOCK[fmt])
    if exact:
        e = torch.randint(0, 3, shape, generator=g)
        s = (e + 7) << 3 if fmt == fq.NVFP4 else e + 127
    else:
        s = torch.randint(0x28, 0x68, shape, generator=g) if fmt == fq.NVFP4 else torch.randint(112, 127, shape, generator=g)
    return codes.to(DEV), s.to(torch.uint8).to(DEV)


class Problem:
    """Inputs of one product and its reference: form "linear" or "matmul", groups None for the dense calls."""

    def __init__(self, form, fmt, m, n, k, counts=None, before=0, behind=0, exact=False, seed=0, out=torch.float32,
                 bias=False, mul=False, residual=False, act=fq.ACT_NONE):
        g = _gen(seed)
        self.form, self.fmt, self.n, self.k, self.act, self.out = form, fmt, n, k, act, out
        self.counts = counts
        groups = 1 if counts is None else len(counts)
        if counts is not None:
            m = before + sum(counts) + behind
            ends = np.concatenate([[before], before + np.cumsum(counts)])
            self.offsets = torch.tensor(ends, dtype=torch.int32, device=DEV)
            self.ends = [int(v) for v in ends]
        else:
            self.ends = [0, m]
        self.m = m
        ws = [_fp4(fmt, n, k, g, exact) for _ in range(groups)]
        self.w_codes = torch.stack([c for c, _ in ws])
        self.w_scales = torch.stack([s for _, s in ws])
        self.tiled = fq.mma_scales(self.w_scales)
        one = torch.ones(groups)
        self.S = (one * 2 if exact else one * 0.01 * (1 + torch.arange(groups))).to(DEV)
        self.x_S = torch.tensor([0.5 if exact else 0.03], device=DEV)
        if form == "matmul":
            self.x, self.x_scales = _fp4(fmt, m, k, g, exact)
        else:
            self.x_scales = None
            x = torch.randint(-3, 4, (m, k), generator=g).float() if exact else torch.randn(m, k, generator=g)
            self.x = x.bfloat16().to(DEV)

        def more(*shape):
            v = torch.randint(-4, 5, shape, generator=g).float() if exact else torch.randn(*shape, generator=g)
            return v.to(out).to(DEV)

        self.bias = more(groups, n) if bias else None
        self.mul = more(m, n) if mul else None
        self.residual = more(m, n) if residual else None

    def run(self, y=None, status=None, stream=None, **kw):
        nv = self.fmt == fq.NVFP4
        y = torch.full((self.m, self.n), 77.0, dtype=self.out, device=DEV) if y is None else y
        status = torch.zeros(1, dtype=torch.int32, device=DEV) if status is None else status
        args = [self.fmt, self.x]
        if self.form == "matmul":
            args += [self.x_scales, self.x_S if nv else None]
        name = "fp4q_" + self.form
        if self.counts is None:
            args += [self.w_codes[0], self.tiled]
        else:
            args += [self.offsets, self.w_codes, self.tiled]
            name += "_group"
        ep = dict(bias=self.bias, act=self.act, mul=self.mul, residual=self.residual)
        ep.update(kw)
        getattr(fq, name)(*args, self.S if nv else None, y, status, stream=stream, **ep)
        return y, status

    def reference(self):
        """(outputs, bound on |y - output|), float64 [m, n]; rows of no group are NaN."""
        nv = self.fmt == fq.NVFP4
        ref = torch.full((self.m, self.n), torch.nan, dtype=torch.float64, device=DEV)
        tol = torch.zeros_like(ref)
        for e in range(len(self.ends) - 1):
            r = slice(self.ends[e], self.ends[e + 1])
            if r.start == r.stop:
                continue
            w = _decode(self.fmt, self.w_codes[e], self.w_scales[e])
            x = _decode(self.fmt, self.x[r], self.x_scales[r]) if self.form == "matmul" else self.x[r].double()
            S = (float(self.S[e]) if nv else 1.0) * (float(self.x_S) if nv and self.form == "matmul" else 1.0)
            ref[r], tol[r] = _bound(
                (x @ w.T) * S, (x.abs() @ w.abs().T) * abs(S), self.k, self.act, self.out,
                None if self.bias is None else self.bias[e].double(),
                None if self.mul is None else self.mul[r].double(),
                None if self.residual is None else self.residual[r].double())
        return ref, tol

    def check(self, y=None, status=None, exact=False):
        if y is None:
            y, status = self.run()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        ref, tol = self.reference()
        inside = torch.zeros(self.m, dtype=torch.bool, device=DEV)
        inside[self.ends[0]:self.ends[-1]] = True
        assert bool((y[~inside] == 77.0).all()), "rows of no group were written"
        got, ref, tol = y[inside].double(), ref[inside], tol[inside]
        if exact:
            bad = got != ref
        else:
            bad = ~((got - ref).abs() <= tol)
        at = bad.nonzero()[:4].tolist()
        assert not bool(bad.any()), (f"{int(bad.sum())} of {bad.numel()} outputs off, first {at}: "
                                     f"{[(float(got[i, j]), float(ref[i, j])) for i, j in at]}")


U = 2.0 ** -24      # half a step of binary32


def _activation(z, act):
    if act == fq.ACT_RELU:
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == fq.ACT_GELU:
        return z * torch.special.ndtr(z)
    if act == fq.ACT_GELU_TANH:
        return z * torch.sigmoid((8 / np.pi) ** 0.5 * (z + 0.044715 * z ** 3))
    if act == fq.ACT_SILU:
        return z * torch.sigmoid(z)
    return z


def _bound(z, absz, k, act, out, bias, mul, residual):
    """The output and how far a result may be from it.

    Sum: a tensor-core step adds 16 or more products to the running sum with
    truncation, i.e. at most one step (2U) of the largest magnitude met per
    product and one more per 16 for the running sum, none above sum|x w|:
    (k + k/16 + 2) * 2U * absz; the two roundings of S (x_S * w_S, acc * S) are
    in the 2.  Bias: half a step.  Activation: slope at most 1.13; its own
    value from functions of a few ulp whose arguments are rounded: the relative
    error grows with |z|^2, where the value falls as exp(-z^2/2) or exp(-|z|),
    so 2^-20 * (1 + |value|) covers it.  mul, residual: half a step each; the
    output half a step of its type."""
    err = (k + k / 16 + 2) * 2 * U * absz
    if bias is not None:
        z = z + bias
        err = err + U * z.abs()
    a = _activation(z, act)
    if act in (fq.ACT_GELU, fq.ACT_GELU_TANH, fq.ACT_SILU):
        err = 1.13 * err + 2.0 ** -20 * (1 + a.abs())
    if mul is not None:
        a = a * mul
        err = err * mul.abs() + U * a.abs()
    if residual is not None:
        a = a + residual
        err = err + U * a.abs()
    return a, err + (a.abs() + err) * torch.finfo(out).eps / 2 + 2.0 ** -133


SHAPES = [(1, 1, 32), (1, 128, 64), (2, 130, 96), (8, 64, 256), (17, 96, 160), (31, 257, 288), (64, 128, 544),
          (65, 200, 512), (129, 257, 1056), (256, 384, 256), (300, 1000, 1056), (1, 1024, 4096), (5, 333, 8192),
          (513, 130, 320),
          # enough rows of W that the wider token tiles are chosen, their last one partly filled
          (40, 19073, 96), (60, 19073, 352), (120, 19073, 288), (300, 19073, 96), (257, 19000, 1056)]


@pytest.mark.parametrize("form,fmt", FORMS, ids=form_ids)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_exact_sums(form, fmt, m, n, k):
    # |x| <= 3 or 6*4, |w| <= 6*4, both multiples of 1/2: at most 8192 * 24 * 24 = 4.7e6 in units of 1/4
    p = Problem(form, fmt, m, n, k, exact=True, seed=m + n + k, bias=True)
    if k * 24 * 24 * 4 >= 1 << 24:      # keep the partial sums exact: fewer, and smaller, terms
        p.w_codes &= 0x99                # elements 0 and +-1/2
        if form == "matmul":
            p.x &= 0x99
    p.check(exact=True)


@pytest.mark.parametrize("form,fmt", FORMS, ids=form_ids)
@pytest.mark.parametrize("counts,before,behind", [
    ([5], 0, 0), ([0, 3, 0, 0, 1], 0, 2), ([1] * 40, 1, 0), ([64, 0, 130, 7, 65], 3, 5), ([0, 0, 300], 0, 1),
    ([257, 0], 0, 0), ([0, 0, 0], 2, 2), ([0] * 1023 + [2], 0, 0), ([2, 16, 17, 32, 33, 128, 129], 0, 3)])
@pytest.mark.parametrize("n,k", [(130, 96), (256, 544)])
def test_exact_groups(form, fmt, counts, before, behind, n, k):
    if len(counts) > 1000 and n > 200:
        pytest.skip("one size of the many groups is enough")
    Problem(form, fmt, 0, n, k, counts=counts, before=before, behind=behind, exact=True, seed=n + len(counts),
            bias=True).check(exact=True)


@pytest.mark.parametrize("form,fmt", FORMS, ids=form_ids)
@pytest.mark.parametrize("counts,n", [([1, 200], 600), ([0, 0, 0, 330], 300), ([5, 400], 601)])
def test_exact_groups_whose_tiles_outnumber_the_clusters(form, fmt, counts, n):
    # few tiles are expected from the average group, so that clusters share K; one group has many
    p = Problem(form, fmt, 0, n, 2336, counts=counts, behind=1, exact=True, bias=True)
    p.w_codes &= 0x99
    p.check(exact=True)


@pytest.mark.parametrize("form,fmt", FORMS, ids=form_ids)
@pytest.mark.parametrize("counts", [[300, 0, 513, 100], [90, 130], [33, 40, 61]])
def test_exact_groups_of_wide_tiles(form, fmt, counts):
    Problem(form, fmt, 0, 10001, 352, counts=counts, behind=3, exact=True, bias=True).check(exact=True)


@pytest.mark.parametrize("form,fmt", FORMS, ids=form_ids)
@pytest.mark.parametrize("act", [fq.ACT_NONE, fq.ACT_RELU, fq.ACT_GELU, fq.ACT_GELU_TANH, fq.ACT_SILU])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_epilogue(form, fmt, act, out):
    for i, (bias, mul, residual) in enumerate(itertools.product((False, True), repeat=3)):
        Problem(form, fmt, 37, 150, 416, act=act, out=out, bias=bias, mul=mul, residual=residual, seed=i).check()


@pytest.mark.parametrize("form,fmt", FORMS, ids=form_ids)
@pytest.mark.parametrize("act", [fq.ACT_NONE, fq.ACT_RELU, fq.ACT_GELU, fq.ACT_GELU_TANH, fq.ACT_SILU])
@pytest.mark.parametrize("m,n", [(5, 130), (37, 136), (300, 19001)])
def test_activations_of_large_infinite_and_missing_sums(form, fmt, act, m, n):
    """The bias makes the sums: columns of NaN, both infinities, and magnitudes up to the largest float."""
    p = Problem(form, fmt, m, n, 64, act=act, exact=True, bias=True)
    p.x.zero_()
    z = torch.tensor([torch.nan, torch.inf, -torch.inf, 0.0, 3e38, -3e38, 1e20, -1e20, 1e5, -1e5, 200.0, -200.0, 90.0, -90.0,
                      20.0, -20.0, 10.5, -10.5, 1e-30, -1e-30], device=DEV)
    p.bias[0] = z.repeat(n // len(z) + 1)[:n]
    y, st = p.run()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    z = p.bias[0]
    want = _activation(z.double(), act).expand(m, n)
    if act == fq.ACT_RELU:
        want = torch.where(torch.isnan(z), z, z.clamp_min(0)).double().expand(m, n)
    # of -inf, z * Phi(z) and the like are -inf * 0, a NaN, as in 64 bits
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    finite = torch.isfinite(want)
    assert torch.equal(y[torch.isinf(want)].double(), want[torch.isinf(want)])
    # the functions' bound of _bound; with 3e38 no result may round to infinity
    assert bool(((y.double() - want).abs()[finite] <= 2.0 ** -20 * (1 + want.abs()[finite])).all())


@pytest.mark.parametrize("form,fmt", FORMS, ids=form_ids)
def test_epilogue_of_groups(form, fmt):
    Problem(form, fmt, 0, 150, 416, counts=[3, 0, 70, 1], before=2, behind=3, act=fq.ACT_SILU, out=torch.bfloat16,
            bias=True, mul=True, residual=True).check()


@pytest.mark.parametrize("form,fmt", FORMS, ids=form_ids)
@pytest.mark.parametrize("m,n,k", [(13, 129, 4128), (13, 136, 4128), (33, 1111, 2080), (50, 2000, 1056)])
def test_epilogue_of_tiles_whose_columns_are_split(form, fmt, m, n, k):
    # w of 0 and +-1/2, scales up to 4, |x| <= 24, |mul| <= 4: at most 4128 * 2 * 24 * 2 * 4 = 1.6e6, in units of 1/4
    for counts in (None, [m, 0, 3]):
        p = Problem(form, fmt, m if counts is None else 0, n, k, counts=counts, behind=2 if counts else 0, bias=True, mul=True,
                    residual=True, exact=True)
        p.w_codes &= 0x99
        p.check(exact=True)
    for out in (torch.float32, torch.bfloat16):
        Problem(form, fmt, m, n, k, act=fq.ACT_SILU, out=out, bias=True, mul=True, residual=True).check()


@pytest.mark.parametrize("form,fmt", FORMS, ids=form_ids)
@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (7, 1000, 14336), (100, 520, 1056), (700, 1111, 4128)])
def test_random(form, fmt, m, n, k):
    Problem(form, fmt, m, n, k, out=torch.bfloat16, seed=k).check()


@pytest.mark.parametrize("form,fmt", FORMS, ids=form_ids)
@pytest.mark.parametrize("m,n,k,counts", [
    (70, 5000, 4128, None), (150, 5001, 6176, None), (20, 19073, 4128, None), (40, 19072, 4128, None), (3, 700, 16384, None),
    (33, 8200, 9216, None), (0, 3001, 4640, [200, 0, 90, 17]), (0, 3000, 4640, [1, 140])])
def test_float_results_of_long_sums(form, fmt, m, n, k, counts):
    # Exact, and on real values within what pieces of 2048 columns allow.  A piece is 128 additions of 16 columns,
    # each truncated: off by less than one step, 2U relative to the running sum.  Over many outputs of independent
    # terms the running sum's norm is at most the result's, so the norm of the error is below 128 * 2U = 1.5e-5 of
    # it for every piece, and the pieces' errors add as their own parts of the result do.
    p = Problem(form, fmt, m, n, k, counts=counts, behind=1 if counts else 0, exact=True, bias=True, mul=True)
    p.w_codes &= 0x99
    if form == "matmul":
        p.x &= 0x99
    p.check(exact=True)
    p = Problem(form, fmt, m, n, k, counts=counts, behind=1 if counts else 0)
    y, st = p.run()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    ref, _ = p.reference()
    inside = ~torch.isnan(ref)
    off = (y.double() - ref)[inside]
    assert float(off.norm() / ref[inside].norm()) <= 128 * 2 * U


def _norm_off(p):
    y, st = p.run()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    ref, _ = p.reference()
    return float((y.double() - ref).norm() / ref.norm())


@pytest.mark.parametrize("fmt", [fq.NVFP4, fq.MXFP4], ids=NAMES.get)
@pytest.mark.parametrize("m,n,k", [(1, 64, 65536), (2, 128, 262144), (4, 16, 1 << 20), (3, 19000, 3520), (8, 5000, 8192)])
def test_float_results_of_few_tokens_on_long_columns(fmt, m, n, k):
    # A piece of 2048 columns is 128 additions of 16 columns, each truncated: off by at most one step, 2U of the
    # running sum, and by half a step, U, on average over many outputs.  The running sum's norm after i of them
    # is sqrt(i / 128) of the piece's, so the norm of the piece's error is below U * 128 * 2/3 of its own.  The
    # pieces (independent, as their terms are) add up like their errors.  The additions of the pieces round to
    # nearest: U each, of either sign; at most 256 per warp here, sqrt(256) * U, well below.
    assert _norm_off(Problem("linear", fmt, m, n, k, seed=k + n)) <= U * 128 * 2 / 3


@pytest.mark.parametrize("fmt", [fq.NVFP4, fq.MXFP4], ids=NAMES.get)
@pytest.mark.parametrize("m,n,k", [(16, 300, 262144), (40, 700, 65536), (120, 10001, 32768), (300, 2048, 65536)])
def test_float_results_of_more_tokens_on_long_columns(fmt, m, n, k):
    # As above, in runs of 2048 columns; one accumulator would be off by 6e-6 to 2.6e-5.
    assert _norm_off(Problem("linear", fmt, m, n, k, seed=k + n)) <= U * 128 * 2 / 3


@pytest.mark.parametrize("fmt", [fq.NVFP4, fq.MXFP4], ids=NAMES.get)
@pytest.mark.parametrize("m,n,k", [(1, 300, 262144), (16, 19073, 16384), (70, 700, 65536), (300, 2048, 16384),
                                   (300, 19073, 8192)])
def test_float_results_of_long_fp4_columns(fmt, m, n, k):
    # As above; a run is 4096 columns, 64 additions of 64 columns each, and at most 64 runs of a block are added.
    assert _norm_off(Problem("matmul", fmt, m, n, k, seed=k + n)) <= U * 64 * 2 / 3


@pytest.mark.parametrize("fmt", [fq.NVFP4, fq.MXFP4], ids=NAMES.get)
@pytest.mark.parametrize("m,n,k,counts", [
    (300, 19073, 4128, None), (170, 19072, 8224, None), (100, 19073, 4128, None), (0, 10001, 4640, [300, 0, 513, 100]),
    (0, 10000, 4640, [129]),
    # and of tiles whose columns a cluster splits
    (128, 4096, 14336, None), (16, 301, 40032, None), (1, 64, 66080, None), (64, 4100, 10272, None),
    (0, 640, 40032, [5, 0, 300])])
def test_exact_long_sums_of_wide_and_split_tiles(fmt, m, n, k, counts):
    # elements 0 and +-1/2, scales up to 4: at most 66080 * 2 * 2 * 4 (mul) = 1.1e6 in units of 1/4
    for out in (torch.float32, torch.bfloat16):
        p = Problem("matmul", fmt, m, n, k, counts=counts, behind=2 if counts else 0, exact=True, bias=True, mul=True, out=out)
        p.w_codes &= 0x99
        p.x &= 0x99
        y, st = p.run()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        ref, _ = p.reference()
        inside = ~torch.isnan(ref)
        assert torch.equal(y[inside], ref[inside].to(out))
        assert bool((y[~inside] == 77.0).all())


@pytest.mark.parametrize("form,fmt", FORMS, ids=form_ids)
@pytest.mark.parametrize("m,n,counts", [(2, 8, None), (5, 16, None), (0, 16, [3, 0, 2])])
def test_bf16_results_of_very_long_columns(form, fmt, m, n, counts):
    # With minus the rounded result as residual an output is a small difference, whose rounding is 2^-9 of at most
    # 2^-9 of the result.  A run is 65536 columns: 4096 additions of 16 columns for linear, 1024 of 64 for matmul,
    # with U of the running sum on average each, as above.
    p = Problem(form, fmt, m, n, 1 << 23, counts=counts, out=torch.bfloat16, seed=n)
    ref, _ = p.reference()
    p.residual = (-ref).bfloat16()
    y, st = p.run()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    off = y.double() - p.residual.double() - ref
    assert float(off.norm() / ref.norm()) <= U * (4096 if form == "linear" else 1024) * 2 / 3 + 2.0 ** -17


@pytest.mark.parametrize("fmt", [fq.NVFP4, fq.MXFP4], ids=["nvfp4", "mxfp4"])
@pytest.mark.parametrize("m,k", [(1, 32), (5, 256), (40, 1024), (33, 1056), (200, 544), (300, 4096)])
def test_token_scales_at_any_word(fmt, m, k):
    # the first and the last rows lie at the ends of the buffer that the loads may not leave
    p = Problem("matmul", fmt, m, 200, k, exact=True)
    want, _ = p.run()
    torch.cuda.synchronize()
    for words in (1, 2, 3):
        buf = torch.full((p.x_scales.numel() + 4 * words,), 255, dtype=torch.uint8, device=DEV)
        p.x_scales = buf[4 * words:].view(p.x_scales.shape).copy_(p.x_scales)
        y, st = p.run()
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and torch.equal(y, want), words


@pytest.mark.parametrize("form,fmt", FORMS, ids=form_ids)
def test_output_on_top_of_an_input(form, fmt):
    p = Problem(form, fmt, 70, 136, 288, out=torch.bfloat16, mul=True, residual=True)
    want, _ = p.run()
    for name in ("mul", "residual"):
        y = getattr(p, name).clone()
        p.run(y, **{name: y})
        torch.cuda.synchronize()
        assert torch.equal(y, want), name


@pytest.mark.parametrize("form,fmt", FORMS, ids=form_ids)
def test_scale_extremes(form, fmt):
    """Every scale byte the formats have, element magnitudes at both ends."""
    m, n, k = 16, 256, 64
    p = Problem(form, fmt, m, n, k, exact=True)
    b = torch.arange(n, device=DEV)
    if fmt == fq.NVFP4:
        b = b % 128
        b = torch.where(b == 127, 0, b)
    else:
        b = b.clamp_max(254)
    p.w_scales[0] = b.to(torch.uint8)[:, None]
    p.tiled = fq.mma_scales(p.w_scales)
    if form == "linear":
        p.x.fill_(0.0)
        p.x[:, ::7] = 0.25
    else:
        p.x.zero_()
        p.x[:, ::7] = 0x01
        p.x_scales.fill_(0x28 if fmt == fq.NVFP4 else 125)
    y, st = p.run()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    ref, _ = p.reference()
    ref32 = ref.float()
    big = ref32.abs() < 2.0 ** -120        # sums of subnormal products may be flushed to the smallest steps
    assert torch.equal(y[~big], ref32[~big])
    assert float((y[big].double() - ref[big]).abs().max() if big.any() else 0.0) <= 2.0 ** -126
    # a NaN scale reaches its own output column only
    p.w_scales[0][5, 1] = 0x7F if fmt == fq.NVFP4 else 255
    p.tiled = fq.mma_scales(p.w_scales)
    y2, _ = p.run()
    torch.cuda.synchronize()
    nan = torch.isnan(y2)
    assert bool(nan[:, 5].all()) and int(nan.sum()) == m
    keep = torch.ones(n, dtype=torch.bool, device=DEV)
    keep[5] = False
    assert torch.equal(y2[:, keep], y[:, keep])


@pytest.mark.parametrize("m,n,k,counts", [(3, 200, 96, None), (16, 512, 4096, None), (300, 1000, 4640, None), (0, 130, 96, [2, 0, 40])])
@pytest.mark.parametrize("w_S,x_S", [(2.0 ** -70, 1.1 * 2.0 ** -70), (1.1 * 2.0 ** -75, 1.3 * 2.0 ** -75), (2.0 ** 52, 1.1 * 2.0 ** 52)])
def test_global_scales_at_the_ends_of_the_quantizers_range(m, n, k, counts, w_S, x_S):
    # 2^-64 / 2688 to 2^64 / 2688 each; their product may lie below the normal numbers
    p = Problem("matmul", fq.NVFP4, m, n, k, counts=counts, behind=1 if counts else 0)
    p.S.fill_(w_S)
    p.x_S.fill_(x_S)
    p.check()


@pytest.mark.parametrize("fmt", [fq.NVFP4, fq.MXFP4], ids=NAMES.get)
@pytest.mark.parametrize("grouped", [False, True])
def test_non_finite_rows_stay_in_their_rows(fmt, grouped):
    p = Problem("linear", fmt, 40, 140, 96, counts=[13, 27] if grouped else None, behind=4 if grouped else 0, exact=True)
    want, _ = p.run()
    p.x[7, 50] = torch.nan
    p.x[12, 3] = torch.inf
    if grouped:
        p.x[40:] = torch.nan        # behind the last group
    got, _ = p.run()
    torch.cuda.synchronize()
    rest = torch.ones(p.m, dtype=torch.bool, device=DEV)
    rest[[7, 12]] = False
    assert torch.equal(got[rest], want[rest])
    assert bool(torch.isnan(got[7]).all())
    w = _decode(fmt, p.w_codes[0], p.w_scales[0])[:, 3]
    assert torch.equal(torch.isnan(got[12]), w == 0)        # inf * 0
    assert bool((got[12][w != 0] == torch.sign(w[w != 0]) * torch.inf).all())


@pytest.mark.parametrize("form,fmt", FORMS, ids=form_ids)
@pytest.mark.parametrize("counts,n,k", [([3, 0, 20], 200, 544), ([300, 1], 10001, 96), ([5, 2], 130, 4128)])
def test_rows_of_no_group_reach_no_result(form, fmt, counts, n, k):
    kw = dict(counts=counts, before=3, behind=40, bias=True, mul=True, residual=True, out=torch.bfloat16, act=fq.ACT_SILU)
    p = Problem(form, fmt, 0, n, k, **kw)
    want, _ = p.run()
    p.check(want, torch.zeros(1, dtype=torch.int32, device=DEV))
    for r in (slice(0, 3), slice(p.m - 40, p.m)):
        if form == "linear":
            p.x[r] = torch.nan
        else:
            p.x[r] = 0xFF
            p.x_scales[r] = 0x7F if fmt == fq.NVFP4 else 255
        p.mul[r] = torch.nan
        p.residual[r] = torch.inf
    got, _ = p.run()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("form,fmt", FORMS, ids=form_ids)
@pytest.mark.parametrize("offsets", [[0, 5, 3, 9], [-1, 2, 3, 9], [0, 2, 3, 10], [0, 2, 2 ** 31 - 1, 9], [9, 0, 0, 0]])
def test_bad_offsets_are_flagged_and_nothing_is_written(form, fmt, offsets):
    p = Problem(form, fmt, 0, 64, 96, counts=[2, 3, 4])
    p.offsets = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    y, st = p.run()
    torch.cuda.synchronize()
    assert int(st.item()) == fq.FLAG_OFFSETS
    assert bool((y == 77.0).all())
    with pytest.raises(fq.Fp4qError):
        fq.check_status(st)


@pytest.mark.parametrize("form,fmt", FORMS, ids=form_ids)
def test_guard_bytes(form, fmt):
    for m, n, k, counts in ((3, 5, 32, None), (67, 131, 96, None), (0, 33, 64, [2, 0, 5])):
        p = Problem(form, fmt, m, n, k, counts=counts, out=torch.bfloat16, exact=True)
        buf = torch.full((p.m * n + 128,), 77.0, dtype=torch.bfloat16, device=DEV)
        y = buf[64:64 + p.m * n].view(p.m, n)
        p.run(y)
        torch.cuda.synchronize()
        assert bool((buf[:64] == 77).all()) and bool((buf[64 + p.m * n:] == 77).all())


@pytest.mark.parametrize("form,fmt", FORMS, ids=form_ids)
@pytest.mark.parametrize("grouped", [False, True])
def test_repeated_calls_two_streams_and_a_graph_agree(form, fmt, grouped):
    kw = dict(counts=[3, 0, 90, 11], behind=2) if grouped else {}
    ps = [Problem(form, fmt, 104, 600, 2080, seed=s, out=torch.bfloat16, bias=True, **kw) for s in (1, 2)]
    want = [p.run()[0] for p in ps]
    torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ys = [torch.full_like(w, 77.0) for w in want]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    for _ in range(20):
        for p, y, s in zip(ps, ys, streams):
            p.run(y, st, stream=s)
    torch.cuda.synchronize()
    for y, w in zip(ys, want):
        assert torch.equal(y, w)
    # one graph with both calls, replayed on other inputs
    graph = torch.cuda.CUDAGraph()
    y2 = [torch.full_like(w, 77.0) for w in want]
    with torch.cuda.graph(graph):
        for p, y in zip(ps, y2):
            p.run(y, st)
    graph.replay()
    torch.cuda.synchronize()
    for y, w in zip(y2, want):
        assert torch.equal(y, w)
    ps[0].x.copy_(ps[1].x)
    other, _ = ps[0].run()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y2[0], other) and not torch.equal(other, want[0])
    assert int(st.item()) == 0


def test_offsets_beyond_32_bits():
    # y has 2^31 + elements, and the weights of the last groups start behind 2^31 bytes
    m, n, k = 70001, 32768, 32
    p = Problem("linear", fq.MXFP4, m, n, k, exact=True, out=torch.bfloat16)
    y, st = p.run()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    w = _decode(p.fmt, p.w_codes[0], p.w_scales[0])
    for r in (0, 65535, 65536, m - 1):
        want = (p.x[r].double() @ w.T).to(torch.bfloat16)
        assert torch.equal(y[r], want), r
    del p, y
    torch.cuda.empty_cache()
    groups, n, k = 130, 4096, 8192
    codes = torch.zeros(groups, n, k // 2, dtype=torch.uint8, device=DEV)
    codes[-1] = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, generator=_gen(3)).to(DEV) & 0x99
    scales = torch.full((groups, n, k // 32), 127, dtype=torch.uint8, device=DEV)
    x = torch.randint(-2, 3, (6, k), generator=_gen(4)).bfloat16().to(DEV)
    off = torch.zeros(groups + 1, dtype=torch.int32, device=DEV)
    off[-1] = 6
    r = fq.linear_group(fq.MXFP4, x, off, codes, fq.mma_scales(scales), out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert int(r.status.item()) == 0
    assert torch.equal(r.y.double(), x.double() @ _decode(fq.MXFP4, codes[-1], scales[-1]).T)


# ------------------------------------------------------------------ with the quantizers, as a model uses them

def _close(got, want, terms, steps):
    """got, want: the same chain, in the library and in 64 bits on the same FP4 values; `terms`: what the outputs sum."""
    off = (got.double() - want).abs()
    tol = steps * 2.0 ** -8 * terms
    assert bool((off <= tol).all()), float((off - tol).max())


def test_a_quantized_layer_equals_its_reconstruction():
    w, x = synth.q_proj(320, 512, seed=1).to(DEV), torch.randn(33, 512, generator=_gen(2)).bfloat16().to(DEV)
    nv, mx = fq.quantize_dual(w.float())
    for fmt, q, S in ((fq.NVFP4, nv, nv.global_scale), (fq.MXFP4, mx, None)):
        r = fq.linear(fmt, x, q.codes, fq.mma_scales(q.scales), S)
        fq.check_status(r.status)
        want = x.double() @ q.deq.double().T
        # the reconstruction rounds q * d once to binary32, the product's sum has 512 + 32 terms: below one more bf16 step
        _close(r.y, want, x.double().abs() @ q.deq.double().abs().T, 1.0)
        tol = want.abs() * 2.0 ** -8 + (512 + 34 + 1) * 2.0 ** -23 * (x.double().abs() @ q.deq.double().abs().T)
        assert bool(((r.y.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("fmt", [fq.NVFP4, fq.MXFP4], ids=NAMES.get)
def test_gated_layer_with_fp4_activations(fmt):
    """gate, up and down projections on activations quantized at every call; MXFP4 rotated, both operands by one mask."""
    tokens, hidden, inner = 50, 256, 672
    masks = {c: torch.from_numpy(synth.sign_masks(c, seed=5).view(np.int32)).to(DEV) for c in (hidden, inner)}

    def quant(t):
        if fmt == fq.NVFP4:
            q = fq.nvfp4_quantize_dynamic(t)
            return q, q.global_scale
        return fq.mxfp4_quantize(t, masks[t.shape[1]]), None

    ws = [quant(synth.q_proj(o, i, seed=o + i + s).to(DEV)) for s, (o, i) in
          enumerate(((inner, hidden), (inner, hidden), (hidden, inner)))]
    tiled = [fq.mma_scales(q.scales) for q, _ in ws]
    x = torch.randn(tokens, hidden, generator=_gen(9)).bfloat16().to(DEV)

    def times(t, i, **kw):
        q, S = quant(t)
        r = fq.matmul(fmt, q.codes, q.scales, S, ws[i][0].codes, tiled[i], ws[i][1], **kw)
        fq.check_status(q.status)
        fq.check_status(r.status)
        S = 1.0 if S is None else float(S) * float(ws[i][1])
        a, w = _decode(fmt, q.codes, q.scales), _decode(fmt, ws[i][0].codes, ws[i][0].scales)
        return r.y, (a @ w.T) * S, (a.abs() @ w.abs().T) * S

    up, want_up, terms = times(x, 1)
    _close(up, want_up, terms, 1.01)
    h, gate, terms = times(x, 0, act=fq.ACT_SILU, mul=up)
    _close(h, _activation(gate, fq.ACT_SILU) * up.double(), 1.13 * terms * up.double().abs() + 1e-3, 1.01)
    y, want, terms = times(h, 2, residual=x)
    _close(y, want + x.double(), terms + x.double().abs(), 1.01)
    # and the layer follows the unquantized one on the weights' values: FP4 keeps about 3 bits of each operand
    if fmt == fq.MXFP4:
        back = [fq.mxfp4_unrotate(q.deq, masks[q.codes.shape[1] * 2]).double() for q, _ in ws]
    else:
        back = [q.deq.double() for q, _ in ws]
    full = _activation(x.double() @ back[0].T, fq.ACT_SILU) * (x.double() @ back[1].T) @ back[2].T
    got = (y.double() - x.double())
    assert float(torch.nn.functional.cosine_similarity(got.flatten(), full.flatten(), dim=0)) > 0.9


@pytest.mark.parametrize("fmt", [fq.NVFP4, fq.MXFP4], ids=NAMES.get)
def test_mixture_of_experts_equals_its_experts_one_by_one(fmt):
    """Rows sorted by expert through the grouped calls, and each expert's rows through the dense ones."""
    experts, hidden, inner, counts = 6, 256, 416, [9, 0, 1, 40, 0, 14]
    ends = np.concatenate([[0], np.cumsum(counts)])
    off = torch.tensor(ends, dtype=torch.int32, device=DEV)
    x = torch.randn(sum(counts), hidden, generator=_gen(1)).bfloat16().to(DEV)
    w = torch.stack([synth.q_proj(inner, hidden, seed=e) for e in range(experts)]).to(DEV)
    qs = [fq.nvfp4_quantize(t) if fmt == fq.NVFP4 else fq.mxfp4_quantize(t) for t in w]
    codes, scales = torch.stack([q.codes for q in qs]), torch.stack([q.scales for q in qs])
    S = torch.cat([q.global_scale for q in qs]) if fmt == fq.NVFP4 else None
    tiled = fq.mma_scales(scales)
    bias = torch.randn(experts, inner, generator=_gen(2)).bfloat16().to(DEV)
    r = fq.linear_group(fmt, x, off, codes, tiled, S, bias=bias, act=fq.ACT_SILU)
    xq = fq.nvfp4_quantize_dynamic(x) if fmt == fq.NVFP4 else fq.mxfp4_quantize(x)
    xS = xq.global_scale if fmt == fq.NVFP4 else None
    r4 = fq.matmul_group(fmt, xq.codes, xq.scales, xS, off, codes, tiled, S, bias=bias, act=fq.ACT_SILU)
    fq.check_status(r.status)
    fq.check_status(r4.status)
    for e in range(experts):
        a, b = int(ends[e]), int(ends[e + 1])
        if a == b:
            continue
        Se = None if S is None else S[e:e + 1]
        one = fq.linear(fmt, x[a:b], codes[e], tiled[e], Se, bias=bias[e], act=fq.ACT_SILU)
        sx = xq.scales[a:b].clone()
        one4 = fq.matmul(fmt, xq.codes[a:b], sx, xS, codes[e], tiled[e], Se, bias=bias[e], act=fq.ACT_SILU)
        # the same sums, perhaps in another order: one bf16 step where a rounding falls the other way
        assert torch.allclose(r.y[a:b].float(), one.y.float(), rtol=2.0 ** -7, atol=1e-3)
        assert torch.allclose(r4.y[a:b].float(), one4.y.float(), rtol=2.0 ** -7, atol=1e-3)
