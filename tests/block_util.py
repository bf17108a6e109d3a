"""Tolerances for the layer norm and linear tests, derived from the arithmetic.

u = 2^-24 bounds the relative error of one fp32 operation; storing in a type t costs at most
half a step, eps(t) / 2 relative to the value (bf16 2^-8, fp32 2^-24). A sum of n terms formed by a
tree whose longest chain is d additions is off by at most d u sum|terms| (first order)."""

import torch

U = 2.0 ** -24


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def assert_within(got, ref, tol, what=""):
    """|got - ref| <= tol element by element (tol a tensor like ref); NaN where ref is NaN."""
    got, ref = got.double(), ref.double()
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    ok = ~(nan | inf)
    bad = (got - ref).abs()[ok] > tol[ok]
    if bad.any():
        worst = ((got - ref).abs()[ok] / tol[ok].clamp_min(1e-300)).max().item()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {worst:.2f} x tolerance")


def strided(rows, cols, pad, offset, dtype, gen, scale=1.0):
    """[rows, cols] normal values whose rows lie cols + pad elements apart, starting `offset`
    elements into their allocation."""
    full = torch.zeros(rows * (cols + pad) + offset + 8, dtype=dtype, device="cuda")
    view = full[offset:].as_strided((rows, cols), (cols + pad, 1)) if rows else full[:0].view(0, 1).expand(0, cols)
    if rows:
        view.copy_(torch.randn((rows, cols), generator=gen, device="cuda") * scale)
    return view


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g
