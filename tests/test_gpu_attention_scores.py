"""spec_verify_attention where whole rows have very negative (or very positive) scores: softmax does not depend on what
all scores of a row have in common.

The bound.  Queries are one power of two in every place, so their low parts are 0 and the products with the codes exact; keys
are -448 in all places but four, where they are multiples of 2^-9 below 16: sums of fewer than 2^15 in steps of 2^-9.  What is
left of a score s (as an exponent of 2) is at most half a step of 32 bits, or a whole one where a sum is truncated, for each
of the 2 D / 32 additions of the product and for the addition of the reference value: (2 D / 32 + 1) * 2^-23 |s|.  The factor of all
scores of a row is off by 2^-23 of itself, which moves the scores beside one another by less than 2^-18 of the 32 that they
spread over.  A weight moves by ln 2 times that, itself and in the sum; the rest is the bound of test_gpu_attention.py:
2^-7 + 2^-11 for the parts of a weight, 2^-13 and `tail` and `peak` for the small ones, 2^-8 for the result."""
import numpy as np
import pytest
import torch

from oracle import operators_oracle as O
from speculative_decoding_verification_34_gb300 import specverify as sv
from tests.test_gpu_attention import SENT, Case

pytestmark = pytest.mark.gpu


def one_sided(seed, lens, size, gmax, Hq, H, D, page, sign=-1.0, **kw):
    """A case whose scores (as exponents of 2) lie about sign * size."""
    c = Case(seed, lens, gmax, Hq, H, D, page, **kw)
    held = c.codes & 0x7F != 0x7F
    keys = np.full(c.codes[0].shape, -448.0)
    # the rest: a spread of about 2 around the common part
    spread = 448.0 * D / size
    keys[..., :4] = np.clip(c.rng.standard_normal(keys[..., :4].shape) * spread, -15, 15)
    c.codes[0] = np.where(held[0], O.e4m3_code(keys), c.codes[0])
    c.codes[1] = np.where(held[1], c.codes[1] & 0x7F, c.codes[1])       # values of one sign: zeros are not an average
    c.exps[0] = np.where(c.exps[0] == 31, 31, -5)
    power = c.rng.integers(-1, 2, (c.B, c.rows, Hq, 1))
    c.q = (torch.from_numpy(2.0 ** power) * -sign * torch.ones(c.B, c.rows, Hq, D)).to(torch.bfloat16)
    c.scale = size / (448 * 2.0 ** -5 * (D - 4) * np.log2(np.e))        # rows of power 0: size
    return c


def check(c, out):
    host = O.Cache(*c.codes, *c.exps)
    for b in range(c.B):
        n = min(max(int(c.num[b]), 0), c.gmax)
        rows = n + (1 if c.root else 0)
        assert (out[b, rows:] == SENT).all(), b
        q = c.q[b, :rows].double().numpy()
        want, bound, _, peak, tail = O.attention(host, c.table[b], int(c.lens[b]), n, q, None if c.parents is None else c.parents[b],
                                                 c.root, c.scale)
        T = int(c.lens[b]) + rows
        s = np.abs(q).max(-1) * 448 * 2.0 ** -5 * c.D * abs(c.scale) * np.log2(np.e)          # the largest |score|
        moved = 2 * np.log(2) * ((2 * c.D / 32 + 1) * 2.0 ** -23 * s + 2.0 ** -18)
        assert moved.max() < 0.6
        rel = 2.0 ** -7 + 2.0 ** -11 + 2.0 ** -13 + np.expm1(moved)[..., None]
        tol = bound * rel + 2.0 ** -3 * tail + np.abs(want) * 2.0 ** -8 + T * 2.0 ** -27.9 * 448 * peak[..., None] + 1e-30
        d = np.abs(out[b, :rows] - want)
        assert (d <= tol).all(), (b, np.argwhere(~(d <= tol))[:4], d.max(), (d / tol).max())


@pytest.mark.parametrize("size", [2000.0, 8000.0, 9950.0, 10100.0, 12000.0, 1e5])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("D,Hq", [(128, 4), (64, 14)])
def test_scores_far_below_zero(size, tree, D, Hq):
    c = one_sided(31, [0, 1, 5, 127, 128, 300, 700], size, 15 if tree else 4, Hq, 2, D, 16, tree=tree)
    out, st = c.run()
    assert st == [0] * c.B
    check(c, out)


def test_scores_far_above_zero():
    c = one_sided(32, [0, 3, 130, 600], 5e4, 4, 4, 2, 128, 32, sign=1.0)
    out, st = c.run()
    assert st == [0] * c.B
    check(c, out)


@pytest.mark.parametrize("Hq,H,L", [(2, 1, 20000), (8, 2, 6000)])
def test_items_shared_by_blocks(Hq, H, L):
    c = one_sided(33, [L, 130], 3e4, 4, Hq, H, 64, 128)
    out, st = c.run()
    assert st == [0, 0]
    check(c, out)


@pytest.mark.parametrize("missing", [8, 9, 24, 30])
@pytest.mark.parametrize("tree", [False, True])
def test_first_pages_missing(missing, tree):
    """A part's first tiles show a row nothing: the first that does sets its reference value, whatever its sign."""
    c = one_sided(34, [200, 500, 480, 512], 4e4, 30 if tree else 6, 4, 2, 128, 16, tree=tree)
    for b in range(c.B):
        c.table[b, : min(missing, int(c.lens[b]) // 16)] = -1
    out, st = c.run()
    assert st == [256] * c.B
    check(c, out)


def test_one_token_of_an_ordinary_scale():
    """One key of -32, one query of 32 in every place, the default scale: a score of -11585; the answer is the value."""
    cache = sv.alloc_kv_cache(1, 1, 16, 128)
    k, v = torch.full((1, 1, 1, 128), -32.0, device="cuda"), torch.linspace(1, 2, 128, device="cuda").view(1, 1, 1, 128)
    table, zero = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    sv.spec_kv_append(k, v, cache, table, zero)
    q = torch.full((1, 1, 1, 128), 32.0, device="cuda", dtype=torch.bfloat16)
    out, key, value = torch.zeros_like(q), torch.zeros_like(v), torch.zeros_like(v)
    sv.spec_verify_attention(q, cache, table, zero, out)
    sv.spec_kv_read(cache, table, None, None, key, value)
    torch.cuda.synchronize()
    assert torch.equal(out.float(), value) and (value > 0.9).all()


def test_a_later_tile_far_above_the_first():
    """Scores that rise by thousands from tile to tile, and fall by as much."""
    for rising in (True, False):
        c = one_sided(35, [900, 400], 3e4, 4, 4, 1, 128, 64)
        pages = c.table.shape[1]
        for b in range(2):
            for g in range(pages):
                at = g if rising else pages - 1 - g
                if c.exps[0, c.table[b, g], 0] != 31:
                    c.exps[0, c.table[b, g]] = -5 - min(at // 2, 5)
        out, _ = c.run()
        check(c, out)
